"""Float64 reference of attention on a mask plan, from the definition, for the GPU tests of fa_fwd_masked and
fa_bwd_masked; its own mask arithmetic (documents as ids, token by token)."""
import math

import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def visible(docs, prefix, N, left, right):
    """[N, N] bool for one sequence: docs a list of offsets, prefix a list or None."""
    ident = torch.full((N,), -1)
    start = torch.zeros(N, dtype=torch.long)
    pre = torch.zeros(N, dtype=torch.long)
    for k, (s, e) in enumerate(zip(docs[:-1], docs[1:])):
        ident[s:e] = k
        start[s:e] = s
        pre[s:e] = prefix[k] if prefix is not None else 0
    i, j = torch.arange(N)[:, None], torch.arange(N)[None]
    seen = (ident[:, None] == ident[None]) & (ident >= 0)[:, None]
    if left >= 0:
        seen &= j >= i - left
    if right >= 0:
        seen &= (j <= i + right) | (j < (start + pre)[None])
    return seen.cuda()


def reference(q, k, v, seen, slopes, sinks, alpha, dout=None):
    """O, LSE, the tolerances' ingredients and (with dout) the gradients, float64.  q [B, N, H, d]; seen: a list of
    [N, N].  Whatever stands in tokens that nobody sees is taken for 0."""
    B, N, H, d = q.shape
    g = H // k.shape[2]
    z = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    r = {"o": z(q), "A": z(q), "lse": torch.zeros(B, H, N, dtype=torch.float64, device="cuda"),
         "dot": torch.zeros(B, H, N, dtype=torch.float64, device="cuda"),
         "far": torch.zeros(B, H, N, dtype=torch.float64, device="cuda"),
         "Afar": z(q)}
    if dout is not None:
        r.update(dq=z(q), dk=z(k), dv=z(v), eq=z(q), ek=z(k), ev=z(v), delta=torch.zeros_like(r["lse"]),
                 edelta=torch.zeros_like(r["lse"]))
    dist = (torch.arange(N)[:, None] - torch.arange(N)[None]).abs().double().cuda()
    for b in range(B):
        live = seen[b].any(0)
        clean = lambda x: torch.where(live[:, None], x.double(), torch.zeros((), dtype=torch.float64, device="cuda"))
        for h in range(H):
            Q, K, V = clean(q[b, :, h]), clean(k[b, :, h // g]), clean(v[b, :, h // g])
            x = alpha * (Q @ K.T)
            bias = torch.zeros_like(x)
            if slopes is not None:
                bias = slopes[h].double() * dist
                x = x - bias
            x = x.masked_fill(~seen[b], -math.inf)
            full = x if sinks is None else torch.cat([x, sinks[h].double().expand(N, 1)], 1)
            lse = torch.logsumexp(full, 1)
            p = torch.where(seen[b], torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]),
                            torch.zeros_like(x))
            o = p @ V
            r["o"][b, :, h], r["A"][b, :, h], r["lse"][b, h] = o, p @ V.abs(), lse
            # a score's error: d steps of the dot product; of the bias, its size
            dot = (Q.abs() @ K.abs().T * alpha).masked_fill(~seen[b], 0.0)
            r["dot"][b, h] = dot.max(1).values
            far = bias.abs().masked_fill(~seen[b], 0.0)
            r["far"][b, h] = (p * far).sum(1)
            r["Afar"][b, :, h] = (p * far) @ V.abs()
            if dout is None:
                continue
            G = clean(dout[b, :, h])
            dp = G @ V.T
            D = (G * o).sum(1, keepdim=True)
            ds = p * (dp - D)
            r["dq"][b, :, h] = alpha * ds @ K
            r["dk"][b, :, h // g] += alpha * ds.T @ Q
            r["dv"][b, :, h // g] += p.T @ G
            # sizes for the tolerances: relative errors of p reach ds through |dp| + |D|, those of O through D
            size = p * (dp.abs() + (G.abs() * o.abs()).sum(1, keepdim=True))
            r["eq"][b, :, h] = alpha * size @ K.abs()
            r["ek"][b, :, h // g] += alpha * size.T @ Q.abs()
            r["ev"][b, :, h // g] += p.T @ G.abs()
            r["delta"][b, h], r["edelta"][b, h] = D[:, 0], (G.abs() * o.abs()).sum(1)
    return r


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def check_forward(o, lse, r, dt, d, alpha, slopes):
    u = U[dt]
    # the score's error; with a bias the FP32 steps of its addition (see test_masked_gpu.py)
    e = d * 2.0 ** -23 * r["dot"] + 2.0 ** -20
    if slopes is not None:
        e = e + 24 * 2.0 ** -24 * (r["far"] + r["lse"].abs().nan_to_num(posinf=0.0) + 8)
    e_rows = e.transpose(1, 2)[..., None]
    tol = 1.05 * (u * (r["A"] + 2 * r["o"].abs()) + 2 * e_rows * r["A"]) + 2.0 ** -24
    bad = (o.double() - r["o"]).abs() > tol
    assert not bad.any(), ("O", int(bad.sum()), float((o.double() - r["o"]).abs().max()))
    dead = torch.isinf(r["lse"])
    assert torch.equal(torch.isinf(lse), dead) and (lse[dead] < 0).all()
    err = (lse.double() - r["lse"]).abs()[~dead]
    lim = (e + 2.0 ** -22 * r["lse"].abs())[~dead]
    assert (err <= lim).all(), ("LSE", float((err / lim).max()))
    assert (o.double().abs().amax(-1)[dead.transpose(1, 2)] == 0).all()


def check_backward(got, r, dt, d, slopes):
    """Tolerances in test_masked_bwd_gpu.py."""
    u = U[dt]
    far = 0.0 if slopes is None else 48 * 2.0 ** -24 * float((r["far"] + r["lse"].abs().nan_to_num(posinf=0.0)).max() + 8)
    e = 2 * d * 2.0 ** -23 * float(r["dot"].max()) + 2.0 ** -18 + far
    worst = {}
    for name, x, size, rounds in (("dq", got[0], r["eq"], 2), ("dk", got[1], r["ek"], 2), ("dv", got[2], r["ev"], 1)):
        tol = 1.05 * (rounds * u + e) * size + u * r[name].abs() + 2.0 ** -24
        off = (x.double() - r[name]).abs()
        assert not (off > tol).any(), (name, int((off > tol).sum()), float((off / tol).max()))
        worst[name] = float((off / tol).max())
    return worst
