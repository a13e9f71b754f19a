"""GPU checks of the distance bias far from the diagonal, where it is large and the weights are not small: slopes below 0,
whose weights lie on the farthest keys (a positive slope's lie on the nearest).  Against float64.

What FP32 leaves, per element, with u the half step of the 16-bit type, s the slope's size and L the largest |LSE|:

* a score less the reference (or the LSE) is rounded at its own size: it is a dot product (d 2^-23 alpha sum |q||k|), the
  bias within a tile in 16 additions and a start of quantities of at most 128 s, and what the tile's distance adds to the
  reference in one FMA: 20 2^-24 128 s; exp2, the sums and the rest 2^-20.  The bias of far tiles itself is not rounded;
* LSE: its reference, the sum's logarithm and the change of base round at L, and the slope in log2 units is off by
  1.5 2^-24 of itself: 5 2^-24 L.  Parts of a row joined through their LSE (the paged cache): 3 2^-24 L each way;
* the backward's P = exp(S - LSE), here from the LSE that it is given: its change of base rounds at L, the slope as
  above times the distance (at most L + max |alpha q k| off): 4 2^-24 L;
* fp16 is spaced by 2^-24 below 2^-14: P and dS are off by 2^-25 there, whatever their size, so that the products lose
  as much of the sum of what they weigh.
The rest as in test_masked_gpu.py and test_masked_bwd_gpu.py."""
import math

import pytest
import torch

import exact_attention_forward_fa_gb300 as fa
from tests._masked import DT, U

pytestmark = pytest.mark.gpu

SLOPES = (-0.7, -0.031, -2.9)


def exact(q, k, v, s, alpha, seen, dist):
    """Scores, LSE, P and O of one head in float64, the largest sum of a score's products."""
    x = alpha * (q.double() @ k.double().T) - float(torch.tensor(s, dtype=torch.float32)) * dist
    x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    return x, lse, p, p @ v.double(), alpha * float((q.double().abs() @ k.double().abs().T).max())


def tolerance(d, dot, s):
    return d * 2.0 ** -23 * dot + 2.0 ** -20 + 20 * 2.0 ** -24 * 128 * abs(s)


@pytest.mark.parametrize("right", [0, -1])
@pytest.mark.parametrize("d,dt", [(64, "fp16"), (128, "fp16"), (64, "bf16"), (128, "bf16")])
def test_masked(gpu_lib, d, dt, right):
    N, H, lo, hi = 12000, len(SLOPES), 101, 11990
    g = torch.Generator("cuda").manual_seed(d)
    q, k = (torch.randn(1, N, H, d, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
    # values and gradients of one sign: errors that P's elements share do not average out
    v, do = ((0.5 + torch.rand(1, N, H, d, generator=g, device="cuda")).to(DT[dt]) for _ in range(2))
    slopes = torch.tensor(SLOPES, dtype=torch.float32, device="cuda")
    plan = fa.mask_plan(torch.tensor([[lo, hi]], dtype=torch.int32, device="cuda"), N, window=(-1, right))
    o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes)
    dq, dk, dv, _ = fa.attention_backward_masked(q, k, v, o, lse, do, plan, slopes=slopes)
    assert fa.fa_check_status() == fa.FA_OK
    u, alpha, n = U[dt], 1 / math.sqrt(d), slice(lo, hi)
    i = torch.arange(hi - lo, device="cuda")
    dist = (i[:, None] - i[None]).abs().double()
    seen = i[None] <= i[:, None] if right == 0 else torch.ones_like(dist, dtype=torch.bool)
    for h, s in enumerate(SLOPES):
        Q, K, V, G = (x[0, n, h] for x in (q, k, v, do))
        x, want, p, wo, dot = exact(Q, K, V, s, alpha, seen, dist)
        L = float(want.abs().max())
        e = tolerance(d, dot, s)
        err = (lse[0, h, n].double() - want).abs().max()
        assert err <= e + 5 * 2.0 ** -24 * L, ("LSE", s, float(err))
        A = p @ V.double().abs()
        off = (o[0, n, h].double() - wo).abs() / (1.05 * (u * (A + 2 * wo.abs()) + 2 * e * A) + 2.0 ** -24)
        assert off.max() <= 1, ("O", s, float(off.max()))
        # the gradients for the LSE and O that the backward gets
        e += 4 * 2.0 ** -24 * L
        p = torch.exp(x - lse[0, h, n].double()[:, None])
        G, V, K, Q, O = (t.double() for t in (G, V, K, Q, o[0, n, h]))
        D = (G * O).sum(1, keepdim=True)
        dp = G @ V.T
        ds = p * (dp - D)
        size = p * (dp.abs() + (G * O).abs().sum(1, keepdim=True))
        del dp
        low, all_seen = (2.0 ** -25 if dt == "fp16" else 0.0), seen.double()
        for name, got, w, a, r, z in (
                ("dv", dv, p.T @ G, p.T @ G.abs(), 1, all_seen.T @ G.abs()),
                ("dq", dq, alpha * ds @ K, alpha * size @ K.abs(), 2, alpha * all_seen @ K.abs()),
                ("dk", dk, alpha * ds.T @ Q, alpha * size.T @ Q.abs(), 2, alpha * all_seen.T @ Q.abs())):
            off = (got[0, n, h].double() - w).abs() / (1.05 * (r * u + e) * a + u * w.abs() + 2.0 ** -24 + low * z)
            assert off.max() <= 1, (name, s, float(off.max()))
    assert not o[0, :lo].any() and not o[0, hi:].any() and not dv[0, :lo].any() and not dk[0, hi:].any()


@pytest.mark.parametrize("d,dt", [(64, "fp16"), (128, "bf16")])
def test_paged(gpu_lib, d, dt):
    """Single tokens and chunks over a long cache, in both directions for the chunks."""
    H, ps = len(SLOPES), 64
    kv, new = [12000, 11111], [1, 300]
    g = torch.Generator("cuda").manual_seed(d + 1)
    u, alpha = U[dt], 1 / math.sqrt(d)
    slopes = torch.tensor(SLOPES, dtype=torch.float32, device="cuda")
    W = -(-max(kv) // ps)
    table = torch.arange(2 * W, dtype=torch.int32, device="cuda").reshape(2, W)
    k_pages = torch.randn(2 * W, ps, H, d, generator=g, device="cuda").to(DT[dt])
    v_pages = (0.5 + torch.rand(2 * W, ps, H, d, generator=g, device="cuda")).to(DT[dt])
    kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
    for lens, window in ((new, (-1, 0)), ([1, 1], (-1, 0)), (new, (-1, -1)), ([0, 300], (5000, 40))):
        T = sum(lens)
        q = torch.randn(T, H, d, generator=g, device="cuda").to(DT[dt])
        cu = torch.tensor([0, lens[0], T], dtype=torch.int32, device="cuda")
        o, lse = fa.attention_paged(q, k_pages, v_pages, table, kv_len, cu, max_q=max(lens), window=window, slopes=slopes)
        assert fa.fa_check_status() == fa.FA_OK
        for b, m in enumerate(lens):
            if m == 0:
                continue
            rows = slice(0, m) if b == 0 else slice(lens[0], T)
            pos = torch.arange(kv[b] - m, kv[b], device="cuda")
            j = torch.arange(kv[b], device="cuda")
            dist = (pos[:, None] - j[None]).abs().double()
            seen = torch.ones_like(dist, dtype=torch.bool)
            if window[0] >= 0:
                seen &= j[None] >= pos[:, None] - window[0]
            if window[1] >= 0:
                seen &= j[None] <= pos[:, None] + window[1]
            for h, s in enumerate(SLOPES):
                K, V = (x[table[b].long()].reshape(-1, H, d)[:kv[b], h] for x in (k_pages, v_pages))
                _, want, p, wo, dot = exact(q[rows, h], K, V, s, alpha, seen, dist)
                L = float(want.abs().max())
                e = tolerance(d, dot, s) + 3 * 2.0 ** -24 * L
                err = (lse[h, rows].double() - want).abs().max()
                assert err <= e + 5 * 2.0 ** -24 * L, ("LSE", lens, window, s, float(err))
                A = p @ V.double().abs()
                off = (o[rows, h].double() - wo).abs() / (1.05 * (u * (A + 2 * wo.abs()) + 2 * e * A) + 2.0 ** -24)
                assert off.max() <= 1, ("O", lens, window, s, float(off.max()))
