"""Rotary positions, masked attention over packed documents, and their serving forms, as measured work: cases over
their real range, their plain forms in elementary torch operations, and their values in 64 bits.

Rotary: pair c of a token at position p turns by the angle p * inv_freq[c], times a scale.  Half layout: pair c is
(x[c], x[c + rot / 2]); interleaved: (x[2c], x[2c + 1]); components from `rot` on stay.

Masked attention: sequence b is packed with documents docs[b, k] .. docs[b, k + 1].  Token i of document [s, e) whose
first p tokens are its prefix sees key j when max(s, i - left) <= j < min(e, max(i + 1 + right, s + p)) (a bound of -1:
none); the score is alpha q.k - slope_h |i - j|.  Tokens outside every document see nothing and are not seen.

The paged cache is that of perf/operators.py.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, dtype="bf16", d=128, H=32, H_kv=8, B=1, N=1, lens=0, **more):
    c = {"name": name, "op": op, "dtype": dtype, "d": d, "H": H, "H_kv": H_kv, "B": B, "N": N, "lens": lens,
         # rotary
         "rot": 128, "interleaved": False, "scaling": "none", "factor": 1.0, "far": 0,
         # documents of doc_min .. doc_max tokens, pad tokens behind the last, prefixes up to a part of the document
         "doc_min": 0, "doc_max": 0, "pad": 0, "prefix": 0.0, "left": -1, "right": 0, "bias": False,
         # paged cache
         "page": 16, "q_min": 1, "q_max": 1, "kv_min": 1, "kv_max": 1}
    c.update(more)
    return c


def listed():
    return [
        # queries and keys of a training step's layer, slices of its fused projection
        _case("rotate_train_b4", "rotate", H=16, H_kv=16, B=4, N=4096, lens=1),
        # the gradient's way back: interleaved pairs of half the head, positions far into a context that was stretched
        _case("rotate_grad_part", "unrotate", "fp16", B=2, N=3001, lens=2, rot=64, interleaved=True, scaling="yarn",
              factor=16.0, far=1 << 20, doc_min=100, doc_max=1500),
        # one new token for each of a serving batch: pure latency
        _case("rotate_append_b64", "rotate_append", B=64, lens=3, kv_min=512, kv_max=8192),
        # a prompt's chunks, their rows slices of a fused projection; the cache was cut, positions run on
        _case("rotate_append_chunks_b4", "rotate_append", "fp16", B=4, lens=4, page=64, q_min=1500, q_max=4096,
              kv_min=4096, kv_max=16384, far=100000, scaling="linear", factor=4.0),
        # a small fine-tuning batch: short documents, padded behind
        _case("documents_short", "attend", "fp16", d=64, H=8, H_kv=8, B=2, N=1000, lens=5, doc_min=20, doc_max=300, pad=60),
        # the ordinary pre-training layer: sequences packed with documents, grouped heads
        _case("documents_train", "attend", B=2, N=8192, lens=6, doc_min=200, doc_max=4000),
        # prefixes that see themselves in both directions, heads of 64
        _case("prefix_d64", "attend", "fp16", d=64, H=32, H_kv=32, B=4, N=4001, lens=7, doc_min=1500, doc_max=4000, prefix=0.7),
        # one long document with a bias that grows with the distance: the largest forward
        _case("distance_long", "attend", H=16, H_kv=16, N=16384, lens=8, doc_min=16384, doc_max=16384, bias=True),
        # the gradients of the ordinary layer: the largest
        _case("documents_grad", "grad", B=2, N=8192, lens=9, doc_min=200, doc_max=4000),
        # the gradients with a bias in both directions, a window and odd sizes
        _case("distance_grad_d64", "grad", "fp16", d=64, H=12, H_kv=4, B=3, N=3001, lens=10, doc_min=300, doc_max=3001, pad=1,
              left=1000, right=-1, bias=True),
        # a decoding step of a model with the distance bias
        _case("distance_tokens_b64", "attend_paged", B=64, lens=11, kv_min=512, kv_max=8192, bias=True),
        # a scheduler's mixed step of the same: prompt chunks beside decoding sequences
        _case("distance_mixed_b24", "attend_paged", "fp16", B=24, lens=12, page=32, q_min=1, q_max=300, kv_min=301,
              kv_max=4096, bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "unrotate", "rotate_append", "attend", "attend", "grad", "grad", "attend_paged"])
    H, H_kv = rng.choice([(32, 8), (16, 16), (16, 2), (8, 1), (12, 4), (24, 8), (32, 4)])
    d = rng.choice([64, 128])
    m = {"lens": rng.randrange(1 << 20)}
    if op in ("rotate", "unrotate", "rotate_append"):
        m["rot"] = rng.choice([d, d, d // 2, d // 4])
        m["interleaved"] = rng.random() < 0.5
        m["scaling"] = rng.choice(["none", "linear", "ntk", "yarn"])
        m["factor"] = rng.choice([2.0, 4.0, 8.0, 16.0]) if m["scaling"] != "none" else 1.0
        m["far"] = rng.choice([0, 0, 1000, 1 << 20])
    if op in ("rotate", "unrotate", "attend", "grad"):
        B = rng.randint(1, 4)
        N = _log_int(rng, 60, 5000 // B if op == "grad" else 8000 // B)
        m["doc_max"] = _log_int(rng, 16, N)
        m["doc_min"] = rng.randint(1, m["doc_max"])
    else:
        B = _log_int(rng, 1, 48)
        N = 1
        m["page"] = rng.choice([16, 32, 64, 128])
        m["kv_max"] = _log_int(rng, 200, min(16384 if B <= 4 else 6000, int(1.1e9 / (4 * B * H_kv * d))))
        m["kv_min"] = rng.randint(max(1, m["kv_max"] // 8), m["kv_max"])
        if rng.random() < 0.6:
            m["q_max"] = min(m["kv_min"], _log_int(rng, 2, 700 if B <= 3 else 250 if B <= 12 else 40))
            m["q_min"] = rng.randint(1, m["q_max"])
    if op in ("attend", "grad"):
        m["pad"] = rng.choice([0, 0, rng.randint(1, N // 4)])
        m["prefix"] = rng.choice([0.0, 0.0, 0.5, 1.0])
        m["right"] = rng.choice([0, 0, -1])
        m["left"] = rng.choice([-1, -1, _log_int(rng, 16, N)])
    if op in ("attend", "grad", "attend_paged"):
        m["bias"] = op == "attend_paged" or rng.random() < 0.5
    c = _case("", op, rng.choice(["bf16", "fp16"]), d, H, H_kv, B, N, **m)
    del c["name"]
    return c


# ---- what a case's numbers stand for (ragged, fixed by the case) ----

def _documents(c):
    """Offsets [B, D + 1] of the documents and their prefixes [B, D] (rows with fewer end in empty documents)."""
    r = random.Random(2000 + c["lens"])
    rows, prefixes = [], []
    for _ in range(c["B"]):
        end, at, p = c["N"] - c["pad"], [0], []
        while at[-1] < end:
            n = min(r.randint(max(1, c["doc_min"]), max(1, c["doc_max"])), end - at[-1])
            at.append(at[-1] + n)
            p.append(r.randint(0, int(c["prefix"] * n)))
        rows.append(at)
        prefixes.append(p)
    D = max(len(p) for p in prefixes)
    docs = [at + [at[-1]] * (D + 1 - len(at)) for at in rows]
    return np.array(docs, dtype=np.int32), np.array([p + [0] * (D - len(p)) for p in prefixes], dtype=np.int32)


def _intervals(c):
    """First visible key and one past the last of every token, [B, N] each (both 0 outside the documents)."""
    docs, prefix = _documents(c)
    lo = np.zeros((c["B"], c["N"]), dtype=np.int64)
    hi = np.zeros_like(lo)
    for b in range(c["B"]):
        for s, e, p in zip(docs[b, :-1], docs[b, 1:], prefix[b]):
            i = np.arange(s, e)
            lo[b, s:e] = np.maximum(s, i - c["left"]) if c["left"] >= 0 else s
            hi[b, s:e] = np.minimum(e, np.maximum(i + 1 + c["right"], s + p)) if c["right"] >= 0 else e
    return lo, hi


def _lens(c):
    """The new tokens and cached tokens of each sequence of a paged case."""
    r = random.Random(1000 + c["lens"])
    kv = [r.randint(c["kv_min"], c["kv_max"]) for _ in range(c["B"])]
    pick = _log_int if c["q_max"] > 10 * c["q_min"] else random.Random.randint
    return [min(pick(r, c["q_min"], c["q_max"]), n) for n in kv], kv


def _frequencies(c):
    """Radians a position for each pair, in 64 bits, and the factor of the rotated values."""
    rot, base, f = c["rot"], 10000.0, c["factor"]
    i = torch.arange(0, rot, 2, dtype=torch.float64) / rot
    w = base ** -i
    if c["scaling"] == "linear":
        return w / f, 1.0
    if c["scaling"] == "ntk":
        return (base * f ** (rot / (rot - 2))) ** -i, 1.0
    if c["scaling"] == "yarn":
        # pairs that turn more than 32 times within the first 4096 positions stay, those below one turn are stretched
        edge = [rot * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
        k = torch.arange(rot // 2, dtype=torch.float64)
        keep = 1.0 - ((k - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return w / f * (1 - keep) + w * keep, 0.1 * math.log(f) + 1.0
    return w, 1.0


def _slopes(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    H, Hk, d, B, N, t = c["H"], c["H_kv"], c["d"], c["B"], c["N"], DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(t)

    s = {"case": c, "alpha": 1.0 / math.sqrt(d), "slopes": _slopes(H) if c["bias"] else None}
    if c["op"] in ("rotate", "unrotate", "rotate_append"):
        freq, s["scale"] = _frequencies(c)
        s["inv_freq"] = freq.to(dev)
    if c["op"] in ("rotate", "unrotate"):
        s["positions"] = None
        if c["far"] or c["doc_max"]:
            # positions that begin anew with every document, somewhere in a long context
            docs = _documents(c)[0]
            at = np.stack([np.arange(N) - row[np.searchsorted(row, np.arange(N), side="right") - 1] for row in docs])
            s["positions"] = torch.tensor(at + c["far"], dtype=torch.int32, device=dev)
        if c["op"] == "rotate":
            rows = normal(B, N, H + 2 * Hk, d)
            s["q"], s["k"] = rows[:, :, :H], rows[:, :, H:H + Hk]
        else:
            s["q"], s["k"] = normal(B, N, H, d), normal(B, N, Hk, d)
        s["q_out"] = torch.empty((B, N, H, d), dtype=t, device=dev)
        s["k_out"] = torch.empty((B, N, Hk, d), dtype=t, device=dev)
        return s
    if c["op"] in ("attend", "grad"):
        docs, prefix = _documents(c)
        s["docs"] = torch.tensor(docs, device=dev)
        s["prefix"] = torch.tensor(prefix, device=dev) if c["prefix"] else None
        s["q"], s["k"], s["v"] = normal(B, N, H, d), normal(B, N, Hk, d), normal(B, N, Hk, d)
        if own:
            import exact_attention_forward_fa_gb300 as fa
            # the layers of a step share the plan of its batch
            s["plan"] = fa.mask_plan(s["docs"], N, prefix=s["prefix"], window=(c["left"], c["right"]))
        if c["op"] == "grad":
            s["o"], s["lse"] = _plain_attend(s)
            s["dout"] = normal(B, N, H, d)
        else:
            s["out"] = torch.empty((B, N, H, d), dtype=t, device=dev)
            s["lse"] = torch.empty((B, H, N), dtype=torch.float32, device=dev)
        return s
    q_len, kv = _lens(c)
    T, ps = sum(q_len), c["page"]
    pages = [-(-n // ps) for n in kv]
    perm = torch.randperm(sum(pages) + 3, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    s.update(table=table, ps=ps, q_max=max(q_len), k_pages=normal(len(perm), ps, Hk, d), v_pages=normal(len(perm), ps, Hk, d),
             kv_len=torch.tensor(kv, dtype=torch.int32, device=dev),
             cu_q=torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device=dev))
    if c["op"] == "rotate_append":
        rows = normal(T, H + 2 * Hk, d)
        s["q"], s["k"], s["v"] = rows[:, :H], rows[:, H:H + Hk], rows[:, H + Hk:]
        s["q_out"] = torch.empty((T, H, d), dtype=t, device=dev)
        # how far the positions of a cut cache run ahead of its lengths
        r = random.Random(3000 + c["lens"])
        s["offsets"] = (torch.tensor([r.randint(0, c["far"]) for _ in kv], dtype=torch.int32, device=dev)
                        if c["far"] else None)
    else:
        s["q"] = normal(T, H, d)
        s["out"] = torch.empty((T, H, d), dtype=t, device=dev)
        s["lse"] = torch.empty((H, T), dtype=torch.float32, device=dev)
    return s


# ---- the plain forms ----

def _plain_turn(x, pos, s, back=False):
    """x [..., heads, d] at positions pos [...], in float32; the angles in 64 bits."""
    rot = s["case"]["rot"]
    a = pos.double()[..., None] * s["inv_freq"]
    cos = (torch.cos(a) * s["scale"]).float()[..., None, :]
    sin = (torch.sin(a) * (-s["scale"] if back else s["scale"])).float()[..., None, :]
    y = x.float().clone()
    if s["case"]["interleaved"]:
        u, w = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = u * cos - w * sin, w * cos + u * sin
    else:
        u, w = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = u * cos - w * sin, w * cos + u * sin
    return y.to(x.dtype)


def _plain_rotate(s):
    c = s["case"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(c["N"], device=s["q"].device).expand(c["B"], c["N"])
    back = c["op"] == "unrotate"
    return _plain_turn(s["q"], pos, s, back), _plain_turn(s["k"], pos, s, back)


def _padded(s):
    """Row index, validity, sequence and position of every (sequence, new token)."""
    cu = s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["q_max"], device=cu.device)
    ok = i[None] < n[:, None]
    pos = (s["kv_len"].long() - n)[:, None] + i[None]
    row = torch.where(ok, cu[:-1, None] + i[None], torch.zeros_like(pos))
    return row, ok, pos


def _plain_rotate_append(s):
    row, ok, pos = _padded(s)
    b = torch.arange(ok.shape[0], device=ok.device)[:, None].expand_as(ok)[ok]
    p, row = pos[ok], row[ok]
    at = p if s["offsets"] is None else p + s["offsets"].long()[b]
    s["q_out"][row] = _plain_turn(s["q"][row], at, s)
    page, slot = s["table"].long()[b, p // s["ps"]], p % s["ps"]
    s["k_pages"][page, slot] = _plain_turn(s["k"][row], at, s)
    s["v_pages"][page, slot] = s["v"][row]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _seen(s, b):
    """[N, N]: whether token i of sequence b sees token j."""
    c, dev = s["case"], s["q"].device
    i = torch.arange(c["N"], device=dev)
    docs = s["docs"][b].long()
    k = torch.searchsorted(docs, i, right=True) - 1                # the last offset at or before i
    k = k.clamp(0, docs.numel() - 2)
    k = torch.where(i < docs[k + 1], k, torch.full_like(k, -1))    # -1: outside
    start = docs[k.clamp(min=0)]
    seen = (k[:, None] == k[None]) & (k >= 0)[:, None]
    if c["left"] >= 0:
        seen &= i[None] >= i[:, None] - c["left"]
    if c["right"] >= 0:
        ahead = i[None] <= i[:, None] + c["right"]
        if s["prefix"] is not None:
            ahead |= i[None] < (start + s["prefix"][b].long()[k.clamp(min=0)])[None]
        seen &= ahead
    return seen


def _plain_scores(s, b, h, seen, dist):
    g = s["case"]["H"] // s["case"]["H_kv"]
    x = torch.matmul(s["q"][b, :, h].float(), s["k"][b, :, h // g].float().T) * s["alpha"]
    if s["slopes"] is not None:
        x = x - s["slopes"][h] * dist
    return torch.where(seen, x, torch.full_like(x, -math.inf))


def _distance(s, N):
    i = torch.arange(N, device=s["q"].device, dtype=torch.float32)
    return (i[:, None] - i[None]).abs() if s["slopes"] is not None else None


def _plain_attend(s):
    c = s["case"]
    g = c["H"] // c["H_kv"]
    out = torch.empty_like(s["q"])
    lse = torch.empty((c["B"], c["H"], c["N"]), dtype=torch.float32, device=out.device)
    dist = _distance(s, c["N"])
    for b in range(c["B"]):
        seen = _seen(s, b)
        for h in range(c["H"]):
            x = _plain_scores(s, b, h, seen, dist)
            top = x.amax(-1, keepdim=True)
            top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
            e = torch.exp(x - top)
            total = e.sum(-1, keepdim=True)
            o = torch.matmul(e, s["v"][b, :, h // g].float())
            out[b, :, h] = (o / torch.where(total > 0, total, torch.ones_like(total))).to(out.dtype)
            lse[b, h] = (torch.log(total) + top)[:, 0]
    return out, lse


def _plain_grad(s):
    c = s["case"]
    g = c["H"] // c["H_kv"]
    dq, dk, dv = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    dist = _distance(s, c["N"])
    for b in range(c["B"]):
        seen = _seen(s, b)
        for hk in range(c["H_kv"]):
            k, v = s["k"][b, :, hk].float(), s["v"][b, :, hk].float()
            sum_k, sum_v = torch.zeros_like(k), torch.zeros_like(v)
            for h in range(hk * g, hk * g + g):
                x = _plain_scores(s, b, h, seen, dist)
                p = torch.exp(torch.where(seen, x - s["lse"][b, h][:, None], x))
                do = s["dout"][b, :, h].float()
                sum_v += torch.matmul(p.T, do)
                delta = (do * s["o"][b, :, h].float()).sum(-1, keepdim=True)
                ds = p * (torch.matmul(do, v.T) - delta) * s["alpha"]
                dq[b, :, h] = torch.matmul(ds, k).to(dq.dtype)
                sum_k += torch.matmul(ds.T, s["q"][b, :, h].float())
            dk[b, :, hk], dv[b, :, hk] = sum_k.to(dk.dtype), sum_v.to(dv.dtype)
    return dq, dk, dv


def _gathered(s, pages):
    """[B, H_kv, L, d] float32 of a cache, by its block table; nothing behind kv_len."""
    x = pages[s["table"].long().clamp(min=0)].float()          # [B, W, ps, H_kv, d]
    x = x.reshape(x.shape[0], -1, x.shape[3], x.shape[4])
    j = torch.arange(x.shape[1], device=x.device)
    x = torch.where((j[None] < s["kv_len"][:, None])[:, :, None, None], x, torch.zeros_like(x))
    return x.transpose(1, 2).contiguous()


def _plain_attend_paged(s):
    c = s["case"]
    row, ok, pos = _padded(s)
    k, v = _gathered(s, s["k_pages"]), _gathered(s, s["v_pages"])
    B, Hk, L, d = k.shape
    Q, H = row.shape[1], c["H"]
    q = s["q"].float()[row].reshape(B, Q, Hk, H // Hk, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(B, Hk, -1, d), k.transpose(2, 3)).reshape(B, Hk, H // Hk, Q, L) * s["alpha"]
    j = torch.arange(L, device=x.device)
    dist = (pos[:, :, None] - j).float()
    x = x - s["slopes"].reshape(1, Hk, H // Hk, 1, 1) * dist[:, None, None]
    seen = (j <= pos[:, :, None]) & ok[:, :, None]
    x = torch.where(seen[:, None, None], x, torch.full_like(x, -math.inf))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(-1)
    o = torch.matmul(e.reshape(B, Hk, -1, L), v).reshape(B, Hk, H // Hk, Q, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    out[row[ok]] = o.permute(0, 3, 1, 2, 4).reshape(B, Q, H, d)[ok].to(out.dtype)
    lse[:, row[ok]] = (torch.log(total) + top[..., 0]).permute(1, 2, 0, 3).reshape(H, B, Q)[:, ok]
    return out, lse


def _own(s):
    import exact_attention_forward_fa_gb300 as fa
    c, op = s["case"], s["case"]["op"]
    if op in ("rotate", "unrotate"):
        return fa.rope(s["q"], s["k"], s["inv_freq"], positions=s["positions"], scale=s["scale"],
                       interleaved=c["interleaved"], inverse=op == "unrotate", q_out=s["q_out"], k_out=s["k_out"])
    if op == "rotate_append":
        q = fa.paged_rope_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["kv_len"], s["cu_q"],
                                 s["inv_freq"], scale=s["scale"], interleaved=c["interleaved"], offsets=s["offsets"],
                                 q_out=s["q_out"])
        return q, s["k_pages"], s["v_pages"]
    if op == "attend":
        return fa.attention_masked(s["q"], s["k"], s["v"], s["plan"], slopes=s["slopes"], alpha=s["alpha"], out=s["out"],
                                   lse=s["lse"])
    if op == "grad":
        return fa.attention_backward_masked(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], s["plan"],
                                            slopes=s["slopes"], alpha=s["alpha"])[:3]
    return fa.attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_len"], s["cu_q"], max_q=s["q_max"],
                              alpha=s["alpha"], out=s["out"], lse=s["lse"], slopes=s["slopes"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    plain = {"rotate": _plain_rotate, "unrotate": _plain_rotate, "rotate_append": _plain_rotate_append,
             "attend": _plain_attend, "grad": _plain_grad, "attend_paged": _plain_attend_paged}
    return plain[op](state)


def work(case):
    c = case
    H, Hk, d, BN = c["H"], c["H_kv"], c["d"], c["B"] * c["N"]
    if c["op"] in ("rotate", "unrotate"):
        return {"bytes": 4 * BN * (H + Hk) * d + (4 * BN if c["far"] or c["doc_max"] else 0),
                "flops": 3 * BN * (H + Hk) * c["rot"]}
    if c["op"] in ("attend", "grad"):
        lo, hi = _intervals(c)
        pairs = int((hi - lo).sum()) * H
        if c["op"] == "attend":
            return {"bytes": 4 * BN * (H + Hk) * d + 4 * BN * H, "flops": 4 * d * pairs}
        return {"bytes": 2 * BN * d * (4 * H + 4 * Hk) + 4 * BN * H, "flops": 10 * d * pairs}
    q_len, kv = _lens(c)
    T = sum(q_len)
    if c["op"] == "rotate_append":
        return {"bytes": 4 * T * d * (H + 2 * Hk), "flops": 3 * T * (H + Hk) * c["rot"]}
    pairs = sum(n - m + i + 1 for m, n in zip(q_len, kv) for i in range(m)) * H
    return {"bytes": 4 * T * H * d + 4 * T * H + 4 * sum(kv) * Hk * d, "flops": 4 * d * pairs}


# ---- the values in 64 bits ----

def _exact_turn(x, pos, freq, scale, rot, interleaved, sign):
    """Each pair as a complex number times scale e^(i angle)."""
    turn = torch.polar(torch.full_like(pos.double()[..., None] * freq, scale), sign * pos.double()[..., None] * freq)
    x = x.double().clone()
    part = x[..., :rot]
    z = (torch.complex(part[..., 0::2], part[..., 1::2]) if interleaved
         else torch.complex(part[..., :rot // 2], part[..., rot // 2:]))
    z = z * turn[..., None, :]
    y = torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
    x[..., :rot] = y
    return x


def _exact_block(s, b, h, lo, hi, x0, x1):
    """Logits in 64 bits of rows [x0, x1) of sequence b against keys [x0, x1), -inf where unseen."""
    c = s["case"]
    hk = h // (c["H"] // c["H_kv"])
    x = s["alpha"] * (s["q"][b, x0:x1, h].double() @ s["k"][b, x0:x1, hk].double().T)
    j = torch.arange(x0, x1, device=x.device)
    if s["slopes"] is not None:
        x -= s["slopes"][h].double() * (j[:, None] - j[None]).abs().double()
    return x.masked_fill((j[None] < lo[b, x0:x1, None]) | (j[None] >= hi[b, x0:x1, None]), -math.inf), hk


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("rotate", "unrotate", "rotate_append"):
        how = (s["inv_freq"], s["scale"], c["rot"], c["interleaved"], -1.0 if c["op"] == "unrotate" else 1.0)
        if c["op"] != "rotate_append":
            pos = s["positions"] if s["positions"] is not None else torch.arange(c["N"], device="cuda").repeat(c["B"], 1)
            return _exact_turn(s["q"], pos, *how), _exact_turn(s["k"], pos, *how)
        q, k, v = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda"), s["k_pages"].double(), s["v_pages"].double()
        at = 0
        for b, (m, n) in enumerate(zip(*_lens(c))):
            p = torch.arange(n - m, n, device="cuda")
            pos = p + (int(s["offsets"][b]) if s["offsets"] is not None else 0)
            page = s["table"][b].long()[p // s["ps"]]
            q[at:at + m] = _exact_turn(s["q"][at:at + m], pos, *how)
            k[page, p % s["ps"]] = _exact_turn(s["k"][at:at + m], pos, *how)
            v[page, p % s["ps"]] = s["v"][at:at + m].double()
            at += m
        return q, k, v
    if c["op"] == "attend_paged":
        o = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
        g, at = c["H"] // c["H_kv"], 0
        for b, (m, n) in enumerate(zip(*_lens(c))):
            j = torch.arange(n, device="cuda")
            p = torch.arange(n - m, n, device="cuda")
            for hk in range(c["H_kv"]):
                k, v = (x[s["table"][b].long()[j // s["ps"]], j % s["ps"], hk].double() for x in (s["k_pages"], s["v_pages"]))
                for h in range(hk * g, hk * g + g):
                    x = s["alpha"] * (s["q"][at:at + m, h].double() @ k.T) - s["slopes"][h].double() * (p[:, None] - j).double()
                    x = x.masked_fill(j[None] > p[:, None], -math.inf)
                    z = torch.logsumexp(x, -1)
                    o[at:at + m, h], lse[h, at:at + m] = torch.exp(x - z[:, None]) @ v, z
            at += m
        return o, lse
    lo, hi = (torch.tensor(x, device="cuda") for x in _intervals(c))
    docs = _documents(c)[0]
    blocks = [(b, int(x0), int(x1)) for b in range(c["B"]) for x0, x1 in zip(docs[b, :-1], docs[b, 1:]) if x1 > x0]
    if c["op"] == "attend":
        o = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for b, x0, x1 in blocks:
            for h in range(c["H"]):
                x, hk = _exact_block(s, b, h, lo, hi, x0, x1)
                z = torch.logsumexp(x, -1)
                lse[b, h, x0:x1] = z
                o[b, x0:x1, h] = torch.exp(x - z[:, None]) @ s["v"][b, x0:x1, hk].double()
        return o, lse
    dq, dk, dv = (torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv")
    for b, x0, x1 in blocks:
        for h in range(c["H"]):
            x, hk = _exact_block(s, b, h, lo, hi, x0, x1)
            p = torch.softmax(x, -1)
            do = s["dout"][b, x0:x1, h].double()
            dp = do @ s["v"][b, x0:x1, hk].double().T
            ds = s["alpha"] * p * (dp - (p * dp).sum(-1, keepdim=True))
            dq[b, x0:x1, h] = ds @ s["k"][b, x0:x1, hk].double()
            dk[b, x0:x1, hk] += ds.T @ s["q"][b, x0:x1, h].double()
            dv[b, x0:x1, hk] += p.T @ do
    return dq, dk, dv
