"""The operators on a paged key/value cache, as measured work: cases over their
real range, their plain forms in elementary torch operations, and their values
in 64 bits.

A paged cache holds K and V as [n_pages, page_size, H_kv, d]; sequence b's
token at position p lives in page block_table[b, p // page_size], slot
p % page_size.  kv_len[b] counts its cached tokens, the new ones among them;
the new tokens of all sequences are packed into rows cu_q[b] .. cu_q[b + 1].
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(name, op, dtype="bf16", d=128, H=32, H_kv=8, page=16, B=1, q=(1, 1), kv=(1, 1), lens=0, left=-1,
          first=0, keep=0, recent=0):
    return {"name": name, "op": op, "dtype": dtype, "d": d, "H": H, "H_kv": H_kv, "page": page, "B": B,
            "q_min": q[0], "q_max": q[1], "kv_min": kv[0], "kv_max": kv[1], "lens": lens, "left": left,
            "first": first, "keep": keep, "recent": recent}


def listed():
    return [
        # one new token for each of a serving batch goes into its pages: pure latency
        _case("append_tokens_b64", "append", B=64, kv=(512, 8192), lens=1),
        # a prompt's chunk from a fused projection (K and V are slices of wider rows) goes into its pages
        _case("append_chunks_b4", "append", "fp16", page=64, B=4, q=(1500, 4096), kv=(4096, 16384), lens=2),
        # one user, a short conversation: the smallest call of the attention
        _case("attend_token_b1", "attend", B=1, kv=(777, 777), lens=3),
        # the ordinary decoding step: a ragged batch, grouped heads
        _case("attend_tokens_b64", "attend", B=64, kv=(512, 8192), lens=4),
        # two long contexts: few rows, the long axis has to be split
        _case("attend_tokens_long_b2", "attend", "fp16", page=64, B=2, kv=(100001, 131072), lens=5),
        # a streaming cache without grouped heads: a window and a few first tokens that stay visible
        _case("attend_stream_d64_b32", "attend", "fp16", d=64, H=16, H_kv=16, page=32, B=32, q=(1, 4),
              kv=(3000, 8192), lens=6, left=2047, first=4),
        # a scheduler's mixed step: a few prompt chunks beside many decoding sequences
        _case("attend_mixed_b24", "attend", page=32, B=24, q=(1, 300), kv=(301, 4096), lens=7),
        # chunks of long prompts over what is cached of them: the largest
        _case("attend_chunks_b3", "attend", page=64, B=3, q=(1000, 2048), kv=(6000, 16384), lens=8),
        # the attention weight that each cached token got in a decoding step
        _case("weigh_tokens_b32", "weigh", B=32, kv=(512, 8192), lens=9),
        # the same over a prompt's chunk
        _case("weigh_chunks_b2", "weigh", page=64, B=2, q=(700, 1024), kv=(3000, 8192), lens=10),
        # a small batch's cache is cut to a quarter
        _case("evict_b2", "evict", B=2, kv=(1025, 2048), lens=11, keep=512, first=4, recent=128),
        # a serving batch's long caches are cut to 2048 tokens; one may be shorter than that
        _case("evict_b16", "evict", "fp16", page=64, B=16, kv=(1500, 16384), lens=12, keep=2048, first=4, recent=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weigh", "evict"])
    H, H_kv = rng.choice([(32, 8), (16, 16), (16, 2), (8, 1), (12, 4), (24, 8), (32, 4)])
    d = rng.choice([64, 128])
    B = _log_int(rng, 1, 48)
    # at most the bytes of the largest listed batch
    top = min(16384 if B <= 4 else 6000, int(1.1e9 / (4 * B * H_kv * d)))
    kv_max = _log_int(rng, 200, top)
    kv_min = rng.randint(max(1, kv_max // 8), kv_max)
    q_max = 1
    if op != "evict" and rng.random() < 0.6:
        q_max = min(kv_min, _log_int(rng, 2, 700 if B <= 3 else 250 if B <= 12 else 40))
    q_min = rng.randint(1, q_max)
    left = _log_int(rng, 100, 4000) if op in ("attend", "weigh") and rng.random() < 0.35 else -1
    keep = _log_int(rng, 64, 4000) if op == "evict" else 0
    c = _case("", op, rng.choice(["bf16", "fp16"]), d, H, H_kv, rng.choice([16, 32, 64, 128]), B, (q_min, q_max),
              (kv_min, kv_max), rng.randrange(1 << 20), left, rng.choice([0, 4, 17]) if left >= 0 or keep else 0,
              keep, rng.randint(0, keep - 17) if keep else 0)
    del c["name"]
    return c


def _lens(c):
    """The new tokens and cached tokens of each sequence: ragged, fixed by the case (a wide range of new tokens
    is spread over its logarithm: few long chunks beside many short ones)."""
    r = random.Random(1000 + c["lens"])
    kv = [r.randint(c["kv_min"], c["kv_max"]) for _ in range(c["B"])]
    pick = _log_int if c["q_max"] > 10 * c["q_min"] else random.Random.randint
    q = [min(pick(r, c["q_min"], c["q_max"]), n) for n in kv]
    return q, kv


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    q_len, kv = _lens(c)
    T, ps, H, Hk, d, t = sum(q_len), c["page"], c["H"], c["H_kv"], c["d"], DT[c["dtype"]]
    pages = [-(-n // ps) for n in kv]
    moved = -(-c["keep"] // ps) if c["op"] == "evict" else 0
    n_pages = sum(pages) + moved * c["B"] + 3
    width = max(pages)
    perm = torch.randperm(n_pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((c["B"], width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(t)

    s = {"case": c, "table": table, "ps": ps, "alpha": 1.0 / math.sqrt(d), "q_max": max(q_len),
         "window": (c["left"], 0), "first": c["first"],
         "k_pages": normal(n_pages, ps, Hk, d), "v_pages": normal(n_pages, ps, Hk, d),
         "kv_len": torch.tensor(kv, dtype=torch.int32, device=dev),
         "cu_q": torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device=dev)}
    if c["op"] == "append":
        # the rows of a fused projection: H query heads, then K, then V
        rows = normal(T, H + 2 * Hk, d)
        s["k"], s["v"] = rows[:, H:H + Hk], rows[:, H + Hk:]
    if c["op"] in ("attend", "weigh"):
        s["q"] = normal(T, H, d)
        s["out"] = torch.empty((T, H, d), dtype=t, device=dev)
        s["lse"] = torch.empty((H, T), dtype=torch.float32, device=dev)
    if c["op"] == "weigh":
        s["lse"] = _plain_attend(s)[1]
        L = width * ps
        s["scores"] = torch.rand((c["B"], Hk, L), generator=g, device=dev) * 3
        s["scores_out"] = torch.zeros((c["B"], Hk, L), dtype=torch.float32, device=dev)
    if c["op"] == "evict":
        L = width * ps
        x = torch.exp(1.5 * torch.randn((c["B"], Hk, L), generator=g, device=dev))
        # tokens that no query has seen yet have exactly no weight
        s["scores"] = torch.where(torch.rand(x.shape, generator=g, device=dev) < 0.2, torch.zeros_like(x), x)
        s["dst_table"] = perm[at:at + moved * c["B"]].reshape(c["B"], moved).contiguous()
        s["kept"] = torch.full((c["B"], Hk, c["keep"]), -1, dtype=torch.int32, device=dev)
        s["scores_out"] = torch.zeros((c["B"], Hk, c["keep"]), dtype=torch.float32, device=dev)
        s["new_len"] = torch.zeros(c["B"], dtype=torch.int32, device=dev)
    return s


# ---- the plain forms: padded to the longest sequence, float32 ----

def _padded(s):
    """Row index, validity and position of every (sequence, new token)."""
    cu = s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["q_max"], device=cu.device)
    ok = i[None] < n[:, None]
    pos = (s["kv_len"].long() - n)[:, None] + i[None]
    row = torch.where(ok, cu[:-1, None] + i[None], torch.zeros_like(pos))
    return row, ok, pos


def _gathered(s, pages):
    """[B, H_kv, L, d] float32 of a cache, by its block table; nothing behind kv_len."""
    t = s["table"].long().clamp(min=0)
    x = pages[t].float()                                       # [B, W, ps, H_kv, d]
    x = x.reshape(t.shape[0], -1, x.shape[3], x.shape[4])
    j = torch.arange(x.shape[1], device=x.device)
    x = torch.where((j[None] < s["kv_len"][:, None])[:, :, None, None], x, torch.zeros_like(x))
    return x.transpose(1, 2).contiguous()


def _visible(s, pos, L):
    """[B, Q, L]: whether the row at a position sees a key."""
    j = torch.arange(L, device=pos.device)
    p = pos[:, :, None]
    seen = (j < s["kv_len"][:, None, None]) & (j <= p)
    left = s["window"][0]
    if left >= 0:
        seen = seen & ((j >= p - left) | (j < s["first"]))
    return seen


def _logits(s):
    row, ok, pos = _padded(s)
    q = s["q"].float()[row]                                    # [B, Q, H, d]
    B, Q, H, d = q.shape
    k = _gathered(s, s["k_pages"])
    Hk, L = k.shape[1], k.shape[2]
    q = q.reshape(B, Q, Hk, H // Hk, d).permute(0, 2, 3, 1, 4)  # [B, H_kv, g, Q, d]
    x = torch.matmul(q.reshape(B, Hk, -1, d), k.transpose(2, 3)).reshape(B, Hk, H // Hk, Q, L) * s["alpha"]
    seen = (_visible(s, pos, L) & ok[:, :, None])[:, None, None]
    return torch.where(seen, x, torch.full_like(x, -math.inf)), row, ok


def _plain_attend(s):
    x, row, ok = _logits(s)
    B, Hk, g, Q, L = x.shape
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(-1)
    o = torch.matmul(e.reshape(B, Hk, g * Q, L), _gathered(s, s["v_pages"])).reshape(B, Hk, g, Q, -1)
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    lse = torch.log(total) + top[..., 0]
    out = torch.empty_like(s["out"])
    out[row[ok]] = o.permute(0, 3, 1, 2, 4).reshape(B, Q, Hk * g, -1)[ok].to(out.dtype)
    stat = torch.empty_like(s["lse"])
    stat[:, row[ok]] = lse.permute(1, 2, 0, 3).reshape(Hk * g, B, Q)[:, ok]
    return out, stat


def _plain_append(s):
    row, ok, pos = _padded(s)
    b = torch.arange(ok.shape[0], device=ok.device)[:, None].expand_as(ok)
    page = s["table"].long()[b[ok], pos[ok] // s["ps"]]
    slot = pos[ok] % s["ps"]
    s["k_pages"][page, slot] = s["k"][row[ok]]
    s["v_pages"][page, slot] = s["v"][row[ok]]
    return s["k_pages"], s["v_pages"]


def _plain_weigh(s):
    x, row, ok = _logits(s)
    B, Hk, g, Q, L = x.shape
    lse = s["lse"][:, row].reshape(Hk, g, B, Q).permute(2, 0, 1, 3)
    w = torch.where(torch.isinf(x), torch.zeros_like(x), torch.exp(x - lse[..., None])).double().sum((2, 3))
    cu = s["cu_q"].long()
    old = s["kv_len"].long() - (cu[1:] - cu[:-1])
    j = torch.arange(L, device=x.device)
    a = torch.where((j[None] < old[:, None])[:, None], s["scores"], torch.zeros_like(s["scores"])) + w
    live = (j[None] < s["kv_len"][:, None])[:, None]
    return torch.where(live, a, torch.zeros_like(a)).float()


def _plain_evict(s):
    c, a = s["case"], s["scores"]
    B, Hk, L = a.shape
    keep, n = c["keep"], s["kv_len"].long()[:, None, None]
    j = torch.arange(L, device=a.device)[None, None].expand(B, Hk, L)
    safe = (j < c["first"]) | (j >= n - c["recent"]) | (n <= keep)
    rank = torch.where(safe, torch.full_like(a, math.inf), a)
    rank = torch.where(j < n, rank, torch.full_like(a, -math.inf))
    if L < keep:
        rank = torch.cat([rank, torch.full((B, Hk, keep - L), -math.inf, device=a.device)], 2)
    order = torch.sort(rank, dim=2, descending=True, stable=True).indices[:, :, :keep]
    new_len = n.clamp(max=keep)
    r = torch.arange(keep, device=a.device)[None, None].expand(B, Hk, keep)
    live = r < new_len
    idx = torch.sort(torch.where(live, order, torch.full_like(order, 1 << 40)), dim=2).values
    kept = torch.where(live, idx, torch.full_like(idx, -1))
    at = idx.clamp(max=L - 1)
    scores = torch.where(live, torch.gather(a, 2, at), torch.zeros_like(at, dtype=a.dtype))
    b = torch.arange(B, device=a.device)[:, None, None].expand(B, Hk, keep)[live]
    h = torch.arange(Hk, device=a.device)[None, :, None].expand(B, Hk, keep)[live]
    src, dst, ps = at[live], r[live], s["ps"]
    sp, dp = s["table"].long()[b, src // ps], s["dst_table"].long()[b, dst // ps]
    for_k, for_v = s["k_pages"][sp, src % ps, h], s["v_pages"][sp, src % ps, h]
    s["k_pages"][dp, dst % ps, h] = for_k
    s["v_pages"][dp, dst % ps, h] = for_v
    return s["k_pages"], s["v_pages"], kept.to(torch.int32), scores, new_len[:, 0, 0].to(torch.int32)


def _own(s):
    import exact_attention_forward_fa_gb300 as fa
    op = s["case"]["op"]
    cache = (s["k_pages"], s["v_pages"])
    if op == "append":
        fa.paged_append(s["k"], s["v"], *cache, s["table"], s["kv_len"], s["cu_q"])
        return cache
    if op == "attend":
        return fa.attention_paged(s["q"], *cache, s["table"], s["kv_len"], s["cu_q"], max_q=s["q_max"],
                                  window=s["window"], first=s["first"], alpha=s["alpha"], out=s["out"],
                                  lse=s["lse"])
    if op == "weigh":
        return fa.paged_scores(s["q"], s["lse"], s["k_pages"], s["table"], s["kv_len"], s["cu_q"],
                               max_q=s["q_max"], scores=s["scores"], window=s["window"], first=s["first"],
                               alpha=s["alpha"], out=s["scores_out"])
    kept, scores, new_len = fa.paged_evict(*cache, s["scores"], s["table"], s["kv_len"], s["dst_table"],
                                           keep=s["case"]["keep"], first=s["first"],
                                           recent=s["case"]["recent"], kept=s["kept"],
                                           scores_out=s["scores_out"], new_len=s["new_len"])
    return cache + (kept, scores, new_len)


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "append":
        return _plain_append(state)
    if op == "attend":
        return _plain_attend(state)
    return _plain_weigh(state) if op == "weigh" else _plain_evict(state)


def _seen(c, p, n):
    """How many keys the row at position p of n cached tokens sees."""
    if c["left"] < 0 or p - c["left"] <= 0:
        return p + 1
    low = p - c["left"]
    return p + 1 - low + min(c["first"], low)


def work(case):
    c = case
    q_len, kv = _lens(c)
    T, H, Hk, d = sum(q_len), c["H"], c["H_kv"], c["d"]
    if c["op"] == "append":
        return {"bytes": 2 * 2 * 2 * T * Hk * d, "flops": 0}
    if c["op"] == "evict":
        rows = sum(min(n, c["keep"]) for n in kv) * Hk
        return {"bytes": 4 * Hk * sum(kv) + rows * (2 * 2 * 2 * d + 8), "flops": 0}
    pairs = sum(_seen(c, n - m + i, n) for m, n in zip(q_len, kv) for i in range(m)) * H
    # the cached tokens that any new token of the sequence sees
    keys = sum(n - max(0, n - m - c["left"] - c["first"]) if c["left"] >= 0 else n for m, n in zip(q_len, kv)) * Hk
    if c["op"] == "attend":
        return {"bytes": 2 * 2 * T * H * d + 4 * T * H + 2 * 2 * keys * d, "flops": 4 * d * pairs}
    return {"bytes": 2 * T * H * d + 4 * T * H + 2 * keys * d + 8 * Hk * sum(kv), "flops": 2 * d * pairs}


# ---- the values in 64 bits, one sequence and K/V head at a time ----

def _cached(s, pages, b, h, n):
    at = torch.arange(n, device=pages.device)
    return pages[s["table"][b].long()[at // s["ps"]], at % s["ps"], h].double()


def _exact_rows(s, b, h):
    """Logits [g, m, n] of sequence b's new tokens against its cache, -inf where unseen."""
    lo, hi, n = int(s["cu_q"][b]), int(s["cu_q"][b + 1]), int(s["kv_len"][b])
    H, Hk = s["case"]["H"], s["case"]["H_kv"]
    g = H // Hk
    q = s["q"][lo:hi, h * g:(h + 1) * g].double().transpose(0, 1)
    x = s["alpha"] * (q @ _cached(s, s["k_pages"], b, h, n).T)
    p = torch.arange(n - (hi - lo), n, device=x.device)[:, None]
    j = torch.arange(n, device=x.device)[None]
    hidden = j > p
    if s["window"][0] >= 0:
        hidden |= (j < p - s["window"][0]) & (j >= s["first"])
    return x.masked_fill(hidden, -math.inf), lo, hi, n, g


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    q_len, kv = _lens(c)
    if c["op"] == "append":
        out = [s["k_pages"].double(), s["v_pages"].double()]
        for x, new in zip(out, (s["k"], s["v"])):
            at = 0
            for b, (m, n) in enumerate(zip(q_len, kv)):
                p = torch.arange(n - m, n, device=x.device)
                x[s["table"][b].long()[p // s["ps"]], p % s["ps"]] = new[at:at + m].double()
                at += m
        return tuple(out)
    if c["op"] == "attend":
        o = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            for h in range(c["H_kv"]):
                x, lo, hi, n, g = _exact_rows(s, b, h)
                z = torch.logsumexp(x, -1)
                o[lo:hi, h * g:(h + 1) * g] = (torch.exp(x - z[..., None]) @ _cached(s, s["v_pages"], b, h, n)
                                               ).transpose(0, 1)
                lse[h * g:(h + 1) * g, lo:hi] = z
        return o, lse
    if c["op"] == "weigh":
        a = torch.zeros(s["scores"].shape, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            for h in range(c["H_kv"]):
                x, lo, hi, n, g = _exact_rows(s, b, h)
                got = torch.exp(x - s["lse"][h * g:(h + 1) * g, lo:hi].double()[..., None]).sum((0, 1))
                got[:n - (hi - lo)] += s["scores"][b, h, :n - (hi - lo)].double()
                a[b, h, :n] = got
        return a
    k, v = s["k_pages"].double(), s["v_pages"].double()
    kept, scores = s["kept"].long(), s["scores_out"].double()
    a = s["scores"].cpu().numpy()
    for b, n in enumerate(kv):
        for h in range(c["H_kv"]):
            ids = np.arange(n)
            if n > c["keep"]:
                mid = ids[c["first"]:n - c["recent"]]
                best = mid[np.lexsort((mid, -a[b, h, mid].astype(np.float64)))]
                best = best[:c["keep"] - c["first"] - c["recent"]]
                ids = np.sort(np.concatenate([ids[:c["first"]], best, ids[n - c["recent"]:]]))
            i = torch.from_numpy(ids).to("cuda")
            r = torch.arange(len(ids), device="cuda")
            dp = s["dst_table"][b].long()[r // s["ps"]]
            k[dp, r % s["ps"], h] = _cached(s, s["k_pages"], b, h, n)[i]
            v[dp, r % s["ps"], h] = _cached(s, s["v_pages"], b, h, n)[i]
            kept[b, h, :len(ids)] = i
            scores[b, h, :len(ids)] = s["scores"][b, h][i].double()
    return k, v, kept, scores, torch.tensor([min(n, c["keep"]) for n in kv], device="cuda")
