"""GPU checks of the operators on a paged key/value cache against float64:
fa_paged_append, fa_fwd_paged, fa_paged_scores and fa_paged_evict.

Tolerances, per element, with u the half step of the 16-bit type (2^-8 bf16,
2^-11 fp16) and everything else FP32:

* O = sum_j p_j v_j / sum_j p_j, p_j rounded to the type before the product
  and summed as rounded, O rounded once: each of numerator and denominator is
  off by at most u relative to sum p |v| and sum p, so
  |dO| <= u (A + |O|) + u |O| with A = softmax-weighted |v|; 5 % is added for
  second-order terms and the FP32 sums.
* A score is an FP32 dot product of d terms: off by at most
  d 2^-23 alpha sum |q||k| (2^-23 a step: the tensor core may truncate).  LSE
  is off by the largest of these, plus 2^-20 for exp2, log2 and the sums, plus
  its own rounding, 2^-22 |LSE|.
* An accumulated weight is a sum of exp(s - LSE), each off by the score's
  error and 2^-19 relative (exp2, and the FP32 rounding of an exponent of at
  most 32), the sum of R terms by R 2^-24, and the addition to what was
  there, 2^-23 relative.
"""
import math
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


class Cache:
    """A paged cache with random tokens, its slots behind every kv_len NaN, its
    unused table entries out of range, and the packed queries of a call."""

    def __init__(self, q_len, kv_len, H=4, H_kv=2, d=64, ps=16, dt="bf16", seed=0, spare=2, side=False,
                 behind=0, gap=0, scale=1.0):
        g = torch.Generator("cuda").manual_seed(seed)
        t, dev = DT[dt], "cuda"
        self.q_len, self.kv, self.H, self.H_kv, self.d, self.ps, self.dt = q_len, kv_len, H, H_kv, d, ps, dt
        pages = [-(-n // ps) for n in kv_len]
        n = sum(pages) + spare
        if side:                    # K and V side by side in one pool
            pool = torch.full((n, 2, ps, H_kv, d), math.nan, dtype=t, device=dev)
            self.k_pages, self.v_pages = pool[:, 0], pool[:, 1]
        else:
            self.k_pages = torch.full((n, ps, H_kv, d), math.nan, dtype=t, device=dev)
            self.v_pages = torch.full((n, ps, H_kv, d), math.nan, dtype=t, device=dev)
        perm = torch.randperm(n, generator=g, device=dev).int()
        self.table = torch.full((len(kv_len), max(1, max(pages)) + 1), 1 << 30, dtype=torch.int32, device=dev)
        self.K, self.V, at = [], [], 0
        for b, m in enumerate(pages):
            self.table[b, :m] = perm[at:at + m]
            at += m
            k = (scale * torch.randn(kv_len[b], H_kv, d, generator=g, device=dev)).to(t)
            v = torch.randn(kv_len[b], H_kv, d, generator=g, device=dev).to(t)
            self.K.append(k.double())
            self.V.append(v.double())
            self.put(b, 0, k, v)
        self.free = perm[at:]
        self.kv_len = torch.tensor(kv_len, dtype=torch.int32, device=dev)
        cu = [0]
        for m in q_len:
            cu.append(cu[-1] + m)
        self.cu, self.T = cu, cu[-1] + behind
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=dev)
        rows = (scale * torch.randn(self.T, H + gap, d, generator=g, device=dev)).to(t)
        self.q = rows[:, :H]

    def put(self, b, p0, k, v):
        p = torch.arange(p0, p0 + k.shape[0], device="cuda")
        page = self.table[b].long()[p // self.ps]
        self.k_pages[page, p % self.ps] = k
        self.v_pages[page, p % self.ps] = v

    def args(self):
        return self.k_pages, self.v_pages, self.table, self.kv_len, self.cu_q

    def rows(self, b, window, first, alpha):
        """Float64 scores [H, m, n] of sequence b (-inf where hidden), and the
        bound of their rounding."""
        m, n = self.q_len[b], self.kv[b]
        q = self.q[self.cu[b]:self.cu[b] + m].double().transpose(0, 1)           # [H, m, d]
        k = self.K[b].transpose(0, 1).repeat_interleave(self.H // self.H_kv, 0)  # [H, n, d]
        s = alpha * q @ k.transpose(1, 2)
        e = abs(alpha) * self.d * 2.0 ** -23 * (q.abs() @ k.abs().transpose(1, 2))
        p = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None]
        hide = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if window[1] >= 0:
            hide |= j > p + window[1]
        if window[0] >= 0:
            hide |= (j < p - window[0]) & (j >= first)
        return s.masked_fill(hide, -math.inf), e.masked_fill(hide, 0.0)


def check_attention(c, o, lse, window=(-1, 0), first=0, alpha=None):
    u = U[c.dt]
    alpha = 1 / math.sqrt(c.d) if alpha is None else alpha
    for b in range(len(c.kv)):
        m, n = c.q_len[b], c.kv[b]
        if m == 0:
            continue
        got = o[c.cu[b]:c.cu[b] + m].double().transpose(0, 1)
        stat = lse[:, c.cu[b]:c.cu[b] + m].double()
        if n == 0:
            assert (got == 0).all() and (stat == -math.inf).all()
            continue
        s, e = c.rows(b, window, first, alpha)
        z = torch.logsumexp(s, -1)
        w = torch.where(torch.isinf(z)[..., None], torch.zeros_like(s), torch.exp(s - z[..., None]))
        v = c.V[b].transpose(0, 1).repeat_interleave(c.H // c.H_kv, 0)
        ref, mag = w @ v, w @ v.abs()
        err = (got - ref).abs()
        tol = 1.05 * u * (mag + 2 * ref.abs()) + 1e-6
        assert torch.isfinite(got).all()
        assert (err <= tol).all(), f"sequence {b}: {float((err / tol).max()):.2f} of the tolerance"
        empty = torch.isinf(z)
        assert (stat[empty] == -math.inf).all() and (got[empty] == 0).all()
        ltol = e.amax(-1) + 2.0 ** -20 + 2.0 ** -22 * z.abs()
        assert ((stat - z).abs()[~empty] <= ltol[~empty]).all()


def attend(fa, c, window=(-1, 0), first=0, alpha=None, **kw):
    o, lse = fa.attention_paged(c.q, *c.args(), max_q=max(1, max(c.q_len)), window=window, first=first,
                                alpha=alpha, **kw)
    assert fa.fa_check_status() == fa.FA_OK
    return o, lse


# (new tokens, cached tokens): single tokens, chunks, their mixture, tile and page edges
LENS = {
    "one": ([1], [1]),
    "tokens": ([1, 1, 1, 1], [7, 128, 129, 1000]),
    "few": ([3, 1, 5, 2], [3, 640, 257, 300]),
    "none": ([0, 2, 0, 0], [50, 70, 0, 1]),
    "empty_rows": ([4, 1, 2, 130], [2, 0, 2, 100]),      # more new tokens than cached: rows that see nothing
    "chunk": ([127, 129], [127, 1023]),
    "prompt": ([300], [300]),
    "mixed": ([1, 200, 1, 33, 1], [900, 513, 64, 65, 1]),
}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dt,d,H,H_kv,ps", [("bf16", 128, 8, 2, 16), ("fp16", 64, 4, 4, 32),
                                            ("bf16", 64, 6, 2, 8), ("fp16", 128, 7, 1, 256)])
def test_attention(gpu_lib, lens, dt, d, H, H_kv, ps):
    c = Cache(*LENS[lens], H, H_kv, d, ps, dt, seed=len(lens), behind=3, gap=2)
    out = torch.full((c.T, H, d), 7.0, dtype=DT[dt], device="cuda")
    lse = torch.full((H, c.T), 7.0, device="cuda")
    attend(gpu_lib, c, out=out, lse=lse)
    check_attention(c, out, lse)
    n = c.cu[-1]                                # rows behind the last sequence stay as they were
    assert (out[n:] == 7).all() and (lse[:, n:] == 7).all()


@pytest.mark.parametrize("window,first", [((-1, -1), 0), ((0, 0), 0), ((0, 0), 1), ((100, 0), 4), ((31, 5), 0),
                                          ((300, -1), 130), ((127, 0), 128), ((64, 0), 2000),
                                          ((2**31 - 1, 2**31 - 1), 2**31 - 1), ((-1, 3), 9)])
@pytest.mark.parametrize("lens", ["tokens", "empty_rows", "mixed"])
def test_attention_masks(gpu_lib, lens, window, first):
    c = Cache(*LENS[lens], 8, 2, 128 if lens == "mixed" else 64, 16, seed=first % 97, side=True)
    o, lse = attend(gpu_lib, c, window, first)
    check_attention(c, o, lse, window, first)


@pytest.mark.parametrize("H,H_kv,q", [(128, 1, 2), (96, 1, 3), (40, 8, 40), (32, 2, 9), (3, 3, 260)])
def test_attention_groups(gpu_lib, H, H_kv, q):
    c = Cache([q, 1], [400, 131], H, H_kv, 64, 64, seed=H)
    o, lse = attend(gpu_lib, c)
    check_attention(c, o, lse)


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (64, "fp16")])
def test_attention_long_axis(gpu_lib, d, dt):
    # few rows against a long cache: the key range is split over the SMs and joined
    c = Cache([1, 2], [70001, 33000], 8, 1, d, 64, dt)
    o, lse = attend(gpu_lib, c)
    check_attention(c, o, lse)
    for _ in range(3):
        o2, lse2 = attend(gpu_lib, c)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attention_many_sequences(gpu_lib):
    c = Cache([1 + (i % 3 == 0) for i in range(900)], [1 + (i * 37) % 400 for i in range(900)], 4, 1, 64, 16)
    o, lse = attend(gpu_lib, c)
    check_attention(c, o, lse)


def test_attention_large_scores(gpu_lib):
    # scores of several hundred: the reference of the exponentials moves often
    c = Cache([40, 1], [700, 900], 4, 2, 64, 16, "fp16", seed=5, scale=6.0)
    o, lse = attend(gpu_lib, c)
    check_attention(c, o, lse)


@pytest.mark.parametrize("q_len", [1, 7, 40])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("tile", [0, 1, 2])
@pytest.mark.parametrize("peak", [14.9999, 15.0001, 15.9985, 15.99975, 15.99995, 16.0001])
def test_attention_one_score_far_above(gpu_lib, q_len, dt, tile, peak):
    # 2^peak against a reference of 0 from other tiles: terms at the edge of
    # fp16's range
    c = Cache([q_len], [384], 4, 1, 64, 64, dt, seed=1)
    c.q.zero_()
    c.q[:, :, 0] = 1
    k = torch.zeros(384, 1, 64, device="cuda")
    k[128 * tile:128 * tile + 128, 0, 0] = -10
    k[128 * tile + 5, 0, 0] = 1
    c.K[0] = k.double()
    c.put(0, 0, k.to(DT[dt]), c.V[0].to(DT[dt]))
    alpha = peak * math.log(2)
    o, lse = attend(gpu_lib, c, (-1, -1), 0, alpha)
    check_attention(c, o, lse, (-1, -1), 0, alpha)


@pytest.mark.parametrize("alpha", [1e-6, 0.01, 2.0])
def test_attention_alpha(gpu_lib, alpha):
    c = Cache([3, 140], [50, 200], seed=1)
    o, lse = attend(gpu_lib, c, alpha=alpha)
    check_attention(c, o, lse, alpha=alpha)


@pytest.mark.parametrize("q_len,H", [([1, 1], 8), ([7, 1], 8), ([200, 90], 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_stays_with_the_rows_that_see_it(gpu_lib, q_len, H, d):
    # one key of sequence 0 and K/V head 1, in the middle of a long key range
    # (which is cut and joined), and one that only the later new tokens see
    c = Cache(q_len, [9000, 500], H, 2, d, 16, seed=d)
    o, lse = attend(gpu_lib, c)
    m, g = q_len[0], H // 2
    for pos in {4321, 9000 - m + m // 2}:
        key = c.K[0][pos:pos + 1].to(DT[c.dt])
        bad = key.clone()
        bad[0, 1, 5] = math.nan
        c.put(0, pos, bad, c.V[0][pos:pos + 1].to(DT[c.dt]))
        o2, lse2 = attend(gpu_lib, c)
        c.put(0, pos, key, c.V[0][pos:pos + 1].to(DT[c.dt]))
        sees = torch.zeros(c.T, H, dtype=torch.bool, device="cuda")
        sees[max(0, pos - (9000 - m)):m, g:] = True
        assert torch.isnan(o2[sees]).all() and torch.isnan(lse2.t()[sees]).all()
        assert torch.equal(o2[~sees], o[~sees]) and torch.equal(lse2.t()[~sees], lse.t()[~sees])


@pytest.mark.parametrize("q,d", [(1, 128), (4, 128), (1, 64), (70, 128)])
def test_pieces_of_many_steps_repeat_their_bits(gpu_lib, q, d):
    # every ring of tiles is passed many times, pieces of odd and even lengths
    lens = [2000 + 137 * i for i in range(24)]
    c = Cache([q] * 24, lens, 8, 2, d, 64, seed=q)
    o, lse = attend(gpu_lib, c)
    check_attention(c, o, lse)
    for _ in range(20):
        o2, lse2 = attend(gpu_lib, c)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_max_q_is_only_a_hint(gpu_lib):
    c = Cache([150, 1], [150, 300], 8, 2, 128, 16, seed=2)
    for hint in (1, 3, 1000):
        o, lse = gpu_lib.attention_paged(c.q, *c.args(), max_q=hint)
        assert gpu_lib.fa_check_status() == gpu_lib.FA_OK
        check_attention(c, o, lse)
        a = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=hint)
        check_scores(c, lse, None, a)


def test_offsets_beyond_32_bits(gpu_lib):
    # pages 2^26 elements apart: the last ones lie beyond 2^31 elements
    c = Cache([2, 1], [300, 250], 4, 2, 64, 16, seed=3)
    n, stride = c.k_pages.shape[0], 1 << 26
    shape, st = c.k_pages.shape, (stride, 2 * 64, 64, 1)
    for name in ("k_pages", "v_pages"):
        flat = torch.zeros((n - 1) * stride + 16 * 2 * 64, dtype=torch.bfloat16, device="cuda")
        far = flat.as_strided(shape, st)
        far.copy_(getattr(c, name))
        setattr(c, name, far)
    assert (n - 1) * stride > 2 ** 31
    o, lse = attend(gpu_lib, c)
    check_attention(c, o, lse)
    a = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=2)
    check_scores(c, lse, None, a)
    k, v = (torch.randn(3, 2, 64, device="cuda").bfloat16() for _ in range(2))
    gpu_lib.paged_append(k, v, *c.args())
    assert torch.equal(c.k_pages[c.table[1, 249 // 16], 249 % 16], k[2])
    assert torch.equal(c.v_pages[c.table[0, 299 // 16], 299 % 16], v[1])


def check_scores(c, lse, old, got, window=(-1, 0), first=0):
    alpha = 1 / math.sqrt(c.d)
    g = c.H // c.H_kv
    for b in range(len(c.kv)):
        m, n = c.q_len[b], c.kv[b]
        if n == 0:
            continue
        ref = torch.zeros(c.H_kv, n, dtype=torch.float64, device="cuda")
        if old is not None and n > m:
            ref[:, :n - m] = old[b, :, :n - m].double()
        tol = 2.0 ** -23 * ref.abs()
        if m:
            s, e = c.rows(b, window, first, alpha)
            z = lse[:, c.cu[b]:c.cu[b] + m].double()[..., None]
            w = torch.where(torch.isinf(s) | torch.isinf(z), torch.zeros_like(s), torch.exp(s - z))
            ref += w.reshape(c.H_kv, g * m, n).sum(1)
            tol = (tol + (w * (e + 2.0 ** -19)).reshape(c.H_kv, g * m, n).sum(1)
                   + (2.0 ** -23 + 2.0 ** -24 * g * m) * ref.abs())
        err = (got[b, :, :n].double() - ref).abs()
        assert (err <= tol + 1e-30).all(), f"sequence {b}: {float((err / (tol + 1e-30)).max()):.2f} of the tolerance"


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dt,d,H,H_kv,ps,window,first", [
    ("bf16", 128, 8, 2, 16, (-1, 0), 0), ("fp16", 64, 6, 2, 8, (50, 0), 3), ("bf16", 64, 4, 4, 64, (20, 6), 0),
    ("fp16", 128, 7, 1, 256, (-1, -1), 0)])
def test_scores(gpu_lib, lens, dt, d, H, H_kv, ps, window, first):
    c = Cache(*LENS[lens], H, H_kv, d, ps, dt, seed=7, behind=2, gap=1)
    o, lse = attend(gpu_lib, c, window, first)
    L = c.table.shape[1] * ps + 5
    old = torch.rand(len(c.kv), H_kv, L, device="cuda") * 4
    kw = dict(max_q=max(1, max(c.q_len)), window=window, first=first)
    got = torch.full_like(old, -5.0)
    a = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], scores=old, out=got, **kw)
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK and a is got
    check_scores(c, lse, old, got, window, first)
    for b, n in enumerate(c.kv):                 # behind kv_len: left as it was
        assert (got[b, :, n:] == -5).all()
    fresh = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], **kw)
    check_scores(c, lse, None, fresh, window, first)
    same = old.clone()                           # in place
    gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], scores=same, out=same, **kw)
    for b, n in enumerate(c.kv):
        assert torch.equal(same[b, :, :n], got[b, :, :n])
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK


def test_scores_of_a_step_sum_to_the_rows(gpu_lib):
    # the weights that one token hands out sum to one for each of its heads
    c = Cache([1, 1], [3001, 40], 8, 2, 128, 16, seed=9)
    _, lse = attend(gpu_lib, c)
    a = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=1)
    assert (a.double().sum(-1) - 4).abs().max() < 1e-4


def test_scores_long_chunk(gpu_lib):
    c = Cache([700, 1, 260], [1500, 9000, 260], 8, 2, 128, 32, seed=4)
    _, lse = attend(gpu_lib, c)
    a = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=700)
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK
    check_scores(c, lse, None, a)


@pytest.mark.parametrize("kv", [[9000, 7777, 300], [12000, 9000, 300], [12100, 100, 16100], [129, 600, 290]])
@pytest.mark.parametrize("d,window,first", [(128, (-1, 0), 0), (64, (5000, 0), 200)])
def test_scores_several_rounds(gpu_lib, kv, d, window, first):
    # more pairs of key tiles than SMs, the last round full, half full, nearly
    # empty; and fewer: odd and even numbers of key and of Q tiles
    c = Cache([40, 90, 290], kv, 16, 4, d, 64, seed=kv[0])
    _, lse = attend(gpu_lib, c, window, first)
    kw = dict(max_q=290, window=window, first=first)
    a = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], **kw)
    check_scores(c, lse, None, a, window, first)
    for _ in range(5):
        b = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], **kw)
        for i, n in enumerate(kv):
            assert torch.equal(a[i, :, :n], b[i, :, :n])
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK


@pytest.mark.parametrize("dt,d,ps,side", [("bf16", 128, 16, False), ("fp16", 64, 8, True)])
@pytest.mark.parametrize("H_kv", [1, 2, 5, 40])
def test_append(gpu_lib, dt, d, ps, side, H_kv):
    q_len, kv = [1, 0, 20, 5, 3], [17, 9, 20, 40, 2]     # the last drops a token without a position
    c = Cache(q_len, kv, H_kv, H_kv, d, ps, dt, seed=1, side=side, behind=2)
    rows = torch.randn(c.T, 2 * H_kv + 1, d, device="cuda").to(DT[dt])
    k, v = rows[:, 1:H_kv + 1], rows[:, H_kv + 1:]
    want_k, want_v = c.k_pages.clone(), c.v_pages.clone()
    for b, (m, n) in enumerate(zip(q_len, kv)):
        for i in range(m):
            p = n - m + i
            if p >= 0:
                page = int(c.table[b, p // ps])
                want_k[page, p % ps], want_v[page, p % ps] = k[c.cu[b] + i], v[c.cu[b] + i]
    gpu_lib.paged_append(k, v, *c.args())
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK
    for got, want in ((c.k_pages, want_k), (c.v_pages, want_v)):
        assert torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16))


def _expected_kept(a, n, keep, first, recent):
    """Positions that stay, for one head's scores (a list of floats)."""
    if n <= keep:
        return list(range(n))
    rank = [(math.inf, 1) if x != x else (x, 0) for x in a[:n]]
    mid = sorted(range(first, n - recent), key=lambda j: (-rank[j][0], -rank[j][1], j))
    return sorted(list(range(first)) + mid[:keep - first - recent] + list(range(n - recent, n)))


def _score_rows(kind, shape, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.rand(shape, generator=g, device="cuda")
    if kind == "ties":
        x = (x * 4).floor() / 4
    elif kind == "equal":
        x = torch.zeros_like(x)
    elif kind == "signs":
        x = torch.where(x < 0.2, -0.0 * x, (x - 0.5) * 10.0 ** (x * 60 - 30))
    elif kind == "special":
        x = torch.where(x < 0.1, torch.full_like(x, math.nan), x)
        x = torch.where((x > 0.9) & (x < 0.93), torch.full_like(x, math.inf), x)
        x = torch.where(x > 0.97, torch.full_like(x, -math.inf), x)
    elif kind == "close":                        # many values that differ in the last bits only
        x = 1.0 + (x * 50).floor() * 2.0 ** -23
    return x


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "signs", "special", "close"])
@pytest.mark.parametrize("keep,first,recent", [(100, 0, 0), (64, 4, 20), (33, 30, 3), (1, 0, 0), (200, 0, 200),
                                               (1000, 7, 100)])
def test_evict(gpu_lib, kind, keep, first, recent):
    ps, H_kv, d = 16, 3, 64
    kv = [1, 33, 100, 101, 777, 1500, 0]
    per = -(-keep // ps)
    c = Cache([1] * len(kv), kv, H_kv, H_kv, d, ps, seed=keep, spare=per * len(kv) + 2, side=kind == "ties")
    dst = c.free[:per * len(kv)].reshape(len(kv), per).contiguous()
    L = 1504
    scores = _score_rows(kind, (len(kv), H_kv, L), keep)
    before_k, before_v = c.k_pages.clone(), c.v_pages.clone()
    kept, out, new_len = gpu_lib.paged_evict(c.k_pages, c.v_pages, scores, c.table, c.kv_len, dst, keep, first,
                                             recent)
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK
    assert new_len.tolist() == [min(n, keep) for n in kv]
    kept_l, rows = kept.tolist(), scores.tolist()
    want_k, want_v = before_k.clone(), before_v.clone()
    for b, n in enumerate(kv):
        m = min(n, keep)
        for h in range(H_kv):
            want = _expected_kept(rows[b][h], n, keep, first, recent)
            assert kept_l[b][h] == want + [-1] * (keep - m)
            i = torch.tensor(want, device="cuda", dtype=torch.long)
            r = torch.arange(m, device="cuda")
            assert torch.equal(out[b, h, :m].nan_to_num(9e9), scores[b, h][i].nan_to_num(9e9))
            assert (out[b, h, m:] == 0).all()
            sp, dp = c.table[b].long()[i // ps], dst[b].long()[r // ps]
            want_k[dp, r % ps, h], want_v[dp, r % ps, h] = before_k[sp, i % ps, h], before_v[sp, i % ps, h]
    for got, want in ((c.k_pages, want_k), (c.v_pages, want_v)):
        assert torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16))


@pytest.mark.parametrize("n,keep", [(40001, 5000), (70000, 65537), (16384, 16383)])
def test_evict_long(gpu_lib, n, keep):
    ps, d = 64, 64
    per = -(-keep // ps)
    c = Cache([1], [n], 1, 1, d, ps, seed=n, spare=per)
    scores = _score_rows("plain", (1, 1, n), n)
    scores[0, 0, 5:9000:3] = 0.5
    kept, out, new_len = gpu_lib.paged_evict(c.k_pages, c.v_pages, scores, c.table, c.kv_len,
                                             c.free[:per].reshape(1, per).contiguous(), keep, 4, 100)
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK
    assert kept[0, 0].tolist() == _expected_kept(scores[0, 0].tolist(), n, keep, 4, 100)
    assert int(new_len) == keep


# ---- what only the device can see ----

def test_bad_pages_and_lengths_are_reported(gpu_lib):
    fa = gpu_lib
    c = Cache([2, 1], [100, 90], 4, 2, 64, 16, seed=6)
    good = attend(fa, c)[0]

    def spoiled(run):
        run()
        assert fa.fa_check_status() == fa.FA_ERR_BAD_INDEX
        assert fa.fa_status_detail()[1] == 8
        assert fa.fa_check_status() == fa.FA_OK

    for page in (-1, c.k_pages.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[1, 2] = page
        out = torch.zeros_like(good)
        spoiled(lambda: fa.attention_paged(c.q, c.k_pages, c.v_pages, table, c.kv_len, c.cu_q, max_q=2, out=out))
        assert torch.equal(out[:2], good[:2])            # the other sequence's rows
    k = torch.ones(3, 2, 64, device="cuda", dtype=torch.bfloat16)
    table = c.table.clone()
    table[1, 89 // 16] = -7
    before = c.k_pages.clone()
    spoiled(lambda: fa.paged_append(k, k, c.k_pages, c.v_pages, table, c.kv_len, c.cu_q))
    before[c.table[0, 98 // 16], 98 % 16], before[c.table[0, 99 // 16], 99 % 16] = 1, 1
    assert torch.equal(c.k_pages.view(torch.int16), before.view(torch.int16))
    lse = torch.zeros(4, 3, device="cuda")
    table[1, 89 // 16] = 1 << 20
    spoiled(lambda: fa.paged_scores(c.q, lse, c.k_pages, table, c.kv_len, c.cu_q, max_q=2))
    scores = torch.rand(2, 2, 200, device="cuda")
    dst = c.free[:1].reshape(1, 1).repeat(2, 1)
    dst[1, 0] = 1 << 24
    spoiled(lambda: fa.paged_evict(c.k_pages, c.v_pages, scores, c.table, c.kv_len, dst, 16))
    for lens in ([-3, 90], [100, 2 ** 31 - 1]):
        kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
        t0 = torch.zeros_like(c.table)                   # every page id in range
        spoiled(lambda: fa.attention_paged(c.q, c.k_pages, c.v_pages, t0, kv, c.cu_q, max_q=2))
        spoiled(lambda: fa.paged_scores(c.q, lse, c.k_pages, t0, kv, c.cu_q, max_q=2,
                                        scores=torch.zeros(2, 2, 4096, device="cuda")))
        spoiled(lambda: fa.paged_append(k, k, c.k_pages, c.v_pages, t0, kv, c.cu_q))
    for cu in ([0, 2, 9], [0, 3, 1], [-1, 2, 3]):
        cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
        spoiled(lambda: fa.attention_paged(c.q, *c.args()[:4], cu_q, max_q=2))
    # scores that are too narrow for the cache
    spoiled(lambda: fa.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=2,
                                    scores=torch.zeros(2, 2, 64, device="cuda")))
    spoiled(lambda: fa.paged_evict(c.k_pages, c.v_pages, scores[:, :, :64].contiguous(), c.table, c.kv_len,
                                   dst.clamp(max=1), 16))


# ---- streams, graphs, and the operators together ----

def test_empty_calls(gpu_lib):
    c = Cache([0, 0], [5, 0], 4, 2, 64, 16)
    o, lse = attend(gpu_lib, c)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    gpu_lib.paged_append(c.q[:, :2], c.q[:, :2], *c.args())
    old = torch.rand(2, 2, 32, device="cuda")
    a = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=1, scores=old)
    assert torch.equal(a[0, :, :5], old[0, :, :5]) and (a[0, :, 5:] == 0).all() and (a[1] == 0).all()
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK


def test_strides_that_no_row_has(gpu_lib):
    # of an empty tensor, and between the heads of one head
    c = Cache([0, 0], [5, 0], 1, 1, 64, 16)
    q = torch.empty(192, device="cuda", dtype=torch.bfloat16).as_strided((0, 1, 64), (1, 1, 1))
    o, lse = gpu_lib.attention_paged(q, *c.args(), max_q=1)
    assert o.shape == (0, 1, 64)
    c = Cache([2, 1], [50, 9], 1, 1, 64, 16)
    want = attend(gpu_lib, c)
    wide = torch.zeros(3, 192, device="cuda", dtype=torch.bfloat16)
    wide[:, :64] = c.q[:, 0]
    o, lse = gpu_lib.attention_paged(wide.as_strided((3, 1, 64), (192, 1, 1)), *c.args(), max_q=2)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK


def test_another_stream(gpu_lib):
    c = Cache([1, 150, 1], [4000, 150, 300], 8, 2, 128, 16, seed=8)
    want = attend(gpu_lib, c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for st in (s, s.cuda_stream):
        for _ in range(4):
            outs.append(gpu_lib.attention_paged(c.q, *c.args(), max_q=150, stream=st))
            torch.empty(1 << 22, device="cuda").fill_(float("nan"))    # takes freed memory of this stream
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_two_streams_at_once(gpu_lib):
    cs = [Cache([1, 1], [20000, 900 + i], 8, 2, 128, 16, seed=i) for i in range(2)]
    want = [attend(gpu_lib, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, c in enumerate(cs):
            got[i].append(gpu_lib.attention_paged(c.q, *c.args(), max_q=1, stream=streams[i]))
    torch.cuda.synchronize()
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_threads_at_once(gpu_lib):
    # on the default stream (whose calls share a workspace) and on streams of
    # the threads' own
    cs = [Cache([1, 3], [6000 + 500 * i, 900], 8, 2, 64, 16, seed=i) for i in range(4)]
    want = [attend(gpu_lib, c) for c in cs]
    torch.cuda.synchronize()
    got, errors = [[] for _ in cs], []

    def work(i, own):
        try:
            with torch.cuda.stream(torch.cuda.Stream() if own else torch.cuda.default_stream()):
                for _ in range(25):
                    got[i].append(gpu_lib.attention_paged(cs[i].q, *cs[i].args(), max_q=3))
        except Exception as e:          # noqa: BLE001 (reported by the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i, i == 3)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and gpu_lib.fa_check_status() == gpu_lib.FA_OK
    for (o, lse), outs in zip(want, got):
        assert len(outs) == 25
        for o2, lse2 in outs:
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_threads_first_call(gpu_lib):
    # a thread that has not used the device yet, outputs given: nothing but the
    # call itself makes the device's context current there
    c = Cache([1], [300], 4, 2, 64, 16)
    o, lse = attend(gpu_lib, c)
    o2, lse2, ws = torch.empty_like(o), torch.empty_like(lse), gpu_lib.paged_workspace(64)
    old = torch.zeros(1, 2, 300, device="cuda")
    a = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=1, scores=old)
    a2 = torch.empty_like(a)
    torch.cuda.synchronize()
    for call in (lambda: gpu_lib.attention_paged(c.q, *c.args(), max_q=1, out=o2, lse=lse2, workspace=ws),
                 lambda: gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=1, scores=old, out=a2)):
        errors = []

        def work():
            try:
                call()
            except Exception as e:      # noqa: BLE001 (reported by the test's own thread)
                errors.append(e)

        t = threading.Thread(target=work)
        t.start()
        t.join()
        assert not errors
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(a, a2)


def test_graphs_with_workspaces_of_their_own(gpu_lib):
    # two captured calls, each with what its capture took, replayed side by side
    fa = gpu_lib
    cs = [Cache([1, 1], [15000, 700 + i], 8, 2, 128, 16, seed=i) for i in range(2)]
    want = [attend(fa, c) for c in cs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.attention_paged(c.q, *c.args(), max_q=1))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert fa.fa_check_status() == fa.FA_OK
    for (o, lse), (o2, lse2) in zip(want, outs):
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_results_of_the_call_before(gpu_lib):
    # chains of calls that read what the last one, another kernel, a copy or
    # another stream wrote, eager and captured
    fa = gpu_lib
    c = Cache([1, 2, 40], [700, 3000, 2000], 8, 2, 128, 16, seed=2)
    n = c.cu[-1]
    k, v = torch.randn(2, n, 2, 128, device="cuda").bfloat16()
    q2 = torch.randn(n, 8, 128, device="cuda").bfloat16()
    q, lens = torch.empty_like(q2), torch.empty_like(c.kv_len)
    pool = c.k_pages.clone(), c.v_pages.clone()
    wide = c.table.shape[1] * 16
    dst = torch.arange(-(-256 // 16) * 3, device="cuda").reshape(3, -1).int() + c.k_pages.shape[0]
    big = [torch.cat([x, torch.zeros_like(x[:dst.numel()])]) for x in pool]
    side = torch.cuda.Stream()

    def chain():
        out = []
        for i in range(3):
            kp, vp = (x.clone() for x in big)                       # (a copy, then the append)
            lens.copy_(c.kv_len)
            here = torch.cuda.current_stream()
            side.wait_stream(here)
            with torch.cuda.stream(side):
                q.copy_(q2)                                         # (another stream, then the attention)
            fa.paged_append(k, v, kp, vp, c.table, lens, c.cu_q)
            here.wait_stream(side)
            o, lse = fa.attention_paged(q, kp, vp, c.table, lens, c.cu_q, max_q=40)
            a = fa.paged_scores(q, lse, kp, c.table, lens, c.cu_q, max_q=40,
                                scores=torch.zeros(3, 2, wide, device="cuda"))
            kept, s, m = fa.paged_evict(kp, vp, a, c.table, lens, dst, 256, 4, 64)
            o1, lse1 = fa.attention_paged(o, kp, vp, dst, m, c.cu_q, max_q=40)
            out += [o, lse, a, kept, s, m, o1, lse1]
        return out

    want = [x.clone() for x in chain()]
    torch.cuda.synchronize()
    for i in range(8):                                              # each pass equals the first
        assert torch.equal(want[i].nan_to_num(9e9), want[i + 8].nan_to_num(9e9))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    for _ in range(20):
        g.replay()
        for x, y in zip(want, got):
            assert torch.equal(x.nan_to_num(9e9), y.nan_to_num(9e9))
    assert fa.fa_check_status() == fa.FA_OK


def test_graph_replays_with_other_lengths(gpu_lib):
    fa = gpu_lib
    c = Cache([1, 1, 1], [400, 300, 2000], 8, 2, 64, 16, seed=3)
    k = torch.randn(3, 2, 64, device="cuda").bfloat16()
    v = torch.randn(3, 2, 64, device="cuda").bfloat16()
    o, lse = torch.empty(3, 8, 64, device="cuda", dtype=torch.bfloat16), torch.empty(8, 3, device="cuda")
    a = torch.zeros(3, 2, 2048, device="cuda")
    ws = fa.paged_workspace(64)

    def step():
        fa.paged_append(k, v, *c.args())
        fa.attention_paged(c.q, *c.args(), max_q=1, out=o, lse=lse, workspace=ws)
        fa.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=1, scores=a, out=a)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    full = list(c.kv)
    for lens in ([400, 300, 2000], [17, 300, 1], [33, 1, 1500]):
        c.kv_len.copy_(torch.tensor(lens))
        old = a.clone()
        g.replay()
        assert fa.fa_check_status() == fa.FA_OK
        for b, n in enumerate(lens):
            c.K[b][n - 1], c.V[b][n - 1] = k[b].double(), v[b].double()
        keep_K, keep_V = c.K, c.V
        c.K, c.V = [x[:n] for x, n in zip(c.K, lens)], [x[:n] for x, n in zip(c.V, lens)]
        c.kv = lens
        check_attention(c, o, lse)
        check_scores(c, lse, old, a)
        c.K, c.V, c.kv = keep_K, keep_V, full


def test_serving_steps(gpu_lib):
    """A prompt, then single tokens, then a cut of the cache, then more tokens,
    against a simulation in float64."""
    fa = gpu_lib
    torch.manual_seed(0)
    H, H_kv, d, ps, keep, first, recent = 4, 2, 64, 16, 48, 2, 8
    g, alpha, dev = H // H_kv, 1 / math.sqrt(64), "cuda"
    prompt = [70, 33]
    B, W = 2, 8
    pool = torch.full((2 * 2 * W, 2, ps, H_kv, d), math.nan, dtype=torch.bfloat16, device=dev)
    kp, vp = pool[:, 0], pool[:, 1]
    table = torch.arange(B * W, device=dev, dtype=torch.int32).reshape(B, W)
    spare = table + B * W
    kv_len = torch.zeros(B, dtype=torch.int32, device=dev)
    scores = torch.zeros(B, H_kv, W * ps, device=dev)
    hist = [[([], [], []) for _ in range(H_kv)] for _ in range(B)]       # k, v, weight of every cached token

    def step(q_len):
        T = sum(q_len)
        cu = torch.tensor([0, q_len[0], T], dtype=torch.int32, device=dev)
        q = torch.randn(T, H, d, device=dev).bfloat16()
        k, v = (torch.randn(T, H_kv, d, device=dev).bfloat16() for _ in range(2))
        kv_len.add_(cu[1:] - cu[:-1])
        fa.paged_append(k, v, kp, vp, table, kv_len, cu)
        o, lse = fa.attention_paged(q, kp, vp, table, kv_len, cu, max_q=max(q_len))
        fa.paged_scores(q, lse, kp, table, kv_len, cu, max_q=max(q_len), scores=scores, out=scores)
        assert fa.fa_check_status() == fa.FA_OK
        t = 0
        for b in range(B):
            for i in range(q_len[b]):
                for h in range(H_kv):
                    ks, vs, ws = hist[b][h]
                    ks.append(k[t + i, h].double())
                    vs.append(v[t + i, h].double())
                    ws.append(0.0)
            for h in range(H_kv):
                ks, vs, ws = hist[b][h]
                K, V, n = torch.stack(ks), torch.stack(vs), len(ks)
                for i in range(q_len[b]):
                    p = n - q_len[b] + i
                    for j in range(g):
                        s = alpha * (K[:p + 1] @ q[t + i, h * g + j].double())
                        w = torch.softmax(s, 0)
                        ref = w @ V[:p + 1]
                        tol = 1.05 * 2.0 ** -8 * (w @ V[:p + 1].abs() + 2 * ref.abs()) + 1e-5
                        assert ((o[t + i, h * g + j].double() - ref).abs() <= tol).all()
                        for x, y in enumerate(w.tolist()):
                            ws[x] += y
                assert torch.allclose(scores[b, h, :n].double().cpu(), torch.tensor(ws, dtype=torch.float64),
                                      rtol=1e-4, atol=1e-6)
            t += q_len[b]

    step(prompt)
    step([1, 1])
    step([1, 3])
    kept, cut, new_len = fa.paged_evict(kp, vp, scores, table, kv_len, spare, keep, first, recent)
    assert fa.fa_check_status() == fa.FA_OK and new_len.tolist() == [48, 37]
    for b in range(B):
        for h in range(H_kv):
            ids = kept[b, h, :int(new_len[b])].tolist()
            n = int(kv_len[b])
            assert ids == _expected_kept(scores[b, h].tolist(), n, keep, first, recent)
            hist[b][h] = tuple([x[i] for i in ids] for x in hist[b][h])
    table.copy_(spare)
    kv_len.copy_(new_len)
    scores[:, :, :keep] = cut
    step([1, 1])
    step([2, 1])


# ---- what a row or a token that is not finite may touch ----

@pytest.mark.parametrize("q_len,H,d,window,first", [
    ([70, 9], 8, 128, (-1, 0), 0), ([70, 9], 8, 64, (20, 0), 3), ([130, 1], 6, 128, (40, 2), 0),
    ([5, 1], 4, 64, (-1, 0), 0), ([7, 2], 4, 128, (6, 0), 2)])
def test_scores_a_nan_row_stays_with_the_tokens_it_sees(gpu_lib, q_len, H, d, window, first):
    c = Cache(q_len, [400, 150], H, 2, d, 16, seed=d)
    _, lse = attend(gpu_lib, c, window, first)
    kw = dict(max_q=max(q_len), window=window, first=first)
    want = gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], **kw)
    assert want.isfinite().all()
    m, n = c.q_len[0], c.kv[0]
    j = torch.arange(want.shape[2], device="cuda")
    for i in (0, m // 2, m - 1):
        bad = lse.clone()
        bad[H - 1, i] = math.nan                 # a head of K/V head 1
        got = gpu_lib.paged_scores(c.q, bad, c.k_pages, *c.args()[2:], **kw)
        p = n - m + i
        sees = (j < n) & ((j <= p + window[1]) if window[1] >= 0 else (j < n))
        if window[0] >= 0:
            sees &= (j >= p - window[0]) | (j < first)
        assert torch.isnan(got[0, 1, sees]).all()
        assert torch.equal(got[0, 1, ~sees], want[0, 1, ~sees])
        assert torch.equal(got[0, 0], want[0, 0]) and torch.equal(got[1], want[1])
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK


@pytest.mark.parametrize("q_len,H,H_kv,d", [([1, 1], 4, 1, 128), ([3, 1], 6, 2, 64), ([90, 40], 6, 2, 128),
                                            ([90, 40], 8, 2, 64)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_an_infinite_key_that_nobody_weighs(gpu_lib, q_len, H, H_kv, d, dt):
    # a score of -inf has weight 0, as one of -30000 / 8 has (2^-5000)
    c = Cache(q_len, [700, 300], H, H_kv, d, 16, dt, seed=d)
    c.q[:, :, 0] = -1
    got = []
    for far in (30000.0, math.inf):
        for pos in (3, 500):
            key = c.K[0][pos:pos + 1].to(DT[dt])
            key[0, 0, 0] = far
            c.put(0, pos, key, c.V[0][pos:pos + 1].to(DT[dt]))
        o, lse = attend(gpu_lib, c)
        got.append((o, lse, gpu_lib.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], max_q=max(q_len))))
    for x, y in zip(*got):
        assert torch.isfinite(x).all() and torch.equal(x, y)
    assert (got[1][2][0, 0, [3, 500]] == 0).all()
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK


# (capacity 80 and 48 tokens) kv_len, cu_q: a full cache, a chunk over the
# edge, offsets behind the packed rows, lengths of any value
@pytest.mark.parametrize("kv,cu", [
    ([81, 40], [0, 1, 4]), ([80, 50], [0, 2, 7]), ([83, 49], [0, 5, 7]), ([70, 48], [0, 3, 11]),
    ([70, 48], [0, 9, 9]), ([-1, 48], [0, 2, 7]), ([2**31 - 1, 30], [0, 4, 7]), ([60, -2**31], [0, 4, 7]),
    ([60, 40], [-2, 4, 7])])
@pytest.mark.parametrize("dt,d", [("bf16", 64), ("fp16", 128)])
def test_append_skips_what_has_no_slot(gpu_lib, kv, cu, dt, d):
    c = Cache([1, 1], [80, 48], 2, 2, d, 16, dt, seed=3)
    table = c.table[:, :5].clone()
    table[1, 3:] = -1
    width = (5, 3)                               # pages that exist
    T = 7
    k, v = torch.randn(2, T, 2, d, device="cuda").to(DT[dt])
    want_k, want_v = c.k_pages.clone(), c.v_pages.clone()
    for b in range(2):
        for t in range(max(cu[b], 0), min(cu[b + 1], T)):
            p = kv[b] - cu[b + 1] + t
            if 0 <= p < 16 * width[b]:
                page = int(table[b, p // 16])
                want_k[page, p % 16], want_v[page, p % 16] = k[t], v[t]
    lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
    cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
    gpu_lib.paged_append(k, v, c.k_pages, c.v_pages, table, lens, cu_q)
    assert gpu_lib.fa_check_status() == gpu_lib.FA_ERR_BAD_INDEX
    for got, want in ((c.k_pages, want_k), (c.v_pages, want_v)):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("q_len,H", [([1, 1, 2], 4), ([40, 1, 7], 8)])
def test_scores_of_lengths_out_of_range(gpu_lib, q_len, H):
    # a sequence whose own numbers are out of range hands out nothing: the
    # weights that its cache has collected stay
    fa = gpu_lib
    c = Cache(q_len, [160, 100, 80], H, 2, 64, 16, seed=4)
    _, lse = attend(fa, c)
    table = c.table[:, :10].contiguous()                 # 160 tokens
    old = torch.rand(3, 2, 170, device="cuda")
    kw = dict(max_q=max(q_len), scores=old)
    want = fa.paged_scores(c.q, lse, c.k_pages, table, c.kv_len, c.cu_q, out=old.clone(), **kw)
    for n0 in (161, 2 ** 31 - 1):
        lens = c.kv_len.clone()
        lens[0] = n0
        got = fa.paged_scores(c.q, lse, c.k_pages, table, lens, c.cu_q, out=old.clone(), **kw)
        assert fa.fa_check_status() == fa.FA_ERR_BAD_INDEX
        assert torch.equal(got[0], old[0]) and torch.equal(got[1:], want[1:])
    cu_q = c.cu_q.clone()
    cu_q[3] = c.T + 1
    got = fa.paged_scores(c.q, lse, c.k_pages, table, c.kv_len, cu_q, out=old.clone(), **kw)
    assert fa.fa_check_status() == fa.FA_ERR_BAD_INDEX
    assert torch.equal(got[2], old[2]) and torch.equal(got[:2], want[:2])


@pytest.mark.parametrize("q_len,H,window,first", [([1, 1], 4, (-1, 0), 0), ([60, 3], 8, (-1, 0), 0),
                                                  ([60, 3], 8, (30, 2), 5), ([5, 60], 8, (-1, -1), 0)])
@pytest.mark.parametrize("L", [1, 100, 128, 256, 299])
def test_scores_narrower_than_the_cache(gpu_lib, q_len, H, window, first, L):
    # the weights that there is room for are those of the whole cache
    fa = gpu_lib
    c = Cache(q_len, [300, 70], H, 2, 64, 16, seed=L)
    _, lse = attend(fa, c, window, first)
    kw = dict(max_q=max(q_len), window=window, first=first)
    old = torch.rand(2, 2, 304, device="cuda")
    want = fa.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], scores=old, out=old.clone(), **kw)
    check_scores(c, lse, old, want, window, first)
    assert fa.fa_check_status() == fa.FA_OK
    cut = old[:, :, :L].contiguous()
    fa.paged_scores(c.q, lse, c.k_pages, *c.args()[2:], scores=cut, out=cut, **kw)
    assert fa.fa_check_status() == fa.FA_ERR_BAD_INDEX
    assert torch.equal(cut, want[:, :, :L])


def check_evicted(c, scores, dst, keep, first, recent, before, kept, out, new_len):
    """Everything that an eviction writes: kept positions, scores, lengths and the rows of both pools."""
    kv, ps, H_kv = c.kv, c.ps, c.H_kv
    assert new_len.tolist() == [min(n, keep) for n in kv]
    kept_l, rows = kept.tolist(), scores.tolist()
    want_k, want_v = (x.clone() for x in before)
    for b, n in enumerate(kv):
        m = min(n, keep)
        r = torch.arange(m, device="cuda")
        dp = dst[b].long()[r // ps]
        for h in range(H_kv):
            want = _expected_kept(rows[b][h], n, keep, first, recent)
            assert kept_l[b][h] == want + [-1] * (keep - m)
            i = torch.tensor(want, device="cuda", dtype=torch.long)
            if out is not None:
                assert torch.equal(out[b, h, :m], scores[b, h][i]) and (out[b, h, m:] == 0).all()
            sp = c.table[b].long()[i // ps]
            want_k[dp, r % ps, h], want_v[dp, r % ps, h] = before[0][sp, i % ps, h], before[1][sp, i % ps, h]
    for got, want in ((c.k_pages, want_k), (c.v_pages, want_v)):
        assert torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16))


def _evict_case(kv, H_kv, d, ps, dt, keep, seed, side=False):
    per = -(-keep // ps)
    c = Cache([1] * len(kv), kv, H_kv, H_kv, d, ps, dt, seed=seed, spare=per * len(kv) + 2, side=side)
    dst = c.free[:per * len(kv)].reshape(len(kv), per).contiguous()
    scores = _score_rows("plain", (len(kv), H_kv, c.table.shape[1] * ps), seed)
    scores[:, :, 1::3] = 0.25                    # equal ones among them
    return c, dst, scores


# B * H_kv at and around the border between choosing and moving in one kernel
# and in two (102 of them on 152 SMs), far above it and below
@pytest.mark.parametrize("B,H_kv,d,ps,dt", [(16, 8, 64, 64, "fp16"), (16, 8, 128, 16, "bf16"), (13, 8, 128, 256, "fp16"),
                                            (51, 2, 64, 8, "bf16"), (101, 1, 64, 16, "fp16"), (40, 5, 128, 32, "fp16"),
                                            (3, 8, 128, 64, "fp16")])
@pytest.mark.parametrize("keep,first,recent", [(96, 4, 20), (70, 0, 0), (64, 40, 24), (1, 0, 0), (130, 0, 129)])
def test_evict_batches(gpu_lib, B, H_kv, d, ps, dt, keep, first, recent):
    some = [keep - 1, keep, keep + 1, 300, 1, 0, 129, 260]       # below, at and above keep
    kv = [some[(3 * i) % 8] for i in range(B)]
    c, dst, scores = _evict_case(kv, H_kv, d, ps, dt, keep, B + keep, side=B == 13)
    before = c.k_pages.clone(), c.v_pages.clone()
    kept, out, new_len = gpu_lib.paged_evict(c.k_pages, c.v_pages, scores, c.table, c.kv_len, dst, keep, first, recent)
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK
    check_evicted(c, scores, dst, keep, first, recent, before, kept, out, new_len)


def test_evict_batch_of_long_caches(gpu_lib):
    # a table too wide for keys in shared memory, no scores wanted, tables and
    # scores of different widths
    fa = gpu_lib
    kv = [100, 49500, 3000, 1024, 1500, 700] + [600] * 7
    keep, first, recent, ps, d, H_kv = 1024, 4, 200, 64, 64, 8
    c, dst, scores = _evict_case(kv, H_kv, d, ps, "bf16", keep, 5)
    assert c.table.shape[1] * ps > 49152
    before = c.k_pages.clone(), c.v_pages.clone()
    kept = torch.full((len(kv), H_kv, keep), -1, dtype=torch.int32, device="cuda")
    new_len = torch.empty(len(kv), dtype=torch.int32, device="cuda")
    rc = fa.fa_paged_evict(c.k_pages, c.v_pages, scores, c.table, c.kv_len, dst, kept, None, new_len, len(kv), H_kv, d,
                           ps, c.k_pages.shape[0], c.table.shape[1], dst.shape[1], scores.shape[2], ps * H_kv * d, keep,
                           first, recent)
    assert rc == fa.FA_OK and fa.fa_check_status() == fa.FA_OK
    check_evicted(c, scores, dst, keep, first, recent, before, kept, None, new_len)


@pytest.mark.parametrize("n,keep,d,ps", [(40001, 5000, 128, 64), (70000, 65537, 64, 256)])
def test_evict_long_moves_its_rows(gpu_lib, n, keep, d, ps):
    c, dst, scores = _evict_case([n], 1, d, ps, "fp16", keep, n)
    before = c.k_pages.clone(), c.v_pages.clone()
    kept, out, new_len = gpu_lib.paged_evict(c.k_pages, c.v_pages, scores, c.table, c.kv_len, dst, keep, 4, 100)
    assert gpu_lib.fa_check_status() == gpu_lib.FA_OK
    check_evicted(c, scores, dst, keep, 4, 100, before, kept, out, new_len)


@pytest.mark.parametrize("B,H_kv", [(16, 8), (3, 4)])
def test_evict_in_place_lengths(gpu_lib, B, H_kv):
    # the new lengths may replace the old ones where they are
    fa = gpu_lib
    kv = [(700 * i) % 1500 + 1 for i in range(B)]
    keep, first, recent = 200, 4, 50
    c, dst, scores = _evict_case(kv, H_kv, 64, 16, "bf16", keep, B)
    before = c.k_pages.clone(), c.v_pages.clone()
    graph, lens, kept, out = torch.cuda.CUDAGraph(), c.kv_len.clone(), None, None
    for turn in range(6):
        for x, y in zip((c.k_pages, c.v_pages), before):
            x.copy_(y)
        lens.copy_(c.kv_len)
        if turn < 2:
            kept, out, m = fa.paged_evict(c.k_pages, c.v_pages, scores, c.table, lens, dst, keep, first, recent,
                                          new_len=lens)
        elif turn == 2:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                kept, out, m = fa.paged_evict(c.k_pages, c.v_pages, scores, c.table, lens, dst, keep, first, recent,
                                              new_len=lens)
        if turn >= 2:
            graph.replay()
        assert m is lens and fa.fa_check_status() == fa.FA_OK
        check_evicted(c, scores, dst, keep, first, recent, before, kept, out, m)


def test_evict_refuses_outputs_that_lie_in_its_inputs(gpu_lib):
    fa = gpu_lib
    c, dst, scores = _evict_case([200, 300], 2, 64, 16, "bf16", 320, 1)
    scores = scores[:, :, :320].contiguous()
    lens = torch.tensor([200, 300, 0], dtype=torch.int32, device="cuda")
    for kw in (dict(scores_out=scores), dict(new_len=lens[1:])):
        with pytest.raises(fa.FaError):
            fa.paged_evict(c.k_pages, c.v_pages, scores, c.table, lens[:2], dst, 320, **kw)
    assert fa.fa_check_status() == fa.FA_OK and lens.tolist() == [200, 300, 0]


def test_pages_of_one_head_in_either_order(gpu_lib):
    c = Cache([2, 1], [100, 33], 4, 1, 64, 16, seed=2)
    want = attend(gpu_lib, c)
    for name in ("k_pages", "v_pages"):
        pages = getattr(c, name)
        n, ps, hk, d = pages.shape
        other = torch.empty(n, hk, ps, d, dtype=pages.dtype, device="cuda").transpose(1, 2)
        setattr(c, name, other.copy_(pages))
    assert c.k_pages.stride(2) != 64
    got = attend(gpu_lib, c)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
