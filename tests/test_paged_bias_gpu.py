"""GPU checks of attention over a paged cache with a bias that depends on the
distance (fa_fwd_paged_bias), against float64.

Tolerances: those of test_paged_gpu.py for O and LSE, and for the bias at most
24 FP32 steps of quantities no larger than the bias, the LSE and 8:
e = 24 2^-24 (|bias| + |LSE| + 8), weighted by the softmax in LSE, and 2 e A
(A: softmax-weighted |v|) in O.
"""
import math

import pytest
import torch

import exact_attention_forward_fa_gb300 as fa
from tests._masked import slopes_of
from tests.test_paged_gpu import DT, LENS, U, Cache

pytestmark = pytest.mark.gpu


def check(c, o, lse, slopes, window=(-1, 0), first=0, alpha=None):
    u, alpha = U[c.dt], 1 / math.sqrt(c.d) if alpha is None else alpha
    for b in range(len(c.kv)):
        m, n = c.q_len[b], c.kv[b]
        if m == 0:
            continue
        got = o[c.cu[b]:c.cu[b] + m].double().transpose(0, 1)
        stat = lse[:, c.cu[b]:c.cu[b] + m].double()
        s, e = c.rows(b, window, first, alpha)
        p = torch.arange(n - m, n, device="cuda")[:, None]
        bias = slopes.double()[:, None, None] * (p - torch.arange(n, device="cuda")[None]).abs()
        s = s - bias
        z = torch.logsumexp(s, -1) if n else torch.full(s.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        empty = torch.isinf(z)
        w = torch.where(empty[..., None], torch.zeros_like(s), torch.exp(s - z[..., None]))
        v = c.V[b].transpose(0, 1).repeat_interleave(c.H // c.H_kv, 0)
        ref, mag = w @ v, w @ v.abs()
        far = 24 * 2.0 ** -24 * ((w * bias.abs()).sum(-1) + z.abs().nan_to_num(posinf=0.0) + 8)
        tol = 1.05 * (u * (mag + 2 * ref.abs()) + 2 * far[..., None] * mag) + 1e-6
        assert torch.isfinite(got).all()
        err = (got - ref).abs()
        assert (err <= tol).all(), f"sequence {b}: {float((err / tol).max()):.2f} of the tolerance"
        assert (stat[empty] == -math.inf).all() and (got[empty] == 0).all()
        ltol = (e.amax(-1) if n else 0.0) + far + 2.0 ** -20 + 2.0 ** -22 * z.abs()
        assert ((stat - z).abs()[~empty] <= ltol[~empty]).all()


def attend(c, slopes, window=(-1, 0), first=0, **kw):
    o, lse = fa.attention_paged(c.q, *c.args(), max_q=max(1, max(c.q_len)), window=window, first=first, slopes=slopes, **kw)
    assert fa.fa_check_status() == fa.FA_OK
    return o, lse


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dt,d,H,H_kv,ps", [("bf16", 128, 8, 2, 16), ("fp16", 64, 4, 4, 32), ("bf16", 64, 6, 2, 8),
                                            ("fp16", 128, 7, 1, 256)])
def test_bias(gpu_lib, lens, dt, d, H, H_kv, ps):
    c = Cache(*LENS[lens], H, H_kv, d, ps, dt, seed=len(lens), behind=3, gap=2)
    out = torch.full((c.T, H, d), 7.0, dtype=DT[dt], device="cuda")
    lse = torch.full((H, c.T), 7.0, device="cuda")
    attend(c, slopes_of(H), out=out, lse=lse)
    check(c, out, lse, slopes_of(H))
    n = c.cu[-1]                                # rows behind the last sequence stay as they were
    assert (out[n:] == 7).all() and (lse[:, n:] == 7).all()


@pytest.mark.parametrize("window,first", [((-1, -1), 0), ((0, 0), 1), ((100, 0), 4), ((31, 5), 0), ((300, -1), 130),
                                          ((2**31 - 1, 2**31 - 1), 2**31 - 1), ((-1, 3), 9)])
@pytest.mark.parametrize("lens", ["tokens", "empty_rows", "mixed"])
def test_bias_and_masks(gpu_lib, lens, window, first):
    c = Cache(*LENS[lens], 8, 2, 128 if lens == "mixed" else 64, 16, seed=first % 97, side=True)
    o, lse = attend(c, slopes_of(8), window, first)
    check(c, o, lse, slopes_of(8), window, first)


@pytest.mark.parametrize("slope", [0.0, 3.0, -0.05, -1.0])
@pytest.mark.parametrize("q", [1, 150])
def test_extreme_slopes(gpu_lib, q, slope):
    """None, one that leaves a few keys, biases that grow with the distance."""
    c = Cache([q, 1], [700, 1500], 4, 2, 128, 16, seed=2)
    slopes = torch.full((4,), slope, device="cuda")
    o, lse = attend(c, slopes)
    check(c, o, lse, slopes)
    if slope == 0.0:
        o2, lse2 = fa.attention_paged(c.q, *c.args(), max_q=q)
        assert (o.float() - o2.float()).abs().max() <= 2.0 ** -7 * 4 and (lse - lse2).abs().max() < 1e-5


def test_long_axis_repeats_its_bits(gpu_lib):
    c = Cache([1, 2], [70001, 33000], 8, 1, 128, 64)
    slopes = slopes_of(8) * 0.01
    o, lse = attend(c, slopes)
    check(c, o, lse, slopes)
    for _ in range(3):
        o2, lse2 = attend(c, slopes)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_serving_chain(gpu_lib):
    """Prompt and tokens of a model with rotary positions and a distance bias through the paged cache equal the
    masked call over the whole document."""
    H, H_kv, d, ps, n, m = 4, 2, 64, 16, 200, 3
    g = torch.Generator("cuda").manual_seed(0)
    q, k, v = (torch.randn(n + m, h, d, generator=g, device="cuda").bfloat16() for h in (H, H_kv, H_kv))
    w, scale = fa.rope_frequencies(d)
    slopes = slopes_of(H)
    pool = torch.full((2, 16, ps, H_kv, d), math.nan, dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(16, generator=g, device="cuda").int()[None]
    got = []
    for lo, hi in [(0, n)] + [(n + i, n + i + 1) for i in range(m)]:
        kv_len = torch.tensor([hi], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda")
        qr = fa.paged_rope_append(q[lo:hi], k[lo:hi], v[lo:hi], pool[0], pool[1], table, kv_len, cu, w, scale=scale)
        o, _ = fa.attention_paged(qr, pool[0], pool[1], table, kv_len, cu, max_q=hi - lo, slopes=slopes)
        got.append(o)
    assert fa.fa_check_status() == fa.FA_OK
    plan = fa.mask_plan(torch.tensor([[0, n + m]], dtype=torch.int32, device="cuda"), n + m)
    qr, kr = fa.rope(q[None], k[None], w, positions=plan.positions, scale=scale)
    o, _ = fa.attention_masked(qr, kr, v[None], plan, slopes=slopes)
    # equal inputs; P is rounded against another reference and O once in each
    assert (torch.cat(got).float() - o[0].float()).abs().max() <= 4 * 2.0 ** -8 * v.float().abs().max()
