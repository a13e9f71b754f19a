"""GPU checks of attention on a mask plan against float64: fa_mask_plan,
fa_fwd_masked.

Tolerances, per element, with u the half step of the 16-bit type and everything
else FP32:

* O = sum_j p_j v_j / sum_j p_j, p_j rounded to the type before the product and
  summed as rounded, O rounded once: |dO| <= u (A + |O|) + u |O| with A the
  softmax-weighted |v|; a score's error e moves O by at most 2 e A; 5 % for
  second-order terms.
* A score is an FP32 dot product of d terms, off by at most d 2^-23 alpha
  sum |q||k| (2^-23 a step: the tensor core may truncate); exp2, log2 and the
  row's sums add 2^-20.  The bias is formed in at most 24 FP32 steps of
  quantities no larger than the bias, the reference (at most LSE + 8 in
  magnitude beside it) and their sum: 24 2^-24 (|bias| + |LSE| + 8), the bias
  weighted by the softmax (what a term weighs little moves little).
"""
import math

import pytest
import torch

import exact_attention_forward_fa_gb300 as fa
from tests._masked import DT, U, check_forward, reference, slopes_of, visible

pytestmark = pytest.mark.gpu


def make(B, N, H, Hk, d, dt, docs, prefix=None, left=-1, right=0, seed=0, scale=1.0, nan=True):
    """Inputs whose padding is NaN, the plan, and the mask from its definition."""
    g = torch.Generator("cuda").manual_seed(seed)
    q, k, v = ((s * torch.randn(B, N, h, d, generator=g, device="cuda")).to(DT[dt])
               for h, s in ((H, scale), (Hk, scale), (Hk, 1.0)))
    seen = [visible(docs[b], prefix[b] if prefix else None, N, left, right) for b in range(B)]
    if nan:
        for b in range(B):
            dead = torch.ones(N, dtype=torch.bool, device="cuda")
            dead[docs[b][0]:docs[b][-1]] = False
            for x in (q, k, v):
                x[b, dead] = math.nan
    plan = fa.mask_plan(torch.tensor(docs, dtype=torch.int32, device="cuda"), N,
                        prefix=torch.tensor(prefix, dtype=torch.int32, device="cuda") if prefix else None,
                        window=(left, right))
    return q, k, v, plan, seen


def pack(N, lens, lo=0):
    """Offsets of documents of these lengths from lo on, cut at N."""
    at = [lo]
    for n in lens:
        at.append(min(at[-1] + n, N))
    return at


# (N, documents of each sequence, prefixes, left, right)
MASKS = [
    (1, [[0, 1]], None, -1, 0),
    (5, [[0, 2, 2, 4]], None, -1, 0),
    (5, [[1, 1]], None, -1, -1),                                     # nothing but padding
    (127, [[0, 127]], [[50]], -1, 0),
    (128, [[0, 1, 128]], None, -1, -1),
    (129, [[0, 128, 129], [3, 100, 100]], [[128, 1], [97, 0]], -1, 0),
    (300, [pack(300, [1] * 300)], None, -1, 0),                      # documents of one token
    (300, [pack(300, [17] * 18)], None, -1, -1),
    (513, [pack(513, [100, 300, 90])], [[10, 300, 0]], -1, 0),
    (513, [pack(513, [256, 257])], None, 37, 0),
    (640, [pack(640, [5, 300, 300], 20)], [[5, 120, 300]], 64, 0),
    (640, [pack(640, [640])], None, 100, 50),
    (1000, [[0, 400, 999], [10, 1000, 1000]], [[390, 0], [500, 0]], -1, 0),
    (1000, [[0, 1000, 1000], [300, 301, 700]], None, -1, -1),
    (1024, [pack(1024, [128] * 8)], None, 0, 0),                     # each token itself
    (1500, [pack(1500, [3, 777, 500], 130)], [[1, 700, 0]], 300, 20),
]
HEADS = [(1, 1, 64, "bf16"), (4, 2, 128, "fp16"), (3, 3, 128, "bf16"), (6, 1, 64, "fp16")]


@pytest.mark.parametrize("m", range(len(MASKS)))
@pytest.mark.parametrize("bias", [False, True])
def test_forward(gpu_lib, m, bias):
    N, docs, prefix, left, right = MASKS[m]
    for H, Hk, d, dt in HEADS:
        q, k, v, plan, seen = make(len(docs), N, H, Hk, d, dt, docs, prefix, left, right, seed=m)
        slopes = slopes_of(H) if bias else None
        sinks = torch.linspace(-2, 3, H, device="cuda") if H == 3 else None
        alpha = 1.0 / math.sqrt(d)
        o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes, sinks=sinks)
        assert fa.fa_check_status() == fa.FA_OK
        r = reference(q, k, v, seen, slopes, sinks, alpha)
        check_forward(o, lse, r, dt, d, alpha, slopes)


def test_plan_positions(gpu_lib):
    docs = [[0, 3, 3, 10], [2, 5, 9, 9]]
    plan = fa.mask_plan(torch.tensor(docs, dtype=torch.int32, device="cuda"), 12)
    assert plan.positions.tolist() == [[0, 1, 2, 0, 1, 2, 3, 4, 5, 6, 0, 0], [0, 0, 0, 1, 2, 0, 1, 2, 3, 0, 0, 0]]


def test_bad_documents_are_cut_off(gpu_lib):
    """Offsets that fall or leave the sequence are reported; what is launched stays in bounds."""
    N, d = 300, 64
    q, k, v = (torch.randn(1, N, 2, d, device="cuda").bfloat16() for _ in range(3))
    for docs in ([[0, 400]], [[-5, 300]], [[200, 100, 300]], [[0, 2 ** 31 - 1, 300]], [[-2 ** 31, 2 ** 31 - 1]]):
        for left, right in ((-1, 0), (-1, -1), (2 ** 31 - 1, 2 ** 31 - 1), (5, 7)):
            plan = fa.mask_plan(torch.tensor(docs, dtype=torch.int32, device="cuda"), N, window=(left, right))
            fa.attention_masked(q, k, v, plan)
            assert fa.fa_check_status() == fa.FA_ERR_BAD_INDEX
    plan = fa.mask_plan(torch.tensor([[0, 100]], dtype=torch.int32, device="cuda"), N,
                        prefix=torch.tensor([[101]], dtype=torch.int32, device="cuda"))
    o, lse = fa.attention_masked(q, k, v, plan)
    assert fa.fa_check_status() == fa.FA_ERR_BAD_INDEX
    check_forward(o, lse, reference(q, k, v, [visible([0, 100], [100], N, -1, 0)], None, None, 0.125), "bf16", d, 0.125, None)


@pytest.mark.parametrize("scale", [0.0, 30.0])
@pytest.mark.parametrize("neg", [False, True])
def test_extreme_scores(gpu_lib, scale, neg):
    """Scores that are all equal, or of hundreds; biases that grow with the distance instead of falling."""
    N, H, d = 700, 4, 64
    docs = [pack(N, [50, 600])]
    q, k, v, plan, seen = make(1, N, H, 2, d, "bf16", docs, None, -1, -1, seed=4, scale=scale)
    slopes = torch.tensor([0.0, 1e-4, 0.7, 3.0], device="cuda") * (-1 if neg else 1)
    o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes)
    check_forward(o, lse, reference(q, k, v, seen, slopes, None, 0.125), "bf16", d, 0.125, slopes)


def test_plain_masks_equal_the_dense_calls(gpu_lib):
    """One document over the whole sequence is the dense kernel's mask; many of them are the calls one by one."""
    B, N, H, Hk, d = 2, 777, 4, 2, 128
    q, k, v, plan, _ = make(B, N, H, Hk, d, "bf16", [[0, N]] * B)
    o, lse = fa.attention_masked(q, k, v, plan)
    oc, lc = fa.attention(q, k, v, causal=True)
    assert (o.float() - oc.float()).abs().max() <= 2 * U["bf16"] * 4 and (lse - lc).abs().max() < 1e-5
    lens = [130, 5, 300, 342]
    docs = [pack(N, lens)] * B
    plan = fa.mask_plan(torch.tensor(docs, dtype=torch.int32, device="cuda"), N)
    o, _ = fa.attention_masked(q, k, v, plan)
    at = 0
    for n in lens:
        part, _ = fa.attention(*(x[:, at:at + n].contiguous() for x in (q, k, v)), causal=True)
        assert (o[:, at:at + n].float() - part.float()).abs().max() <= 2 * U["bf16"] * 4
        at += n


def test_slices_and_outputs(gpu_lib):
    """Slices of fused rows give the bits of contiguous tensors; given outputs; no LSE."""
    B, N, H, Hk, d = 2, 300, 4, 2, 64
    rows = torch.randn(B, N, H + 2 * Hk, d, device="cuda").half()
    q, k, v = rows[:, :, :H], rows[:, :, H:H + Hk], rows[:, :, H + Hk:]
    plan = fa.mask_plan(torch.tensor([[0, 100, 290]] * B, dtype=torch.int32, device="cuda"), N, window=(-1, -1))
    o, lse = fa.attention_masked(q, k, v, plan)
    o2, lse2 = fa.attention_masked(q.contiguous(), k.contiguous(), v.contiguous(), plan)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    out = torch.full_like(o, 5.0)
    got, none = fa.attention_masked(q, k, v, plan, out=out, want_lse=False)
    assert got is out and none is None and torch.equal(out, o)


def test_repeats_its_bits(gpu_lib):
    N = 2000
    q, k, v, plan, _ = make(2, N, 8, 2, 128, "bf16", [pack(N, [900, 30, 700]), [0, N, N, N]], nan=False)
    first = fa.attention_masked(q, k, v, plan, slopes=slopes_of(8))
    for _ in range(5):
        again = fa.attention_masked(q, k, v, plan, slopes=slopes_of(8))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_many_units(gpu_lib):
    """More units than SMs several times over, many heads in groups, a long ragged sequence."""
    N, H, d = 5000, 48, 64
    docs = [pack(N, [1, 2000, 64, 1500, 1400])]
    q, k, v, plan, seen = make(1, N, H, 4, d, "bf16", docs, [[0, 500, 64, 0, 1000]], 1800, 0, seed=9)
    slopes = slopes_of(H)
    o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes)
    assert fa.fa_check_status() == fa.FA_OK
    for h in (0, 13, 47):
        r = reference(q[:, :, h:h + 1], k[:, :, h // 12:h // 12 + 1], v[:, :, h // 12:h // 12 + 1], seen, slopes[h:h + 1], None, 0.125)
        check_forward(o[:, :, h:h + 1], lse[:, h:h + 1], r, "bf16", d, 0.125, slopes[h:h + 1])


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_reaches_the_rows_that_see_it(gpu_lib, d, bias):
    """A NaN key makes the rows that see it NaN, a NaN query its own row, and no others."""
    N, H = 700, 2
    docs = [pack(N, [100, 450, 140])]
    q, k, v, plan, seen = make(1, N, H, H, d, "bf16", docs, None, 200, 0, seed=21)
    slopes = slopes_of(H) if bias else None
    clean = fa.attention_masked(q, k, v, plan, slopes=slopes)
    q, k = q.clone(), k.clone()
    k[0, 300, 1, 5] = math.nan
    q[0, 610, 1, 0] = math.nan
    o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes)
    hit = seen[0][:, 300].clone()
    hit[610] = True
    assert torch.isnan(o[0, hit, 1]).all() and torch.isnan(lse[0, 1, hit]).all()
    # the other rows: their maximum may have been taken at another tile, nothing else
    assert torch.equal(o[0, :, 0], clean[0][0, :, 0]) and torch.equal(lse[0, 0], clean[1][0, 0])
    rest = ~hit
    assert torch.isfinite(o[0, rest, 1]).all()
    assert (o[0, rest, 1].float() - clean[0][0, rest, 1].float()).abs().max() <= 2 * U["bf16"] * 4
    same = lse[0, 1, rest], clean[1][0, 1, rest]
    assert ((same[0] - same[1]).abs().nan_to_num() < 1e-5).all()
