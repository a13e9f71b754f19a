"""GPU checks of the gradients of attention on a mask plan (fa_bwd_masked)
against float64 and against differences.

Tolerances, per element, u the half step of the 16-bit type:

* P = exp(S - LSE) is off, relative, by the errors of S and of LSE (each d 2^-23
  alpha sum |q||k| and, with a bias, 24 2^-24 (|bias| + |LSE| + 8); see
  test_masked_gpu.py) and 2^-18 (exp2 of an argument in FP32, the sums);
* dV = P^T dO: P is rounded to the type: (u + e) sum P |dO|, and u |dV| for the
  output;
* dS = P (dP - D), D = dO . O with O rounded to the type (u sum |dO||O|): with
  size = P (|dP| + sum |dO||O|), off by (u + e) size, rounded again: 2 u size;
  the products sum size times |K| (|Q|), the output's rounding is u of it.
5 % for second-order terms and the FP32 sums.
"""
import math

import pytest
import torch

import exact_attention_forward_fa_gb300 as fa
from tests._masked import DT, check_backward, check_forward, reference, slopes_of
from tests.test_masked_gpu import HEADS, MASKS, make, pack

pytestmark = pytest.mark.gpu


def gradient(q, docs, dt, seed=1, nan=True):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(q.shape, generator=g, device="cuda").to(DT[dt])
    if nan:
        for b, at in enumerate(docs):
            x[b, :at[0]] = math.nan
            x[b, at[-1]:] = math.nan
    return x


@pytest.mark.parametrize("m", range(len(MASKS)))
@pytest.mark.parametrize("bias", [False, True])
def test_backward(gpu_lib, m, bias):
    N, docs, prefix, left, right = MASKS[m]
    for H, Hk, d, dt in HEADS:
        q, k, v, plan, seen = make(len(docs), N, H, Hk, d, dt, docs, prefix, left, right, seed=m)
        dout = gradient(q, docs, dt)
        slopes = slopes_of(H) if bias else None
        sinks = torch.linspace(-2, 3, H, device="cuda") if H == 3 else None
        alpha = 1.0 / math.sqrt(d)
        o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes, sinks=sinks)
        *got, dsinks = fa.attention_backward_masked(q, k, v, o, lse, dout, plan, slopes=slopes, sinks=sinks)
        assert fa.fa_check_status() == fa.FA_OK
        r = reference(q, k, v, seen, slopes, sinks, alpha, dout)
        check_forward(o, lse, r, dt, d, alpha, slopes)
        check_backward(got, r, dt, d, slopes)
        if sinks is not None:
            live = ~torch.isinf(r["lse"])
            p = torch.where(live, torch.exp(sinks.double()[None, :, None] - r["lse"]), torch.zeros_like(r["lse"]))
            want, size = -(p * r["delta"]).sum((0, 2)), (p * r["edelta"]).sum((0, 2))
            assert ((dsinks.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -14) * size + 1e-6).all()


def test_against_differences(gpu_lib):
    """The gradient of a sum over O along a direction, against differences of the forward in float64."""
    N, H, Hk, d = 90, 2, 1, 64
    docs, prefix = [[3, 40, 88]], [[20, 0]]
    q, k, v, plan, seen = make(1, N, H, Hk, d, "fp16", docs, prefix, 25, 0, seed=6, nan=False)
    slopes = slopes_of(H)
    dout = gradient(q, docs, "fp16", nan=False)
    o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes)
    dq, dk, dv, _ = fa.attention_backward_masked(q, k, v, o, lse, dout, plan, slopes=slopes)
    g = torch.Generator("cuda").manual_seed(3)
    for name, x, dx in (("q", q, dq), ("k", k, dk), ("v", v, dv)):
        way = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        f = []
        for sign in (1, -1):
            t = {"q": q.double(), "k": k.double(), "v": v.double()}
            t[name] = t[name] + sign * h * way
            f.append(float((reference(t["q"], t["k"], t["v"], seen, slopes, None, 0.125)["o"] * dout.double()).sum()))
        want = (f[0] - f[1]) / (2 * h)
        size = float((dx.double() * way).norm())
        # thousands of independent roundings of at most 3 u each
        assert abs(float((dx.double() * way).sum()) - want) <= 12 * 2.0 ** -11 * size + 1e-5 * abs(want), name


def test_bad_documents_stay_in_bounds(gpu_lib):
    N, d = 300, 64
    q, k, v, do = (torch.randn(1, N, 2, d, device="cuda").bfloat16() for _ in range(4))
    for docs in ([[0, 400]], [[-5, 300]], [[200, 100, 300]], [[0, 2 ** 31 - 1, 300]]):
        plan = fa.mask_plan(torch.tensor(docs, dtype=torch.int32, device="cuda"), N, window=(5, 7))
        o, lse = fa.attention_masked(q, k, v, plan)
        fa.attention_backward_masked(q, k, v, o, lse, do, plan)
        assert fa.fa_check_status() == fa.FA_ERR_BAD_INDEX


def test_one_document_equals_the_dense_backward(gpu_lib):
    B, N, H, d = 2, 900, 3, 128
    q, k, v, plan, _ = make(B, N, H, H, d, "bf16", [[0, N]] * B)
    do = gradient(q, [[0, N]] * B, "bf16")
    o, lse = fa.attention(q, k, v, causal=True)
    dense = fa.attention_backward(q, k, v, o, lse, do, causal=True)
    got = fa.attention_backward_masked(q, k, v, o, lse, do, plan)
    for x, y in zip(got, dense):
        # the same products in the same order up to the masked tiles' zeros
        assert (x.float() - y.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max()


def test_repeats_its_bits_and_captured(gpu_lib):
    """Eager, again, and replayed with other documents in the same plan."""
    N, H, Hk, d = 1200, 8, 2, 64
    lists = [pack(N, [500, 30, 600]), [0, 100, N, N]]
    q, k, v, plan, _ = make(2, N, H, Hk, d, "bf16", lists, nan=False)
    do = gradient(q, lists, "bf16", nan=False)
    slopes = slopes_of(H)

    def step():
        o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes)
        return (o, lse) + fa.attention_backward_masked(q, k, v, o, lse, do, plan, slopes=slopes)[:3]

    first = step()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, step()))
    docs = torch.tensor(lists, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            fa.mask_plan(docs, N, out=plan)
            outs = step()
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, outs))
    docs.copy_(torch.tensor([pack(N, [1, 2, 1100]), [5, 700, 701, 701]], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    fresh = fa.mask_plan(docs, N)
    o, lse = fa.attention_masked(q, k, v, fresh, slopes=slopes)
    again = (o, lse) + fa.attention_backward_masked(q, k, v, o, lse, do, fresh, slopes=slopes)[:3]
    assert all(torch.equal(x, y) for x, y in zip(again, outs))
    assert fa.fa_check_status() == fa.FA_OK


def test_many_units(gpu_lib):
    N, H, Hk, d = 3000, 24, 4, 128
    docs = [pack(N, [1, 1200, 64, 900, 800])]
    q, k, v, plan, seen = make(1, N, H, Hk, d, "bf16", docs, [[0, 500, 64, 0, 700]], 1000, 0, seed=9)
    do = gradient(q, docs, "bf16")
    slopes = slopes_of(H)
    o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes)
    *got, _ = fa.attention_backward_masked(q, k, v, o, lse, do, plan, slopes=slopes)
    assert fa.fa_check_status() == fa.FA_OK
    r = reference(q, k, v, seen, slopes, None, 1 / math.sqrt(d), do)
    check_backward(got, r, "bf16", d, slopes)


def test_training_layer(gpu_lib):
    """A layer's attention as a training step runs it -- plan, rotation of slices of a fused projection, attention,
    gradients, rotation back -- against automatic differentiation in float64, eager and captured.

    Tolerance: the chain's steps as above, taken together in the norm: q and k are rounded after the rotation (u
    each of the scores' arguments), the gradients' errors (at most 3 u of their size, independent from element
    to element) pass the rotation and are rounded again; 8 u of the norm bounds them with the scores' errors, which
    move P by alpha |q| |k| u ~ sqrt(d) u."""
    B, N, H, Hk, d = 2, 333, 4, 2, 64
    docs, prefix = [[0, 100, 101, 320], [5, 200, 333, 333]], [[40, 0, 100], [0, 133, 0]]
    g = torch.Generator("cuda").manual_seed(11)
    rows = torch.randn(B, N, H + 2 * Hk, d, generator=g, device="cuda").bfloat16()
    dout = gradient(rows[:, :, :H], docs, "bf16", nan=False)
    slopes, alpha = slopes_of(H), 1 / math.sqrt(d)
    w, scale = fa.rope_frequencies(d // 2, scaling="yarn", factor=4.0, original=64)
    offsets = torch.tensor(docs, dtype=torch.int32, device="cuda")
    plan = fa.mask_plan(offsets, N, prefix=torch.tensor(prefix, dtype=torch.int32, device="cuda"))

    def step():
        q, k, v = rows[:, :, :H], rows[:, :, H:H + Hk], rows[:, :, H + Hk:]
        qr, kr = fa.rope(q, k, w, positions=plan.positions, scale=scale)
        o, lse = fa.attention_masked(qr, kr, v, plan, slopes=slopes)
        dq, dk, dv, _ = fa.attention_backward_masked(qr, kr, v, o, lse, dout, plan, slopes=slopes)
        dq, dk = fa.rope(dq, dk, w, positions=plan.positions, scale=scale, inverse=True, q_out=dq, k_out=dk)
        return o, dq, dk, dv

    got = step()
    # float64: the same mathematics on leaves of its own
    from tests._masked import visible
    leaf = [x.double().requires_grad_() for x in (rows[:, :, :H], rows[:, :, H:H + Hk], rows[:, :, H + Hk:])]
    a = plan.positions.double()[..., None, None] * w

    def turn(x):
        u, v = x[..., :d // 4], x[..., d // 4:d // 2]
        c, s = torch.cos(a) * scale, torch.sin(a) * scale
        return torch.cat([u * c - v * s, v * c + u * s, x[..., d // 2:]], -1)

    q, k = turn(leaf[0]), turn(leaf[1])
    dist = (torch.arange(N)[:, None] - torch.arange(N)[None]).abs().double().cuda()
    outs = []
    for b in range(B):
        seen = visible(docs[b], prefix[b], N, -1, 0)
        alive = seen.any(1)[:, None]
        for h in range(H):
            x = alpha * q[b, :, h] @ k[b, :, h // 2].T - slopes[h].double() * dist
            p = torch.softmax(x.masked_fill(~seen & alive, -math.inf), -1) * alive
            outs.append(p @ leaf[2][b, :, h // 2])
    o = torch.stack(outs).reshape(B, H, N, d).transpose(1, 2)
    (o * dout.double()).sum().backward()
    for x, y in zip(got, [o.detach()] + [x.grad for x in leaf]):
        assert float((x.double() - y).norm() / y.norm()) <= 8 * 2.0 ** -8
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = step()
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, captured))
    assert fa.fa_check_status() == fa.FA_OK


def test_two_streams_and_threads(gpu_lib):
    """Calls on two streams at once, and from two host threads, give the bits of calls one after the other."""
    import threading
    cases = []
    for seed, (N, d) in enumerate([(1100, 64), (700, 128)]):
        docs = [pack(N, [300, 390])]
        q, k, v, plan, _ = make(1, N, 8, 4, d, "bf16", docs, None, -1, -1, seed=seed, nan=False)
        do = gradient(q, docs, "bf16", nan=False)
        cases.append((q, k, v, plan, do, slopes_of(8)))

    def step(c):
        q, k, v, plan, do, slopes = c
        o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes)
        return (o, lse) + fa.attention_backward_masked(q, k, v, o, lse, do, plan, slopes=slopes)[:3]

    alone = [step(c) for c in cases]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got[i] = step(cases[i])
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert fa.fa_check_status() == fa.FA_OK
