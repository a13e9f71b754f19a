"""GPU checks of fa_bwd_masked in fp16 over the range of its inputs: small gradients, small values and long documents, whose
P and dS lie where fp16 is spaced by 2^-24 whatever their size.

Tolerances, u = 2^-11 the half step:

* in the norm of a gradient: every P, dS and O is rounded by at most u of itself, independently of the others, and
  the outputs once more; what such roundings leave of a sum over thousands of terms is at most 2 u of its norm.  Outputs
  below 2^-14 are spaced by 2^-24, each off by 2^-25 at most: 2^-25 sqrt(elements).
* dsinks = -sum p D, by D's error: O is rounded by u of itself, 2 u sum p sum |dO||O| with the FP32 sums;
* equal weights: P = 1 / N is one number, its rounding does not average out: u of sum P |dO|, 2^-18 for LSE and exp2, and
  the output's u.  Nor do the sum's truncations, of terms of one sign: the tensor core may drop what of a term lies below
  2^-23 of the sum so far (test_masked_gpu.py), which grows evenly: n 2^-24 of it for n terms.  (60000: 3.6e-3, of which
  3.3e-4 were seen; every 97th alone: 4e-5.)"""
import math

import pytest
import torch

import exact_attention_forward_fa_gb300 as fa
from tests._masked import reference, slopes_of, visible
from tests.test_masked_gpu import pack

pytestmark = pytest.mark.gpu
U16 = 2.0 ** -11


def near(got, want, name):
    err, lim = float((got.double() - want).norm()), 2 * U16 * float(want.norm()) + 2.0 ** -25 * math.sqrt(want.numel())
    assert err <= lim, (name, err / lim)


def inputs(N, H, Hk, d, docs, g_scale, v_scale, seed):
    """q, k, v slices of fused rows, dout; padding NaN."""
    g = torch.Generator("cuda").manual_seed(seed)
    rows = torch.randn(1, N, H + 2 * Hk, d, generator=g, device="cuda")
    rows[:, :, H + Hk:] *= v_scale
    rows[:, :docs[0]] = rows[:, docs[-1]:] = math.nan
    rows = rows.half()
    do = torch.randn(1, N, H, d, generator=g, device="cuda") * g_scale
    do[:, :docs[0]] = do[:, docs[-1]:] = math.nan
    return rows[:, :, :H], rows[:, :, H:H + Hk], rows[:, :, H + Hk:], do.half()


@pytest.mark.parametrize("g_exp,v_exp", [(0, 0), (-6, 0), (-10, 0), (-13, 0), (0, -9), (-8, -6), (6, 2)])
@pytest.mark.parametrize("d,bias", [(64, False), (64, True), (128, False), (128, True)])
def test_small_gradients(gpu_lib, d, bias, g_exp, v_exp):
    N, H, Hk = 4200, 2, 1
    docs = [70, 4166]
    q, k, v, do = inputs(N, H, Hk, d, docs, 2.0 ** g_exp, 2.0 ** v_exp, seed=d)
    slopes = 0.002 * slopes_of(H) if bias else None
    sinks = torch.tensor([1.0, 6.0], device="cuda")
    plan = fa.mask_plan(torch.tensor([docs], dtype=torch.int32, device="cuda"), N, window=(-1, -1))
    o, lse = fa.attention_masked(q, k, v, plan, slopes=slopes, sinks=sinks)
    dq, dk, dv, ds = fa.attention_backward_masked(q, k, v, o, lse, do, plan, slopes=slopes, sinks=sinks)
    assert fa.fa_check_status() == fa.FA_OK
    r = reference(q, k, v, [visible(docs, None, N, -1, -1)], slopes, sinks, 1 / math.sqrt(d), do)
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        near(x, r[name], name)
    live = ~torch.isinf(r["lse"])
    p = torch.where(live, torch.exp(sinks.double()[None, :, None] - r["lse"]), torch.zeros_like(r["lse"]))
    want, size = -(p * r["delta"]).sum((0, 2)), (p * r["edelta"]).sum((0, 2))
    assert ((ds.double() - want).abs() <= 2 * U16 * size).all(), (ds, want)


@pytest.mark.parametrize("each", [1, 97])
@pytest.mark.parametrize("d", [64, 128])
def test_equal_weights_of_a_long_document(gpu_lib, d, each):
    """q = 0: P = 1 / N, 279.6 of fp16's smallest steps; the products follow from sums over the document.  Gradients at
    every token, or at every 97th."""
    N, g = 60000, torch.Generator("cuda").manual_seed(d)
    q = torch.zeros(1, N, 1, d, dtype=torch.float16, device="cuda")
    k, v = (torch.randn(1, N, 1, d, generator=g, device="cuda").half() for _ in range(2))
    do = (0.5 + torch.rand(1, N, 1, d, generator=g, device="cuda")).half()
    do[:, torch.arange(N, device="cuda") % each > 0] = 0
    plan = fa.mask_plan(torch.tensor([[0, N]], dtype=torch.int32, device="cuda"), N, window=(-1, -1))
    o, lse = fa.attention_masked(q, k, v, plan)
    dq, dk, dv, _ = fa.attention_backward_masked(q, k, v, o, lse, do, plan)
    assert fa.fa_check_status() == fa.FA_OK
    K, V, G = (x[0, :, 0].double() for x in (k, v, do))
    want = G.mean(0)
    assert ((dv[0, :, 0].double() - want).abs() <= (2 * U16 + 2.0 ** -18 + N / each * 2.0 ** -24) * want).all()
    D = (G * V.mean(0)).sum(1, keepdim=True)
    near(dq[0, :, 0], (G @ (V.T @ K) - D * K.sum(0)) / (N * math.sqrt(d)), "dq")
    assert not dk.any()


def test_nothing_to_learn(gpu_lib):
    """dout = 0 gives gradients of 0, whatever the scale."""
    N, d = 500, 64
    q, k, v, do = inputs(N, 2, 2, d, [0, N], 0.0, 1.0, seed=1)
    plan = fa.mask_plan(torch.tensor([[0, 200, N]], dtype=torch.int32, device="cuda"), N)
    o, lse = fa.attention_masked(q, k, v, plan)
    assert not any(x.any() for x in fa.attention_backward_masked(q, k, v, o, lse, do, plan)[:3])


def test_infinities_stay_where_they_are(gpu_lib):
    """An infinity in dout takes the scale away; documents that share no tile with its keep their gradients."""
    N, d = 1024, 64
    docs = [0, 384, 1024]
    q, k, v, do = inputs(N, 2, 1, d, docs, 1.0, 1.0, seed=5)
    plan = fa.mask_plan(torch.tensor([docs], dtype=torch.int32, device="cuda"), N)
    o, lse = fa.attention_masked(q, k, v, plan)
    clean = fa.attention_backward_masked(q, k, v, o, lse, do, plan)[:3]
    do = do.clone()
    do[0, 100, 1, 7] = math.inf
    for x, y in zip(fa.attention_backward_masked(q, k, v, o, lse, do, plan)[:3], clean):
        # (each is within 2 u of the same gradient)
        assert float((x[:, 384:].double() - y[:, 384:].double()).norm()) <= 4 * U16 * float(y[:, 384:].double().norm())
        assert torch.isfinite(y).all() and not torch.isfinite(x[:, :384]).all()


def test_captured_with_gradients_of_another_size(gpu_lib):
    """The scale is found anew at each replay; a call repeats its bits; two streams at once."""
    N, H, Hk, d = 1500, 8, 2, 64
    docs = pack(N, [600, 30, 800])
    q, k, v, do = inputs(N, H, Hk, d, [docs[0], docs[-1]], 1.0, 1.0, seed=8)
    do = torch.nan_to_num(do)
    plan = fa.mask_plan(torch.tensor([docs], dtype=torch.int32, device="cuda"), N)
    o, lse = fa.attention_masked(q, k, v, plan)

    def step(g):
        return fa.attention_backward_masked(q, k, v, o, lse, g, plan)[:3]

    small = (do * 2.0 ** -9)
    first, other = step(do), step(small)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, step(do)))
    side, buf = torch.cuda.Stream(), do.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = step(buf)
    torch.cuda.current_stream().wait_stream(side)
    for g, want in ((do, first), (small, other), (do, first)):
        buf.copy_(g)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, g in zip(streams, (do, small)):
            with torch.cuda.stream(s):
                got.append(step(g))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(x, (first, other)[i % 2]))
    assert fa.fa_check_status() == fa.FA_OK
