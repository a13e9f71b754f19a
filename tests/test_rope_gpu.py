"""GPU checks of rotary positions against float64: fa_rope and
fa_paged_rope_append.

Tolerance, per element, with u the half step of the 16-bit type (2^-8 bf16,
2^-11 fp16), pair (x0, x1), scale m: the angle is off by pi (2^-25 + 2^-31) rad
(its conversion to FP32 half-turns) and by p 2^-52 (64-bit angles, here and in
the reference), cos and sin by two FP32 steps (2^-22), the two products and
their sum by half a step each (together 2^-23 of |x0| + |x1|): below
(2^-20.5 + p 2^-52) m (|x0| + |x1|).  The result is rounded once, u |y|, or half
a subnormal step, 2^-25 (fp16).
"""
import math

import pytest
import torch

import exact_attention_forward_fa_gb300 as fa

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def turned(x, pos, freq, scale, inter, back=False):
    """(y, |x0| + |x1| of each element's pair), float64; x [..., heads, d], pos [...]."""
    rot = 2 * freq.numel()
    a = pos.double()[..., None] * freq
    c, s = torch.cos(a)[..., None, :] * scale, torch.sin(a)[..., None, :] * scale
    if back:
        s = -s
    x = x.double()
    y, size = x.clone(), torch.zeros_like(x)
    i0 = slice(0, rot, 2) if inter else slice(0, rot // 2)
    i1 = slice(1, rot, 2) if inter else slice(rot // 2, rot)
    u, w = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = u * c - w * s, w * c + u * s
    size[..., i0] = size[..., i1] = u.abs() + w.abs()
    return y, size


def check(got, x, pos, freq, scale, inter, dt, back=False):
    y, size = turned(x, pos, freq, scale, inter, back)
    far = pos.double().abs()[..., None, None]
    tol = U[dt] * y.abs() + (2.0 ** -20.5 + far * 2.0 ** -52) * abs(scale) * size + 2.0 ** -25
    rot = 2 * freq.numel()
    assert torch.equal(got[..., rot:], x[..., rot:])
    bad = (got.double() - y).abs() > tol
    assert not bad.any(), (int(bad.sum()), float((got.double() - y).abs().max()))


def randn(*shape, dt="bf16", seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dt])


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 48), (256, 256), (256, 112)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_rope(gpu_lib, d, rot, inter, dt):
    for B, N, H, Hk in [(1, 1, 1, 1), (2, 37, 3, 1), (1, 300, 12, 4)]:
        q, k = randn(B, N, H, d, dt=dt, seed=N), randn(B, N, Hk, d, dt=dt, seed=N + 1)
        w, m = fa.rope_frequencies(rot, scaling="yarn", factor=8.0, original=2048)
        pos = torch.arange(N, device="cuda").expand(B, N)
        qo, ko = fa.rope(q, k, w, scale=m, interleaved=inter)
        check(qo, q, pos, w, m, inter, dt)
        check(ko, k, pos, w, m, inter, dt)
        # back again, with positions of their own
        at = torch.randint(-5, 1 << 20, (B, N), device="cuda", dtype=torch.int32)
        qb, kb = fa.rope(q, k, w, positions=at, scale=m, interleaved=inter, inverse=True)
        check(qb, q, at, w, m, inter, dt, back=True)
        check(kb, k, at, w, m, inter, dt, back=True)


@pytest.mark.parametrize("pos", [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 24, 987654321])
def test_far_positions(gpu_lib, pos):
    """Whole turns are dropped exactly: frequencies that are dyadic fractions of a
    turn have known angles at any position."""
    w = 2 * math.pi * torch.tensor([0.25, 0.125, 2.0 ** -20, 0.5, 1.0, 3.25, 2.0 ** -31, 0.0], dtype=torch.float64,
                                   device="cuda")
    x = randn(1, 1, 64, seed=3)
    at = torch.tensor([pos], dtype=torch.int32, device="cuda")
    y, _ = fa.rope(x, None, w, positions=at)
    # the turns taken modulo one in integers (each frequency times 2^31 is whole)
    f = [1 << 29, 1 << 28, 1 << 11, 1 << 30, 1 << 31, 13 << 29, 1, 0]
    turn = torch.tensor([(pos * i % (1 << 31)) / 2.0 ** 31 for i in f], dtype=torch.float64, device="cuda")
    want, size = turned(x, torch.ones(1, device="cuda"), 2 * math.pi * turn, 1.0, False)
    # (2 pi f rounded to 53 bits turns p 2^-53 relative away from p f)
    tol = U["bf16"] * want.abs() + (2.0 ** -20.5 + abs(pos) * 21 * 2.0 ** -52) * size
    assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("base,scaling,factor", [(1e4, None, 1.0), (5e5, "linear", 4.0), (1e4, "ntk", 8.0),
                                                 (1e4, "yarn", 16.0)])
def test_frequencies(gpu_lib, base, scaling, factor):
    rot = 64
    w, m = fa.rope_frequencies(rot, base, scaling, factor, original=4096)
    w = w.cpu()
    for c in range(rot // 2):
        plain = base ** (-2 * c / rot)
        if scaling is None:
            want = plain
        elif scaling == "linear":
            want = plain / factor
        elif scaling == "ntk":
            want = (base * factor ** (rot / (rot - 2))) ** (-2 * c / rot)
        else:
            assert plain / factor * (1 - 1e-15) <= w[c] <= plain * (1 + 1e-15)
            turns = 4096 * plain / (2 * math.pi)
            if turns > 32 * 1.4:        # (the ramp's ends are whole pairs: one pair is a factor of 1.34)
                want = plain
            elif turns < 1 / 1.4:
                want = plain / factor
            else:
                continue
        assert abs(w[c] - want) <= 1e-14 * want
    assert m == pytest.approx(0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def test_layouts(gpu_lib):
    """Slices of fused rows, packed tensors, in place, q alone, no tokens."""
    B, N, H, Hk, d = 2, 19, 4, 2, 64
    w, _ = fa.rope_frequencies(d)
    rows = randn(B, N, H + 2 * Hk, d, seed=5)
    q, k = rows[:, :, :H], rows[:, :, H:H + Hk]
    pos = torch.arange(N, device="cuda").expand(B, N)
    qo, ko = fa.rope(q, k, w)
    check(qo, q, pos, w, 1.0, False, "bf16")
    check(ko, k, pos, w, 1.0, False, "bf16")
    before = rows.clone()
    fa.rope(q, k, w, q_out=q, k_out=k)                       # in place within the fused rows
    assert torch.equal(rows[:, :, :H], qo) and torch.equal(rows[:, :, H:H + Hk], ko)
    assert torch.equal(rows[:, :, H + Hk:], before[:, :, H + Hk:])
    packed = before.reshape(B * N, H + 2 * Hk, d)
    at = pos.reshape(-1).int().contiguous()
    qp, kp = fa.rope(packed[:, :H], packed[:, H:H + Hk], w, positions=at)
    assert torch.equal(qp.reshape(qo.shape), qo) and torch.equal(kp.reshape(ko.shape), ko)
    alone, none = fa.rope(q.contiguous(), None, w)
    assert none is None
    empty, _ = fa.rope(q[:, :0], None, w)
    assert empty.shape == (B, 0, H, d)
    # an output in the part of the rows that is no input of the call
    wide = before.clone()
    fa.rope(wide[:, :, :2], None, w, q_out=wide[:, :, 4:6])
    assert torch.equal(wide[:, :, 4:6], qo[:, :, :2]) and torch.equal(wide[:, :, :4], before[:, :, :4])


def test_gradient(gpu_lib):
    """<dy, rope(x)> = <rope_inverse(dy), x>, and against differences in float64."""
    w, m = fa.rope_frequencies(64, scaling="yarn", factor=4.0, original=128)
    x, dy = randn(1, 50, 3, 64, dt="fp16", seed=8), randn(1, 50, 3, 64, dt="fp16", seed=9)
    dx, _ = fa.rope(dy, None, w, scale=m, inverse=True)
    pos = torch.arange(50, device="cuda").expand(1, 50)
    check(dx, dy, pos, w, m, False, "fp16", back=True)
    leaf = x.double().requires_grad_()
    (turned(leaf, pos, w, m, False)[0] * dy.double()).sum().backward()
    assert ((dx.double() - leaf.grad).abs() <= U["fp16"] * leaf.grad.abs() + 2.0 ** -20 * 8).all()
    # the rotation is linear: a difference of any step is the derivative
    i, h = (0, 49, 2, 5), 0.5
    up, down = x.double(), x.double()
    up[i] += h
    down[i] -= h
    f = [(turned(v, pos, w, m, False)[0] * dy.double()).sum() for v in (up, down)]
    assert abs(float((f[0] - f[1]) / (2 * h) - leaf.grad[i])) < 1e-9


def paged(q_len, kv, H, Hk, d, ps, dt, seed=0, width=0):
    g = torch.Generator("cuda").manual_seed(seed)
    pages = [-(-n // ps) for n in kv]
    n = sum(pages) + 2
    perm = torch.randperm(n, generator=g, device="cuda").int()
    table = torch.full((len(kv), max(max(pages), width, 1)), 1 << 30, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(pages):
        table[b, :m] = perm[at:at + m]
        at += m
    T = sum(q_len)
    rows = torch.randn((T, H + 2 * Hk, d), generator=g, device="cuda").to(DT[dt])
    kp = torch.randn((n, ps, Hk, d), generator=g, device="cuda").to(DT[dt])
    vp = torch.randn((n, ps, Hk, d), generator=g, device="cuda").to(DT[dt])
    cu = torch.tensor([0] + torch.tensor(q_len).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    return (rows[:, :H], rows[:, H:H + Hk], rows[:, H + Hk:], kp, vp, table,
            torch.tensor(kv, dtype=torch.int32, device="cuda"), cu)


@pytest.mark.parametrize("q_len,kv", [([1], [1]), ([1], [40]), ([1, 0, 5, 1], [17, 9, 5, 64]), ([33, 1, 70], [33, 1, 200])])
@pytest.mark.parametrize("d,rot,H,Hk,ps,inter,dt", [(64, 64, 4, 4, 16, False, "bf16"), (128, 64, 12, 2, 32, True, "fp16"),
                                                    (128, 128, 8, 1, 8, False, "bf16"), (64, 32, 1, 1, 64, True, "fp16")])
def test_paged_append(gpu_lib, q_len, kv, d, rot, H, Hk, ps, inter, dt):
    q, k, v, kp, vp, table, kv_len, cu = paged(q_len, kv, H, Hk, d, ps, dt)
    w, m = fa.rope_frequencies(rot, scaling="linear", factor=2.0)
    k0, v0 = kp.clone(), vp.clone()
    off = torch.tensor([1000 * b for b in range(len(kv))], dtype=torch.int32, device="cuda")
    for offsets in (None, off):
        kp.copy_(k0)
        vp.copy_(v0)
        out = fa.paged_rope_append(q, k, v, kp, vp, table, kv_len, cu, w, scale=m, interleaved=inter, offsets=offsets)
        want_v, touched = v0.clone(), torch.zeros(k0.shape[:2], dtype=torch.bool, device="cuda")
        at = 0
        for b, (nq, n) in enumerate(zip(q_len, kv)):
            for i in range(nq):
                p = n - nq + i
                page, slot = int(table[b, p // ps]), p % ps
                pos = torch.tensor([p + (1000 * b if offsets is not None else 0)], device="cuda")
                check(kp[page, slot][None], k[at:at + 1], pos, w, m, inter, dt)
                check(out[at:at + 1], q[at:at + 1], pos, w, m, inter, dt)
                want_v[page, slot] = v[at]
                touched[page, slot] = True
                at += 1
        assert torch.equal(vp, want_v)
        assert torch.equal(kp[~touched], k0[~touched])
    assert fa.fa_check_status() == fa.FA_OK


def test_paged_equals_rope_then_append(gpu_lib):
    """The fused call gives the bits of fa_rope and fa_paged_append one after the other."""
    q, k, v, kp, vp, table, kv_len, cu = paged([300, 1, 77], [300, 500, 99], 8, 2, 128, 16, "bf16")
    w, _ = fa.rope_frequencies(128)
    pos = torch.cat([torch.arange(0, 300), torch.tensor([499]), torch.arange(22, 99)]).int().cuda()
    q1, k1 = fa.rope(q, k, w, positions=pos)
    kp1, vp1 = kp.clone(), vp.clone()
    fa.paged_append(k1, v.contiguous(), kp1, vp1, table, kv_len, cu)
    out = fa.paged_rope_append(q, k, v, kp, vp, table, kv_len, cu, w)
    assert torch.equal(out, q1) and torch.equal(kp, kp1) and torch.equal(vp, vp1)


@pytest.mark.parametrize("q_len", [[1] * 5000 + [0, 7] + [2] * 1500, [3, 0, 1, 4000, 0, 0, 1, 65, 4100, 2, 129]])
def test_runs_over_sequences_and_pages(gpu_lib, q_len):
    """More tokens than warps: a warp's tokens go on into the next page and sequence,
    past empty ones, to rows behind the last."""
    kv = [n + (17 * b) % 23 for b, n in enumerate(q_len)]
    q, k, v, kp, vp, table, kv_len, cu = paged(q_len, kv, 2, 1, 64, 8, "bf16")
    w, _ = fa.rope_frequencies(64)
    off = torch.tensor([(31 * b) % 1001 for b in range(len(kv))], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n - m, n) + (31 * b) % 1001 for b, (m, n) in enumerate(zip(q_len, kv))]).int().cuda()
    q1, k1 = fa.rope(q, k, w, positions=pos)
    kp1, vp1 = kp.clone(), vp.clone()
    fa.paged_append(k1, v.contiguous(), kp1, vp1, table, kv_len, cu)
    q, k, v = (torch.cat([x, x[:3000]]).contiguous() for x in (q, k, v))
    out = torch.full_like(q, 7.0)
    fa.paged_rope_append(q, k, v, kp, vp, table, kv_len, cu, w, offsets=off, q_out=out)
    T = sum(q_len)
    assert torch.equal(out[:T], q1) and (out[T:] == 7).all()
    assert torch.equal(kp, kp1) and torch.equal(vp, vp1)
    assert fa.fa_check_status() == fa.FA_OK


def test_paged_behind_and_full(gpu_lib):
    """Rows behind cu_q[B] stay; tokens without a slot are dropped and reported."""
    q, k, v, kp, vp, table, kv_len, cu = paged([2, 3], [10, 12], 2, 1, 64, 8, "bf16")
    w, _ = fa.rope_frequencies(64)
    q, k, v = (torch.cat([x, x[:4]]).contiguous() for x in (q, k, v))
    out = torch.full_like(q, 7.0)
    fa.paged_rope_append(q, k, v, kp, vp, table, kv_len, cu, w, q_out=out)
    assert (out[5:] == 7).all() and not (out[:5] == 7).all()
    assert fa.fa_check_status() == fa.FA_OK
    k0 = kp.clone()
    full = torch.tensor([table.shape[1] * 8 + 1, 2], dtype=torch.int32, device="cuda")   # a full cache; 3 new of 2
    fa.paged_rope_append(q, k, v, kp, vp, table, full, cu, w, q_out=out)
    torch.cuda.synchronize()
    assert fa.fa_check_status() == fa.FA_ERR_BAD_INDEX
    assert fa.fa_check_status() == fa.FA_OK
    changed = (kp != k0).flatten(2).any(-1)
    assert int(changed.sum()) <= 1 + 2          # the last slot of row 0's table (if a page), places 0 and 1 of row 1


def test_graph_and_stream(gpu_lib):
    q, k, v, kp, vp, table, kv_len, cu = paged([1] * 9, [5 + 7 * b for b in range(9)], 8, 2, 128, 16, "bf16", width=8)
    w, _ = fa.rope_frequencies(128)
    out = torch.zeros(9, 8, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.paged_rope_append(q, k, v, kp, vp, table, kv_len, cu, w, q_out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            fa.paged_rope_append(q, k, v, kp, vp, table, kv_len, cu, w, q_out=out)
    torch.cuda.current_stream().wait_stream(side)
    first = out.clone()
    kv_len += 1
    graph.replay()
    torch.cuda.synchronize()
    pos = (kv_len - 1).long()
    check(out, q, pos, w, 1.0, False, "bf16")
    assert not torch.equal(out, first)
    # a stream argument
    a, _ = fa.rope(q, None, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b, _ = fa.rope(q, None, w)
    assert torch.equal(a, b)
    assert fa.fa_check_status() == fa.FA_OK
