"""Host-side checks (no GPU) of the entry points for masks of documents and
prefixes, rotary positions and the paged attention with a distance bias: argument
validation returns the documented codes before touching CUDA, and the torch
wrappers refuse layouts that the C entry points could not be told about."""
import pytest
import torch

import exact_attention_forward_fa_gb300 as fa
from exact_attention_forward_fa_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


A = 0x10000          # fake, 16-byte aligned device addresses (never dereferenced)
INV, UNS, MIS, BIG = (fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_MISALIGNED, fa.FA_ERR_TOO_LARGE)
LAUNCH = (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)         # what a valid call returns without a GPU
M = 1 << 20          # a distance at which the tensors of these calls share nothing


def _plan(lib, docs=A, prefix=None, plan=A, pos=None, B=2, N=300, D=3, wl=-1, wr=0):
    return lib.fa_mask_plan(docs, prefix, plan, pos, B, N, D, wl, wr, None)


@pytest.mark.parametrize("kw,code", [
    (dict(docs=None), INV), (dict(plan=None), INV), (dict(B=0), INV), (dict(N=0), INV), (dict(D=0), INV),
    (dict(wl=-2), INV), (dict(wr=-2), INV), (dict(N=-5), INV),
    (dict(docs=A + 2), MIS), (dict(prefix=A + 1), MIS), (dict(pos=A + 2), MIS), (dict(plan=A + 8), MIS),
    (dict(B=65536), BIG), (dict(N=(1 << 30) + 1), BIG), (dict(D=(1 << 30) + 1), BIG),
])
def test_plan_codes(lib, kw, code):
    assert _plan(lib, **kw) == code


def test_plan_bytes(lib):
    # live 16 B, pairs 32 per 256 tokens, two lists of 16 per 128, two intervals of 8 per token
    assert lib.fa_mask_plan_bytes(1, 1) == 16 + 32 + 16 + 16 + 16 + 16
    assert lib.fa_mask_plan_bytes(2, 300) == 32 + 2 * 2 * 32 + 2 * 2 * 3 * 16 + 2 * 2 * 300 * 8
    assert lib.fa_mask_plan_bytes(3, 1 << 30) > 3 * 16 * (1 << 30)
    for B, N in ((0, 5), (5, 0), (65536, 5), (1, (1 << 30) + 1)):
        assert lib.fa_mask_plan_bytes(B, N) == -1


def _fwd(lib, q=A, k=A + M, v=A + 2 * M, o=A + 3 * M, lse=None, plan=A, slopes=None, sinks=None, B=2, H=4, Hk=2, N=300,
         d=64, qs=None, ks=None, vs=None, alpha=0.1, dt=0):
    return lib.fa_fwd_masked(q, k, v, o, lse, plan, slopes, sinks, B, H, Hk, N, d, qs or H * d, ks or Hk * d, vs or Hk * d,
                             alpha, dt, None)


def _bwd(lib, q=A, k=A + M, v=A + 2 * M, o=A + 3 * M, dout=A + 4 * M, lse=A, ws=A, plan=A, slopes=None, sinks=None,
         dq=A + 5 * M, dk=A + 6 * M, dv=A + 7 * M, ds=None, B=2, H=4, Hk=2, N=300, d=64, qs=None, ks=None, vs=None,
         alpha=0.1, dt=0):
    return lib.fa_bwd_masked(q, k, v, o, dout, lse, ws, plan, slopes, sinks, dq, dk, dv, ds, B, H, Hk, N, d, qs or H * d,
                             ks or Hk * d, vs or Hk * d, alpha, dt, None)


BOTH = [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(o=None), INV), (dict(plan=None), INV),
    (dict(B=0), INV), (dict(H=0), INV), (dict(Hk=0), INV), (dict(H=5), INV), (dict(N=0), INV), (dict(d=0), INV),
    (dict(alpha=0.0), INV), (dict(alpha=-1.0), INV), (dict(alpha=float("nan")), INV), (dict(alpha=float("inf")), INV),
    (dict(alpha=1e-40), INV), (dict(dt=2), INV), (dict(qs=255 - 7), INV), (dict(ks=120), INV), (dict(vs=120), INV),
    (dict(d=256), UNS), (dict(d=96), UNS),
    (dict(q=A + 8), MIS), (dict(k=A + M + 2), MIS), (dict(v=A + 2 * M + 4), MIS), (dict(o=A + 3 * M + 8), MIS),
    (dict(plan=A + 8), MIS), (dict(lse=A + 2), MIS), (dict(slopes=A + 2), MIS), (dict(sinks=A + 1), MIS),
    (dict(qs=256 + 4), MIS), (dict(ks=128 + 4), MIS), (dict(vs=128 + 2), MIS),
    (dict(B=65536), BIG), (dict(N=(1 << 30) + 1), BIG), (dict(qs=1 << 34), BIG), (dict(H=1 << 16, Hk=1, B=1 << 14, N=1000), BIG),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(o=A), INV), (dict(o=A + M), INV), (dict(o=A + 2 * M + 16), INV),
    (dict(q=A + 128, qs=1024, o=A, N=1), INV),           # within the same rows
])
def test_forward_codes(lib, kw, code):
    assert _fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(dout=None), INV), (dict(lse=None), INV), (dict(ws=None), INV), (dict(dq=None), INV), (dict(dk=None), INV),
    (dict(dv=None), INV), (dict(ds=A), INV), (dict(dout=A + 4 * M + 8), MIS), (dict(ws=A + 8), MIS),
    (dict(dq=A + 5 * M + 8), MIS), (dict(dk=A + 6 * M + 2), MIS), (dict(dv=A + 7 * M + 4), MIS),
    (dict(sinks=A, ds=A + 2), MIS),
    (dict(dq=A), INV), (dict(dk=A + M), INV), (dict(dv=A + 2 * M), INV), (dict(dq=A + 4 * M), INV), (dict(dk=A + 3 * M), INV),
    (dict(dk=A + 5 * M), INV), (dict(dv=A + 6 * M + 16), INV),
])
def test_backward_codes(lib, kw, code):
    assert _bwd(lib, **kw) == code


def _rope(lib, q=A, k=A + M, qo=A + 2 * M, ko=A + 3 * M, pos=None, w=A, B=2, N=50, H=4, Hk=2, d=64, rot=64, qs=None, ks=None,
          qos=None, kos=None, scale=1.0, inter=0, inv=0, dt=0):
    return lib.fa_rope(q, k, qo, ko, pos, w, B, N, H, Hk, d, rot, qs or H * d, ks or Hk * d, qos or H * d, kos or Hk * d,
                       scale, inter, inv, dt, None)


ROPE = [
    (dict(q=None), INV), (dict(qo=None), INV), (dict(w=None), INV), (dict(H=0), INV), (dict(d=0), INV), (dict(rot=0), INV),
    (dict(rot=128), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(inter=2), INV),
    (dict(dt=2), INV), (dict(qs=248), INV), (dict(qos=248), INV), (dict(ks=120), INV),
    (dict(d=96), UNS), (dict(rot=24), UNS), (dict(rot=2), UNS),
    (dict(q=A + 8), MIS), (dict(k=A + M + 2), MIS), (dict(qo=A + 2 * M + 8), MIS), (dict(w=A + 4), MIS),
    (dict(qs=256 + 4), MIS), (dict(qos=256 + 2), MIS), (dict(ks=128 + 4), MIS),
    (dict(qs=1 << 39), BIG), (dict(qos=1 << 39), BIG), (dict(H=(1 << 20) + 1, qs=1 << 30, qos=1 << 30), BIG),
    (dict(qo=A + 16), INV), (dict(qo=A, qos=512), INV), (dict(qo=A + M), INV),        # overlaps that are not in place
]


@pytest.mark.parametrize("kw,code", ROPE + [
    (dict(k=None), INV), (dict(ko=None), INV), (dict(Hk=-1), INV), (dict(B=0), INV), (dict(N=0), INV), (dict(inv=3), INV),
    (dict(kos=120), INV), (dict(pos=A + 2), MIS), (dict(ko=A + 3 * M + 8), MIS), (dict(kos=128 + 4), MIS),
    (dict(B=1 << 16, N=1 << 16), BIG), (dict(kos=1 << 39), BIG),
    (dict(ko=A + M + 16), INV), (dict(ko=A), INV), (dict(ko=A + 2 * M), INV),
])
def test_rope_codes(lib, kw, code):
    assert _rope(lib, **kw) == code


def _rappend(lib, q=A, k=A + M, v=A + 2 * M, qo=A + 3 * M, kp=A, vp=A, tb=A, kl=A, cu=A, off=None, w=A, B=1, H=4, Hk=2, d=64,
             rot=64, T=3, ps=16, n=4, W=2, qs=None, ks=None, qos=None, pst=None, scale=1.0, inter=0, dt=0):
    return lib.fa_paged_rope_append(q, k, v, qo, kp, vp, tb, kl, cu, off, w, B, H, Hk, d, rot, T, ps, n, W, qs or H * d,
                                    ks or Hk * d, qos or H * d, pst or 16 * 2 * 64, scale, inter, dt, None)


@pytest.mark.parametrize("kw,code", [x for x in ROPE if x[0] != dict(qo=A + M)] + [
    (dict(kp=None), INV), (dict(vp=None), INV), (dict(tb=None), INV), (dict(kl=None), INV), (dict(cu=None), INV),
    (dict(k=None), INV), (dict(v=None), INV), (dict(T=-1), INV), (dict(Hk=0), INV), (dict(B=0), INV), (dict(W=0), INV),
    (dict(pst=2040), INV), (dict(d=256, rot=64, pst=1 << 20), UNS), (dict(ps=24, pst=1 << 20), UNS),
    (dict(kp=A + 8), MIS), (dict(v=A + 2 * M + 8), MIS), (dict(tb=A + 2), MIS), (dict(kl=A + 2), MIS), (dict(cu=A + 2), MIS),
    (dict(off=A + 2), MIS), (dict(pst=2052), MIS), (dict(B=65536), BIG), (dict(qo=A + M), INV), (dict(qo=A + 2 * M), INV),
])
def test_rope_append_codes(lib, kw, code):
    assert _rappend(lib, **kw) == code


def _bias(lib, slopes=A, d=128, H=4, ws=A):
    return lib.fa_fwd_paged_bias(A, A, A, A, A, A, A, A, ws, slopes, 1, H, 2, 3, 3, d, 16, 4, 2, H * d, 16 * 2 * d, 0.1, -1, 0, 0,
                                 0, None)


@pytest.mark.parametrize("kw,code", [(dict(slopes=None), INV), (dict(slopes=A + 2), MIS), (dict(d=96), UNS), (dict(H=5), INV),
                                     (dict(ws=None), INV), (dict(ws=A + 16), MIS)])
def test_paged_bias_codes(lib, kw, code):
    assert _bias(lib, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(), dict(qo=A, ko=A + M), dict(Hk=0, k=None, ko=None), dict(rot=16), dict(d=256, rot=256),
    # q and k are slices of the same rows, rotated where they are or into the rows' third part
    dict(q=A, k=A + 512, qo=A, ko=A + 512, qs=512, ks=512, qos=512, kos=512),
    dict(q=A, Hk=0, k=None, qo=A + 512, ko=None, qs=512, qos=512),
])
def test_valid_rope_calls_reach_the_device(lib, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the gpu tests")
    assert _rope(lib, **kw) in LAUNCH


def test_valid_calls_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the gpu tests")
    for call in (_plan, _fwd, _bwd, _rappend, _bias):
        assert call(lib) in LAUNCH
    # slices of fused rows
    assert _fwd(lib, q=A, k=A + 512, v=A + 768, qs=512, ks=512, vs=512) in LAUNCH


# ---- the torch wrappers ----

def _t(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt)


def _fake_plan(B=2, N=8):
    return fa.MaskPlan(B, N, (-1, 0), torch.zeros(16, dtype=torch.uint8), torch.zeros(B, N, dtype=torch.int32))


@pytest.mark.parametrize("q,k,v", [
    (_t(2, 8, 4, 64).float(), _t(2, 8, 2, 64), _t(2, 8, 2, 64)),
    (_t(2, 8, 4, 64).half(), _t(2, 8, 2, 64), _t(2, 8, 2, 64)),
    (_t(2, 8, 4, 64), _t(2, 8, 2, 64), _t(2, 8, 1, 64)),
    (_t(2, 8, 4, 64), _t(2, 7, 2, 64), _t(2, 7, 2, 64)),
    (_t(2, 8, 4, 64), _t(2, 8, 2, 128), _t(2, 8, 2, 128)),
    (_t(2, 9, 4, 64), _t(2, 9, 2, 64), _t(2, 9, 2, 64)),             # not the plan's N
    (_t(8, 4, 64), _t(8, 2, 64), _t(8, 2, 64)),
    (_t(2, 8, 64, 4).transpose(2, 3), _t(2, 8, 2, 64), _t(2, 8, 2, 64)),
    (_t(2, 4, 8, 64).transpose(1, 2), _t(2, 8, 2, 64), _t(2, 8, 2, 64)),
    (_t(2, 16, 4, 64)[:, :8], _t(2, 8, 2, 64), _t(2, 8, 2, 64)),     # sequences at another distance than their tokens
    (_t(2, 8, 4, 64), _t(2, 8, 2, 64), _t(2, 8, 2, 64)),             # not on a GPU
])
def test_masked_wrappers_refuse(q, k, v):
    with pytest.raises((ValueError, TypeError)):
        fa.attention_masked(q, k, v, _fake_plan())
    with pytest.raises((ValueError, TypeError)):
        fa.attention_backward_masked(q, k, v, q, torch.zeros(2, 4, 8), q, _fake_plan())


@pytest.mark.parametrize("kw", [dict(slopes=torch.zeros(3)), dict(slopes=torch.zeros(4).half()), dict(sinks=torch.zeros(4, 1)),
                                dict(slopes=torch.zeros(8)[::2])])
def test_masked_wrappers_refuse_slopes_and_sinks(kw):
    with pytest.raises(ValueError, match="float32"):
        fa.attention_masked(_t(2, 8, 4, 64), _t(2, 8, 2, 64), _t(2, 8, 2, 64), _fake_plan(), **kw)
    c = dict(k_pages=_t(4, 16, 2, 64), v_pages=_t(4, 16, 2, 64), block_table=torch.zeros(1, 2, dtype=torch.int32),
             kv_len=torch.ones(1, dtype=torch.int32), cu_q=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.attention_paged(_t(3, 4, 64), max_q=3, slopes=torch.zeros(3), **c)


@pytest.mark.parametrize("docs,kw", [
    (torch.zeros(2, 3), {}), (torch.zeros(2, 3, dtype=torch.int64), {}), (torch.zeros(3, dtype=torch.int32), {}),
    (torch.zeros(2, 1, dtype=torch.int32), {}), (torch.zeros(2, 6, dtype=torch.int32)[:, ::2], {}),
    (torch.zeros(2, 3, dtype=torch.int32), dict(prefix=torch.zeros(2, 3, dtype=torch.int32))),
    (torch.zeros(2, 3, dtype=torch.int32), dict(window=(2**32, 0))), (torch.zeros(2, 3, dtype=torch.int32), dict(window=(0, -2**40))),
    (torch.zeros(2, 3, dtype=torch.int32), {}),                      # not on a GPU
])
def test_mask_plan_refuses(docs, kw):
    with pytest.raises(ValueError):
        fa.mask_plan(docs, 8, **kw)


W64 = torch.zeros(32, dtype=torch.float64)


@pytest.mark.parametrize("q,k,w,kw", [
    (_t(2, 8, 4, 64).float(), None, W64, {}), (_t(4, 64), None, W64, {}), (_t(2, 8, 4, 64), None, W64.float(), {}),
    (_t(2, 8, 4, 64), None, W64[None], {}), (_t(2, 8, 4, 64), _t(2, 7, 2, 64), W64, {}),
    (_t(2, 8, 4, 64), _t(2, 8, 2, 64).half(), W64, {}), (_t(2, 8, 4, 64), None, W64, dict(k_out=_t(2, 8, 4, 64))),
    (_t(2, 8, 4, 64), None, W64, dict(positions=torch.zeros(2, 8))),
    (_t(2, 8, 4, 64), None, W64, dict(positions=torch.zeros(16, dtype=torch.int32))),
    (_t(2, 8, 4, 64), None, W64, dict(q_out=_t(2, 8, 2, 64))), (_t(2, 8, 4, 64), None, W64, dict(q_out=_t(2, 8, 4, 64).half())),
    (_t(2, 4, 8, 64).transpose(1, 2), None, W64, {}), (_t(2, 8, 4, 64), None, W64, {}),
])
def test_rope_refuses(q, k, w, kw):
    with pytest.raises((ValueError, TypeError)):
        fa.rope(q, k, w, **kw)


@pytest.mark.parametrize("change", [
    dict(k=_t(3, 1, 64)), dict(v=_t(3, 2, 64).half()), dict(q=_t(2, 4, 64)), dict(q=_t(3, 4, 64).half()), dict(v=_t(3, 4, 64)[:, :2]),
    dict(inv_freq=W64.float()), dict(offsets=torch.zeros(2, dtype=torch.int32)), dict(offsets=torch.zeros(1)),
    dict(q_out=_t(3, 4, 128)), dict(cu_q=torch.zeros(3, dtype=torch.int32)), {},
])
def test_rope_append_refuses(change):
    c = dict(q=_t(3, 4, 64), k=_t(3, 2, 64), v=_t(3, 2, 64), k_pages=_t(4, 16, 2, 64), v_pages=_t(4, 16, 2, 64),
             block_table=torch.zeros(1, 2, dtype=torch.int32), kv_len=torch.ones(1, dtype=torch.int32),
             cu_q=torch.zeros(2, dtype=torch.int32), inv_freq=W64)
    c.update(change)
    with pytest.raises((ValueError, TypeError)):
        fa.paged_rope_append(**c)


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, base=1.0), dict(rot_dim=64, factor=0.5),
                                dict(rot_dim=64, scaling="cubic"), dict(rot_dim=64, scaling="yarn"),
                                dict(rot_dim=2, scaling="ntk", factor=2.0)])
def test_rope_frequencies_refuses(kw):
    with pytest.raises(ValueError):
        fa.rope_frequencies(device="cpu", **kw)
