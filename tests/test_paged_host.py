"""Host-side checks of the paged-cache entry points (no GPU): argument
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
INV, UNS, MIS, BIG = (fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_MISALIGNED,
                      fa.FA_ERR_TOO_LARGE)

# refusals that every entry point shares
SHARED = [
    (dict(kp=None), INV), (dict(tb=None), INV), (dict(kl=None), INV),
    (dict(B=0), INV), (dict(Hk=0), INV), (dict(d=0), INV), (dict(ps=0), INV), (dict(n=0), INV),
    (dict(W=0), INV), (dict(pst=16 * 2 * 128 - 8), INV),
    (dict(d=256), UNS), (dict(d=96), UNS), (dict(ps=4, pst=1 << 20), UNS), (dict(ps=24, pst=1 << 20), UNS),
    (dict(kp=A + 8), MIS), (dict(tb=A + 2), MIS), (dict(kl=A + 1), MIS), (dict(pst=(1 << 20) + 4), MIS),
    (dict(pst=1 << 39), BIG), (dict(B=65536), BIG), (dict(Hk=65536, H=65536, pst=1 << 30, qst=1 << 30), BIG),
]


def _append(lib, k=A, v=A, kp=A, vp=A, tb=A, kl=A, cu=A, B=1, Hk=2, H=None, d=128, T=3, ps=16, n=4, W=2,
            kst=None, pst=None, qst=None):
    return lib.fa_paged_append(k, v, kp, vp, tb, kl, cu, B, Hk, d, T, ps, n, W, kst or qst or 2 * 128,
                               pst or 16 * 2 * 128, None)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(k=None), INV), (dict(v=None), INV), (dict(vp=None), INV), (dict(cu=None), INV), (dict(T=-1), INV),
    (dict(kst=2 * 128 - 8), INV), (dict(kst=2 * 128 + 4), MIS), (dict(k=A + 2), MIS), (dict(vp=A + 4), MIS),
    (dict(cu=A + 2), MIS), (dict(kst=1 << 39), BIG),
])
def test_append_codes(lib, kw, code):
    assert _append(lib, **kw) == code


def _attend(lib, q=A, kp=A, vp=A, tb=A, kl=A, cu=A, o=A, lse=A, ws=A, B=1, H=4, Hk=2, T=3, mq=3, d=128, ps=16,
            n=4, W=2, qst=None, pst=None, alpha=0.1, wl=-1, wr=0, first=0, dt=0):
    return lib.fa_fwd_paged(q, kp, vp, tb, kl, cu, o, lse, ws, B, H, Hk, T, mq, d, ps, n, W, qst or H * d,
                            pst or 16 * 2 * 128, alpha, wl, wr, first, dt, None)


ATTN = [
    (dict(q=None), INV), (dict(cu=None), INV), (dict(T=-1), INV), (dict(mq=0), INV), (dict(H=5), INV),
    (dict(H=0), INV), (dict(qst=4 * 128 - 8), INV), (dict(wl=-2), INV), (dict(wr=-2), INV),
    (dict(first=-1), INV), (dict(alpha=float("nan")), INV), (dict(alpha=float("inf")), INV), (dict(dt=2), INV),
    (dict(alpha=0.0), INV), (dict(alpha=-0.1), INV), (dict(alpha=1e-40), INV), (dict(alpha=3e38), INV),
    (dict(H=258, qst=1 << 20), UNS), (dict(q=A + 8), MIS), (dict(cu=A + 2), MIS), (dict(lse=A + 2), MIS),
    (dict(qst=4 * 128 + 4), MIS), (dict(qst=1 << 39), BIG),
]


@pytest.mark.parametrize("kw,code", SHARED + ATTN + [
    (dict(vp=None), INV), (dict(o=None), INV), (dict(ws=None), INV), (dict(vp=A + 8), MIS), (dict(o=A + 8), MIS),
    (dict(ws=A + 8), MIS), (dict(ws=A + 16), MIS),
])
def test_attention_codes(lib, kw, code):
    assert _attend(lib, **kw) == code


def _scores(lib, q=A, lse=A, kp=A, tb=A, kl=A, cu=A, sin=A, s=A, B=1, H=4, Hk=2, T=3, mq=3, d=128, ps=16, n=4,
            W=2, L=32, qst=None, pst=None, alpha=0.1, wl=-1, wr=0, first=0, dt=0):
    return lib.fa_paged_scores(q, lse, kp, tb, kl, cu, sin, s, B, H, Hk, T, mq, d, ps, n, W, L, qst or H * d,
                               pst or 16 * 2 * 128, alpha, wl, wr, first, dt, None)


@pytest.mark.parametrize("kw,code", SHARED + ATTN + [
    (dict(lse=None), INV), (dict(s=None), INV), (dict(L=0), INV), (dict(s=A + 2), MIS), (dict(sin=A + 1), MIS),
])
def test_scores_codes(lib, kw, code):
    assert _scores(lib, **kw) == code


def _evict(lib, kp=A, vp=A, s=A, tb=A, kl=A, dt=A, kept=A, so=None, nl=A, B=1, Hk=2, H=None, d=128, ps=16, n=4,
           W=2, Wd=1, L=32, pst=None, keep=16, first=2, recent=4, qst=None):
    return lib.fa_paged_evict(kp, vp, s, tb, kl, dt, kept, so, nl, B, Hk, d, ps, n, W, Wd, L,
                              pst or 16 * 2 * 128, keep, first, recent, None)


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(vp=None), INV), (dict(s=None), INV), (dict(dt=None), INV), (dict(kept=None), INV), (dict(nl=None), INV),
    (dict(keep=0), INV), (dict(first=-1), INV), (dict(recent=-1), INV), (dict(first=17), INV),
    (dict(first=13), INV), (dict(first=2**31 - 1, recent=2**31 - 1), INV), (dict(Wd=0), INV), (dict(L=0), INV),
    (dict(keep=17), INV),                                # more than the fresh pages hold
    (dict(vp=A + 8), MIS), (dict(s=A + 2), MIS), (dict(dt=A + 2), MIS), (dict(kept=A + 2), MIS),
    (dict(so=A + 2), MIS), (dict(nl=A + 2), MIS),
])
def test_evict_codes(lib, kw, code):
    assert _evict(lib, **kw) == code


def test_valid_calls_without_gpu_report_cuda_errors(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the gpu tests")
    for call in (_append, _attend, _scores, _evict):
        assert call(lib) in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)
    assert fa.fa_paged_workspace_bytes(128) == -1
    assert fa.fa_paged_workspace_bytes(96) == -1


def test_bad_index_status_has_a_name(lib):
    assert fa.status_string(fa.FA_ERR_BAD_INDEX) == "FA_ERR_BAD_INDEX"


def _cache(n=4, ps=16, hk=2, d=64, dt=torch.bfloat16):
    i32 = dict(dtype=torch.int32)
    return dict(k_pages=torch.zeros(n, ps, hk, d, dtype=dt), v_pages=torch.zeros(n, ps, hk, d, dtype=dt),
                block_table=torch.zeros(1, 2, **i32), kv_len=torch.ones(1, **i32), cu_q=torch.zeros(2, **i32))


@pytest.mark.parametrize("name,change,err", [
    ("k_pages", lambda x: x.float(), TypeError),
    ("k_pages", lambda x: x[:, :8], ValueError),                        # not the shape of v_pages
    ("k_pages", lambda x: x.transpose(1, 2).contiguous().transpose(1, 2), ValueError),
    ("k_pages", lambda x: x[0], ValueError),
    ("v_pages", lambda x: x.half(), ValueError),
    ("block_table", lambda x: x.long(), ValueError),
    ("block_table", lambda x: x.repeat(1, 2)[:, ::2], ValueError),      # gaps
    ("kv_len", lambda x: x.repeat(2), ValueError),
    ("cu_q", lambda x: x[:1], ValueError),
])
def test_wrappers_refuse_layouts(name, change, err):
    c = _cache()
    c[name] = change(c[name])
    with pytest.raises(err):
        fa.attention_paged(torch.zeros(3, 4, 64, dtype=torch.bfloat16), max_q=3, **c)


@pytest.mark.parametrize("q", [
    torch.zeros(3, 4, 64, dtype=torch.float16),                         # another type than the pages
    torch.zeros(3, 4, 128, dtype=torch.bfloat16),                       # another head dim
    torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2),        # rows that are not whole
    torch.zeros(3, 4, 128, dtype=torch.bfloat16)[:, :, :64],
])
def test_wrappers_refuse_queries(q):
    with pytest.raises(ValueError):
        fa.attention_paged(q, max_q=3, **_cache())
    lse = torch.zeros(q.shape[1], 3)
    c = _cache()
    c.pop("v_pages")
    with pytest.raises(ValueError):
        fa.paged_scores(q, lse, max_q=3, **c)


def test_wrappers_refuse_outputs():
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.attention_paged(q, max_q=3, out=torch.zeros(3, 4, 64), **_cache())
    with pytest.raises(ValueError):
        fa.attention_paged(q, max_q=3, lse=torch.zeros(3, 4), **_cache())
    c = _cache()
    c.pop("cu_q")
    c["scores"] = torch.zeros(1, 2, 32)
    dst = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.paged_evict(dst_table=dst, keep=8, kept=torch.zeros(1, 2, 9, dtype=torch.int32), **c)
    with pytest.raises(ValueError):
        fa.paged_evict(dst_table=dst, keep=8, scores_out=torch.zeros(1, 2, 9), **c)
    c["scores"] = torch.zeros(1, 3, 32)
    with pytest.raises(ValueError):
        fa.paged_evict(dst_table=dst, keep=8, **c)


@pytest.mark.parametrize("k,v", [
    (torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(3, 2, 64, dtype=torch.float16)),
    (torch.zeros(3, 1, 64, dtype=torch.bfloat16), torch.zeros(3, 1, 64, dtype=torch.bfloat16)),
    (torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)),
    (torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 4, 64, dtype=torch.bfloat16)[:, :2]),
])
def test_append_wrapper_refuses(k, v):
    with pytest.raises(ValueError):
        fa.paged_append(k, v, **_cache())


@pytest.mark.parametrize("kw", [
    dict(B=3, nl=A + 4), dict(B=3, kl=A + 8), dict(so=A), dict(so=A + 4 * 63), dict(s=A + 4 * 31, so=A),
])
def test_evict_refuses_overlapping_arrays(lib, kw):
    # [1][2][32] scores, [1][2][16] kept ones; lengths shifted against the old ones
    assert _evict(lib, **kw) == INV


@pytest.mark.parametrize("kw", [dict(B=3, nl=A + 12), dict(B=3, kl=A + 12), dict(so=A + 4 * 64), dict(s=A + 4 * 32, so=A),
                                dict(B=3)])
def test_evict_takes_neighbours_and_lengths_in_place(lib, kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the gpu tests")
    assert _evict(lib, **kw) in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED)


@pytest.mark.parametrize("kw", [dict(window=(2**32, 0)), dict(window=(-1, 2**32)), dict(first=2**32 + 4),
                                dict(max_q=2**32 + 1), dict(window=(-2**31 - 1, 0)), dict(window=(2**63, 0))])
def test_wrappers_refuse_numbers_beyond_32_bits(kw):
    # ctypes passes their lowest 32 bits: a window of 2**32 tokens would be one of none
    q, kw = torch.zeros(3, 4, 64, dtype=torch.bfloat16), {"max_q": 3, **kw}
    with pytest.raises(ValueError, match="32 bits"):
        fa.attention_paged(q, **_cache(), **kw)
    c = _cache()
    c.pop("v_pages")
    with pytest.raises(ValueError, match="32 bits"):
        fa.paged_scores(q, torch.zeros(4, 3), **c, **kw)


@pytest.mark.parametrize("kw", [dict(keep=2**32 + 8), dict(first=2**32), dict(recent=2**32)])
def test_evict_wrapper_refuses_numbers_beyond_32_bits(kw):
    c, kw = _cache(), {"keep": 8, **kw}
    c.pop("cu_q")
    with pytest.raises(ValueError, match="32 bits"):
        fa.paged_evict(scores=torch.zeros(1, 2, 32), dst_table=torch.zeros(1, 1, dtype=torch.int32), **c, **kw)


def test_a_stream_of_another_device_is_refused():
    # (the call would have gone to the current stream of the tensors' device)
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="cuda:1"):
        fa._launch_on(torch.device("cuda", 0), Stream())


def test_pages_of_one_head_in_either_order():
    # [n, 1, page_size, d] seen as [n, page_size, 1, d]: whole rows, whatever the
    # stride between heads that there is only one of
    c = _cache(hk=1)
    for name in ("k_pages", "v_pages"):
        c[name] = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16).transpose(1, 2)
        assert c[name].stride(2) != 64
    with pytest.raises(ValueError, match="must be on the GPU"):
        fa.attention_paged(torch.zeros(3, 4, 64, dtype=torch.bfloat16), max_q=3, **c)
