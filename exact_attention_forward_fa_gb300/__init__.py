"""Python binding of libfa (exact attention forward on GB300, sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libfa.so``.  The names mirror the C ABI in ``include/fa.h``.
If the library has not been built, every entry point raises -- there is no
fallback implementation.

Tensors are [B, N, H, d] (batch, sequence, head, head dim) and contiguous;
LSE is float32 [B, H, N].
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_MISALIGNED = 3
FA_ERR_TOO_LARGE = 4
FA_ERR_CUDA = 5
FA_ERR_TIMEOUT = 6
FA_ERR_BAD_INDEX = 7

FA_BF16 = 0
FA_FP16 = 1

FA_SCALE_TILE = 0
FA_SCALE_HEAD = 1
FA_SCALE_TENSOR = 2

# Every symbol include/fa.h declares (checked by the tests).
EXPORTS = ("fa_fwd", "fa_fwd_gqa", "fa_fwd_gqa_packed", "fa_fwd_ext", "fa_fwd_splitkv", "fa_splitkv_workspace_floats",
           "fa_splitkv_auto", "fa_quantize_fp8", "fa_quantize_fp8_granular", "fa_fwd_fp8", "fa_fwd_fp8_gqa", "fa_bwd", "fa_bwd_ext", "fa_bwd_noalloc",
           "fa_paged_append", "fa_fwd_paged", "fa_paged_workspace_bytes", "fa_paged_scores", "fa_paged_evict",
           "fa_check_status", "fa_status_detail", "fa_selftest_wait_timeout",
           "fa_status_string", "fa_version")

_lib = None


class FaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


def load():
    """Load libfa.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
            "(the CUDA path has no fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_gqa.restype = i
    lib.fa_fwd_gqa_packed.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_gqa_packed.restype = i
    lib.fa_fwd_ext.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, f, vp, i, vp]
    lib.fa_fwd_ext.restype = i
    lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, i, vp, vp]
    lib.fa_fwd_splitkv.restype = i
    lib.fa_splitkv_workspace_floats.argtypes = [i, i, i, i, i]
    lib.fa_splitkv_workspace_floats.restype = ctypes.c_longlong
    lib.fa_splitkv_auto.argtypes = [i, i, i, i]
    lib.fa_splitkv_auto.restype = i
    lib.fa_quantize_fp8.argtypes = [vp, vp, vp, vp, i, i, i, i, vp]
    lib.fa_quantize_fp8.restype = i
    lib.fa_quantize_fp8_granular.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.fa_quantize_fp8_granular.restype = i
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_fwd_fp8_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_fp8_gqa.restype = i
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_ext.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i,
                               f, vp, vp, i, vp]
    lib.fa_bwd_ext.restype = i
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    lib.fa_bwd_noalloc.restype = i
    ll = ctypes.c_longlong
    lib.fa_paged_append.argtypes = [vp] * 7 + [i] * 7 + [ll, ll, vp]
    lib.fa_paged_append.restype = i
    lib.fa_fwd_paged.argtypes = [vp] * 9 + [i] * 9 + [ll, ll, f, i, i, i, i, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_paged_workspace_bytes.argtypes = [i]
    lib.fa_paged_workspace_bytes.restype = ll
    lib.fa_paged_scores.argtypes = [vp] * 8 + [i] * 10 + [ll, ll, f, i, i, i, i, vp]
    lib.fa_paged_scores.restype = i
    lib.fa_paged_evict.argtypes = [vp] * 9 + [i] * 8 + [ll, i, i, i, vp]
    lib.fa_paged_evict.restype = i
    lib.fa_selftest_wait_timeout.argtypes = [vp, vp]
    lib.fa_selftest_wait_timeout.restype = i
    lib.fa_check_status.argtypes = [vp]
    lib.fa_check_status.restype = i
    lib.fa_status_detail.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.fa_status_detail.restype = None
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_version.argtypes = []
    lib.fa_version.restype = i
    _lib = lib
    return lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def status_string(code: int) -> str:
    return load().fa_status_string(int(code)).decode()


def fa_fwd(q, k, v, o, lse, B: int, H: int, N: int, d: int, alpha: float,
           causal: int, dtype: int, stream=None) -> int:
    """Direct call of the C entry point; returns the fa_status code.

    Pointer arguments may be torch tensors or integer device addresses;
    ``lse`` may be None.  ``stream`` is a torch stream, a raw cudaStream_t
    integer, or None for torch's current stream."""
    return load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                         int(B), int(H), int(N), int(d), float(alpha),
                         int(causal), int(dtype), _stream(stream))


def fa_fwd_gqa(q, k, v, o, lse, B: int, H: int, H_kv: int, N: int, d: int, alpha: float,
               causal: int, dtype: int, stream=None) -> int:
    """Direct call of the C entry point: K/V with H_kv heads shared by groups
    of H / H_kv query heads (see include/fa.h)."""
    return load().fa_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(H),
                             int(H_kv), int(N), int(d), float(alpha), int(causal), int(dtype),
                             _stream(stream))


def fa_fwd_gqa_packed(q, k, v, o, lse, B: int, H: int, H_kv: int, N: int, d: int,
                      alpha: float, causal: int, dtype: int, stream=None) -> int:
    """Direct call of the C entry point: fa_fwd_gqa with the query heads of
    each K/V head packed into the rows of one Q tile (see include/fa.h)."""
    return load().fa_fwd_gqa_packed(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B),
                                    int(H), int(H_kv), int(N), int(d), float(alpha),
                                    int(causal), int(dtype), _stream(stream))


def fa_fwd_ext(q, k, v, o, lse, B: int, H: int, H_kv: int, N: int, d: int, alpha: float,
               window_left: int, window_right: int, softcap: float, sinks, dtype: int,
               stream=None) -> int:
    """Direct call of the C entry point: local window, softcap and per-head
    sinks (see include/fa.h); ``sinks`` may be None."""
    return load().fa_fwd_ext(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(H),
                             int(H_kv), int(N), int(d), float(alpha), int(window_left),
                             int(window_right), float(softcap), _ptr(sinks), int(dtype),
                             _stream(stream))


def attention_ext(q, k, v, window=(-1, -1), softcap: float = 0.0, sinks=None,
                  alpha: float | None = None, out=None, lse=None, want_lse: bool = True,
                  stream=None):
    """Forward with the score and mask variants for torch tensors on the GPU:
    window = (left, right) key bounds around the diagonal (-1: none),
    softcap c (0: none), sinks float32 [H] on the GPU or None.  K/V may have
    fewer heads than Q (grouped).  Returns (O, LSE or None)."""
    import torch
    if q.dtype == torch.bfloat16:
        dt = FA_BF16
    elif q.dtype == torch.float16:
        dt = FA_FP16
    else:
        raise TypeError(f"unsupported dtype {q.dtype}")
    B, N, H, d = q.shape
    if alpha is None:
        alpha = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    rc = fa_fwd_ext(q, k, v, out, lse, B, H, k.shape[2], N, d, alpha, int(window[0]),
                    int(window[1]), float(softcap), sinks, dt, stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_ext")
    return out, lse


def fa_fwd_splitkv(q, k, v, o, lse, B: int, H: int, N: int, d: int, alpha: float, causal: int,
                   dtype: int, n_splits: int, workspace, stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h)."""
    return load().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(H),
                                 int(N), int(d), float(alpha), int(causal), int(dtype),
                                 int(n_splits), _ptr(workspace), _stream(stream))


def fa_splitkv_workspace_floats(B: int, H: int, N: int, d: int, n_splits: int) -> int:
    return load().fa_splitkv_workspace_floats(int(B), int(H), int(N), int(d), int(n_splits))


def fa_splitkv_auto(B: int, H: int, N: int, d: int) -> int:
    return load().fa_splitkv_auto(int(B), int(H), int(N), int(d))


def attention_splitkv(q, k, v, causal: bool = False, alpha: float | None = None,
                      n_splits: int = 0, want_lse: bool = True, stream=None):
    """Split-KV forward for torch tensors on the GPU (n_splits 0: the
    library's choice for this device).  Returns (O, LSE or None)."""
    import torch
    dt = FA_BF16 if q.dtype == torch.bfloat16 else FA_FP16
    B, N, H, d = q.shape
    if alpha is None:
        alpha = 1.0 / math.sqrt(d)
    if n_splits <= 0:
        n_splits = fa_splitkv_auto(B, H, N, d)
    out = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if want_lse else None
    ws = torch.empty((fa_splitkv_workspace_floats(B, H, N, d, n_splits),), dtype=torch.float32,
                     device=q.device)
    rc = fa_fwd_splitkv(q, k, v, out, lse, B, H, N, d, alpha, int(bool(causal)), dt, n_splits,
                        ws, stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_splitkv")
    return out, lse


def fa_quantize_fp8(x, x8, scales, hadamard_signs, B: int, H: int, N: int,
                    d: int, stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h)."""
    return load().fa_quantize_fp8(_ptr(x), _ptr(x8), _ptr(scales), _ptr(hadamard_signs),
                                  int(B), int(H), int(N), int(d), _stream(stream))


def fa_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, B: int, H: int,
               N: int, d: int, alpha: float, causal: int, stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h)."""
    return load().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(q_scale), _ptr(k_scale),
                             _ptr(v_scale), _ptr(o), _ptr(lse), int(B), int(H), int(N),
                             int(d), float(alpha), int(causal), _stream(stream))


def fa_quantize_fp8_granular(x, x8, scales, hadamard_signs, B: int, H: int, N: int,
                             d: int, granularity: int, stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h)."""
    return load().fa_quantize_fp8_granular(_ptr(x), _ptr(x8), _ptr(scales),
                                           _ptr(hadamard_signs), int(B), int(H), int(N),
                                           int(d), int(granularity), _stream(stream))


def quantize_fp8(x, hadamard_signs=None, stream=None, granularity: int = FA_SCALE_TILE):
    """bf16 [B,N,H,d] on the GPU -> (uint8 e4m3 codes, float scales [B,H,ceil(N/128)]);
    ``granularity`` FA_SCALE_HEAD / FA_SCALE_TENSOR give one scale per head /
    per tensor, repeated over the tiles."""
    import torch
    B, N, H, d = x.shape
    x8 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    sc = torch.empty((B, H, (N + 127) // 128), dtype=torch.float32, device=x.device)
    if granularity == FA_SCALE_TILE:
        rc = fa_quantize_fp8(x, x8, sc, hadamard_signs, B, H, N, d, stream)
    else:
        rc = fa_quantize_fp8_granular(x, x8, sc, hadamard_signs, B, H, N, d, granularity,
                                      stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_quantize_fp8")
    return x8, sc


def fa_fwd_fp8_gqa(q8, k8, v8, q_scale, k_scale, v_scale, o, lse, B: int, H: int, H_kv: int,
                   N: int, d: int, alpha: float, causal: int, stream=None) -> int:
    """Direct call of the C entry point: fa_fwd_fp8 with K/V (codes and
    scales) over H_kv heads (see include/fa.h)."""
    return load().fa_fwd_fp8_gqa(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(q_scale), _ptr(k_scale),
                                 _ptr(v_scale), _ptr(o), _ptr(lse), int(B), int(H), int(H_kv),
                                 int(N), int(d), float(alpha), int(causal), _stream(stream))


def attention_fp8(q8, k8, v8, q_scale, k_scale, v_scale, causal: bool = False,
                  alpha: float | None = None, out=None, lse=None, want_lse: bool = True,
                  stream=None):
    """FP8 forward on quantized inputs; returns (O bf16, LSE or None).  K/V
    may have fewer heads than Q (fa_fwd_fp8_gqa)."""
    import torch
    B, N, H, d = q8.shape
    H_kv = k8.shape[2]
    if alpha is None:
        alpha = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty(q8.shape, dtype=torch.bfloat16, device=q8.device)
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    if H_kv == H:
        rc = fa_fwd_fp8(q8, k8, v8, q_scale, k_scale, v_scale, out, lse, B, H, N, d, alpha,
                        int(bool(causal)), stream)
    else:
        rc = fa_fwd_fp8_gqa(q8, k8, v8, q_scale, k_scale, v_scale, out, lse, B, H, H_kv, N, d,
                            alpha, int(bool(causal)), stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_fp8")
    return out, lse


def bwd_workspace_floats(B: int, H: int, N: int) -> int:
    """Size of fa_bwd's workspace: float [2][B][H][ceil(N/128)*128]."""
    return 2 * B * H * ((N + 127) // 128) * 128


def fa_bwd(q, k, v, o, dout, lse, workspace, dq, dk, dv, B: int, H: int, N: int, d: int,
           alpha: float, causal: int, dtype: int, stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h)."""
    return load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                         _ptr(workspace), _ptr(dq), _ptr(dk), _ptr(dv), int(B), int(H), int(N),
                         int(d), float(alpha), int(causal), int(dtype), _stream(stream))


def fa_bwd_ext(q, k, v, o, dout, lse, workspace, dq, dk, dv, B: int, H: int, H_kv: int, N: int,
               d: int, alpha: float, window_left: int, window_right: int, softcap: float, sinks,
               dsinks, dtype: int, stream=None) -> int:
    """Direct call of the C entry point: the backward of fa_fwd_ext with a
    local window and softcap; sinks/dsinks may be None (see include/fa.h)."""
    return load().fa_bwd_ext(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                             _ptr(workspace), _ptr(dq), _ptr(dk), _ptr(dv), int(B), int(H),
                             int(H_kv), int(N), int(d), float(alpha), int(window_left),
                             int(window_right), float(softcap), _ptr(sinks), _ptr(dsinks), int(dtype),
                             _stream(stream))


def attention_backward_ext(q, k, v, o, lse, dout, window=(-1, -1), softcap: float = 0.0,
                           sinks=None, alpha: float | None = None, stream=None):
    """Gradients (dQ, dK, dV, dsinks or None) for the forward of
    ``attention_ext`` with a window, softcap and optional sinks."""
    import torch
    if q.dtype == torch.bfloat16:
        dt = FA_BF16
    elif q.dtype == torch.float16:
        dt = FA_FP16
    else:
        raise TypeError(f"unsupported dtype {q.dtype}")
    B, N, H, d = q.shape
    if alpha is None:
        alpha = 1.0 / math.sqrt(d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty((bwd_workspace_floats(B, H, N),), dtype=torch.float32, device=q.device)
    ds = None if sinks is None else torch.empty((H,), dtype=torch.float32, device=q.device)
    rc = fa_bwd_ext(q, k, v, o, dout, lse, ws, dq, dk, dv, B, H, k.shape[2], N, d, alpha,
                    int(window[0]),
                    int(window[1]), float(softcap), sinks, ds, dt, stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd_ext")
    return dq, dk, dv, ds


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, B: int, H: int, N: int, d: int,
                   alpha: float, causal: int, dtype: int, stream=None) -> int:
    """Direct call of the C entry point: fa_bwd with the library's own
    16 MiB device workspace, for callers that must not allocate (see
    include/fa.h; overlapping calls race on that workspace)."""
    return load().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), int(B), int(H), int(N), int(d),
                                 float(alpha), int(causal), int(dtype), _stream(stream))


def attention_backward(q, k, v, o, lse, dout, causal: bool = False,
                       alpha: float | None = None, stream=None):
    """Gradients (dQ, dK, dV) for torch tensors on the GPU; ``o`` and ``lse``
    come from ``attention`` on the same inputs.  Allocates the outputs and
    the workspace with torch; raises FaError on a non-OK status."""
    import torch
    if q.dtype == torch.bfloat16:
        dt = FA_BF16
    elif q.dtype == torch.float16:
        dt = FA_FP16
    else:
        raise TypeError(f"unsupported dtype {q.dtype}")
    B, N, H, d = q.shape
    if alpha is None:
        alpha = 1.0 / math.sqrt(d)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty((bwd_workspace_floats(B, H, N),), dtype=torch.float32, device=q.device)
    rc = fa_bwd(q, k, v, o, dout, lse, ws, dq, dk, dv, B, H, N, d, alpha,
                int(bool(causal)), dt, stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_bwd")
    return dq, dk, dv


# ---- paged key/value cache (see include/fa.h) ----

def fa_paged_append(k, v, k_pages, v_pages, block_table, kv_len, cu_q, B: int, H_kv: int, d: int,
                    total_q: int, page_size: int, n_pages: int, table_width: int, kv_stride: int,
                    page_stride: int, stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h)."""
    return load().fa_paged_append(_ptr(k), _ptr(v), _ptr(k_pages), _ptr(v_pages),
                                  _ptr(block_table), _ptr(kv_len), _ptr(cu_q), B, H_kv, d, total_q,
                                  page_size, n_pages, table_width, kv_stride, page_stride,
                                  _stream(stream))


def fa_fwd_paged(q, k_pages, v_pages, block_table, kv_len, cu_q, o, lse, workspace, B: int, H: int,
                 H_kv: int, total_q: int, max_q: int, d: int, page_size: int, n_pages: int,
                 table_width: int, q_stride: int, page_stride: int, alpha: float, window_left: int,
                 window_right: int, first: int, dtype: int, stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h); ``lse`` may be None."""
    return load().fa_fwd_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table),
                               _ptr(kv_len), _ptr(cu_q), _ptr(o), _ptr(lse), _ptr(workspace), B, H,
                               H_kv, total_q, max_q, d, page_size, n_pages, table_width, q_stride,
                               page_stride, alpha, window_left, window_right, first, dtype,
                               _stream(stream))


def fa_paged_workspace_bytes(d: int) -> int:
    return load().fa_paged_workspace_bytes(int(d))


def fa_paged_scores(q, lse, k_pages, block_table, kv_len, cu_q, scores_in, scores, B: int, H: int,
                    H_kv: int, total_q: int, max_q: int, d: int, page_size: int, n_pages: int,
                    table_width: int, score_width: int, q_stride: int, page_stride: int,
                    alpha: float, window_left: int, window_right: int, first: int, dtype: int,
                    stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h); ``scores_in`` may
    be None."""
    return load().fa_paged_scores(_ptr(q), _ptr(lse), _ptr(k_pages), _ptr(block_table),
                                  _ptr(kv_len), _ptr(cu_q), _ptr(scores_in), _ptr(scores), B, H,
                                  H_kv, total_q, max_q, d, page_size, n_pages, table_width,
                                  score_width, q_stride, page_stride, alpha, window_left,
                                  window_right, first, dtype, _stream(stream))


def fa_paged_evict(k_pages, v_pages, scores, block_table, kv_len, dst_table, kept, scores_out,
                   new_len, B: int, H_kv: int, d: int, page_size: int, n_pages: int,
                   table_width: int, dst_width: int, score_width: int, page_stride: int, keep: int,
                   first: int, recent: int, stream=None) -> int:
    """Direct call of the C entry point (see include/fa.h); ``scores_out`` may
    be None."""
    return load().fa_paged_evict(_ptr(k_pages), _ptr(v_pages), _ptr(scores), _ptr(block_table),
                                 _ptr(kv_len), _ptr(dst_table), _ptr(kept), _ptr(scores_out),
                                 _ptr(new_len), B, H_kv, d, page_size, n_pages, table_width,
                                 dst_width, score_width, page_stride, keep, first, recent,
                                 _stream(stream))


# Single tokens make host time count: the checks below compare device indices
# (-1: not on a GPU) instead of devices, and the module is looked up once.
_torch = None


def _use_torch():
    global _torch
    import torch
    _torch = torch
    return torch


def _check_paged(at: int, dtype, k, v, block_table, kv_len, last, last_shape) -> None:
    """The layout that the C entry points are told by sizes and strides: pools
    [n_pages, page_size, H_kv, d] of ``dtype`` with whole rows (v may be
    None), int32 index tensors [B, W], [B] and ``last_shape`` without gaps,
    everything on GPU ``at``."""
    torch = _torch or _use_torch()
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("pages are [n_pages, page_size, H_kv, d]")
    kt = k.dtype
    if kt is not torch.bfloat16 and kt is not torch.float16:
        raise TypeError(f"unsupported dtype {kt}")
    if kt is not dtype:
        raise ValueError("the pages and the new tokens differ in type")
    n, ps, hk, d = shape
    st = k.stride()
    if st[3] != 1 or (st[2] != d and hk > 1) or st[1] != hk * d:
        raise ValueError("a page's rows [page_size, H_kv, d] must be contiguous")
    if k.get_device() != at:
        raise ValueError("tensors on different devices")
    if v is not None and (v.dtype is not dtype or v.shape != shape or v.stride() != st or v.get_device() != at):
        raise ValueError("k_pages and v_pages differ in type, shape, strides or device")
    table_shape = block_table.shape
    _check_int(block_table, table_shape, at)
    _check_int(kv_len, table_shape[:1], at)
    _check_int(last, last_shape, at)
    if at < 0:
        raise ValueError("tensors must be on the GPU")


def _check_int(x, shape, at: int) -> None:
    if x.dtype is not _torch.int32 or x.shape != shape or not x.is_contiguous():
        raise ValueError(f"index tensors are contiguous int32; expected {tuple(shape)}, got "
                         f"{x.dtype} {tuple(x.shape)}")
    if x.get_device() != at:
        raise ValueError("tensors on different devices")


# ctypes would keep the lowest 32 bits of a number that a C int does not hold.
_BEYOND_32 = "windows and counts have to fit 32 bits"


def _check_float(x, shape, at: int) -> None:
    if x.dtype is not _torch.float32 or x.shape != shape or not x.is_contiguous() or x.get_device() != at:
        raise ValueError(f"expected a contiguous float32 {tuple(shape)} on GPU {at}, got {x.dtype} "
                         f"{tuple(x.shape)} on {x.device}")


def _packed_stride(x, name: str) -> int:
    """The elements between the tokens of a packed [T, heads, d] tensor, whose
    rows are whole (a slice of wider rows is fine)."""
    T, heads, d = x.shape
    s = x.stride()
    if T and (s[2] != 1 or (s[1] != d and heads > 1)):    # (strides of an empty tensor say nothing)
        raise ValueError(f"{name} is [T, heads, d] with contiguous [heads, d] rows")
    return s[0] if T > 1 else heads * d


class _launch_on:
    """Makes the tensors' device current and ``stream`` (a raw cudaStream_t, a
    torch stream, or None: the device's current one) the stream that torch
    allocates for and launches on: what a call allocates is then reused only
    behind its kernels."""

    def __init__(self, device, stream):
        import torch
        self.device = device
        if isinstance(stream, int):
            stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                      else torch.cuda.default_stream(device))
        elif stream is not None and stream.device != device:
            raise ValueError(f"a stream of {stream.device} for tensors on {device}")
        self.ctx = torch.cuda.stream(stream) if stream is not None else None
        self.guard = (torch.cuda.device(device)
                      if device.index != torch.cuda.current_device() else None)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        if self.guard is not None:
            self.guard.__exit__(*exc)


# The workspace of attention_paged's calls on a device's legacy default stream,
# by (device index, d): that stream is never destroyed nor captured, so its
# calls run one after the other.  The lock keeps the launches of one call
# together when several host threads call.
_paged_ws: dict = {}
_paged_ws_lock = threading.Lock()


def _new_paged_workspace(d: int, device):
    """A new workspace on ``device``, which is current."""
    import torch
    n = fa_paged_workspace_bytes(d)
    if n < 0:
        raise FaError(FA_ERR_UNSUPPORTED, "fa_paged_workspace_bytes")
    return torch.empty((n,), dtype=torch.uint8, device=device)


def paged_workspace(d: int, device="cuda"):
    """A workspace for ``attention_paged`` at head dim d (uint8 tensor); calls
    that may overlap in time need one each."""
    import torch
    with torch.cuda.device(device):
        return _new_paged_workspace(d, torch.device("cuda", torch.cuda.current_device()))


def paged_append(k, v, k_pages, v_pages, block_table, kv_len, cu_q, stream=None) -> None:
    """Writes the new tokens' K and V (packed [T, H_kv, d], rows of a wider
    tensor allowed) into their pages [n_pages, page_size, H_kv, d]; kv_len
    counts them already."""
    torch = _torch or _use_torch()
    at = k.get_device()
    if stream is not None or (at >= 0 and at != torch._C._cuda_getDevice()):
        with _launch_on(k.device, stream):
            return paged_append(k, v, k_pages, v_pages, block_table, kv_len, cu_q)
    B, W = block_table.shape
    T, hk, d = k.shape
    _check_paged(at, k.dtype, k_pages, v_pages, block_table, kv_len, cu_q, (B + 1,))
    n, ps, hp, dp = k_pages.shape
    ks = _packed_stride(k, "k")
    if k.shape != v.shape or k.dtype != v.dtype or v.get_device() != at or _packed_stride(v, "v") != ks:
        raise ValueError("k and v differ in type, shape, strides or device")
    if hk != hp or d != dp:
        raise ValueError("k, v and the pages differ in heads or head dim")
    rc = load().fa_paged_append(
        k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
        kv_len.data_ptr(), cu_q.data_ptr(), B, hk, d, T, ps, n, W, ks, k_pages.stride(0),
        torch._C._cuda_getCurrentRawStream(at))
    if rc != FA_OK:
        raise FaError(rc, "fa_paged_append")


def attention_paged(q, k_pages, v_pages, block_table, kv_len, cu_q, max_q: int, window=(-1, 0),
                    first: int = 0, alpha: float | None = None, out=None, lse=None,
                    want_lse: bool = True, workspace=None, stream=None):
    """Attention of the new tokens (packed q [T, H, d], sequence b's in rows
    cu_q[b] .. cu_q[b + 1]) over the cache that holds them: causal by default,
    window = (left, right) key bounds around a token's position (-1: none),
    the first ``first`` tokens visible beside a left bound.  ``max_q``: the
    most new tokens of one sequence.  Returns (O [T, H, d], LSE [H, T] or
    None); rows behind cu_q[B] (a padded batch) are left as they were,
    uninitialised where O and LSE are allocated here."""
    torch = _torch or _use_torch()
    at, dtype = q.get_device(), q.dtype
    if stream is not None or (at >= 0 and at != torch._C._cuda_getDevice()):
        with _launch_on(q.device, stream):
            return attention_paged(q, k_pages, v_pages, block_table, kv_len, cu_q, max_q, window, first,
                                   alpha, out, lse, want_lse, workspace)
    T, H, d = q.shape
    B, W = block_table.shape
    left, right = window
    if not (-0x80000000 <= max_q <= 0x7fffffff and -0x80000000 <= left <= 0x7fffffff
            and -0x80000000 <= right <= 0x7fffffff and -0x80000000 <= first <= 0x7fffffff):
        raise ValueError(_BEYOND_32)
    _check_paged(at, dtype, k_pages, v_pages, block_table, kv_len, cu_q, (B + 1,))
    n, ps, hk, dk = k_pages.shape
    qs = _packed_stride(q, "q")
    if dk != d:
        raise ValueError("q and the pages differ in head dim")
    if alpha is None:
        alpha = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty((T, H, d), dtype=dtype, device=q.device)
    elif (out.shape != q.shape or out.dtype is not dtype or out.get_device() != at
            or not out.is_contiguous()):
        raise ValueError(f"out is a contiguous {dtype} {tuple(q.shape)} on {q.device}")
    if lse is not None:
        _check_float(lse, (H, T), at)
    elif want_lse:
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    raw = torch._C._cuda_getCurrentRawStream(at)
    shared = workspace is None and raw == 0
    if shared:
        workspace = _paged_ws.get((at, d))
        if workspace is None:
            workspace = _paged_ws.setdefault((at, d), _new_paged_workspace(d, q.device))
        _paged_ws_lock.acquire()
    elif workspace is None:
        workspace = _new_paged_workspace(d, q.device)
    elif (workspace.get_device() != at
            or workspace.numel() * workspace.element_size() < fa_paged_workspace_bytes(d)):
        raise ValueError(f"the workspace is {fa_paged_workspace_bytes(d)} bytes on {q.device}")
    try:
        rc = load().fa_fwd_paged(
            q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
            kv_len.data_ptr(), cu_q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
            workspace.data_ptr(), B, H, hk, T, max_q, d, ps, n, W, qs, k_pages.stride(0), alpha,
            left, right, first, FA_BF16 if dtype is torch.bfloat16 else FA_FP16, raw)
    finally:
        if shared:
            _paged_ws_lock.release()
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd_paged")
    return out, lse


def paged_scores(q, lse, k_pages, block_table, kv_len, cu_q, max_q: int, scores=None,
                 window=(-1, 0), first: int = 0, alpha: float | None = None, out=None, stream=None):
    """The attention weight that every cached token gets from the new ones,
    per K/V head, added to ``scores`` (float32 [B, H_kv, L], None: zeros); q,
    lse, window, first and alpha as in ``attention_paged``.  ``out`` may be
    ``scores``; entries behind kv_len are left as they were (zeros where it
    is allocated here).  Returns out."""
    torch = _torch or _use_torch()
    at, dtype = q.get_device(), q.dtype
    if stream is not None or (at >= 0 and at != torch._C._cuda_getDevice()):
        with _launch_on(q.device, stream):
            return paged_scores(q, lse, k_pages, block_table, kv_len, cu_q, max_q, scores, window, first,
                                alpha, out)
    T, H, d = q.shape
    B, W = block_table.shape
    left, right = window
    if not (-0x80000000 <= max_q <= 0x7fffffff and -0x80000000 <= left <= 0x7fffffff
            and -0x80000000 <= right <= 0x7fffffff and -0x80000000 <= first <= 0x7fffffff):
        raise ValueError(_BEYOND_32)
    _check_paged(at, dtype, k_pages, None, block_table, kv_len, cu_q, (B + 1,))
    n, ps, hk, dk = k_pages.shape
    qs = _packed_stride(q, "q")
    if dk != d:
        raise ValueError("q and the pages differ in head dim")
    like = scores if scores is not None else out
    shape = (B, hk, W * ps if like is None else like.shape[2])
    _check_float(lse, (H, T), at)
    if scores is not None:
        _check_float(scores, shape, at)
    if out is None:
        out = torch.zeros(shape, dtype=torch.float32, device=q.device)
    else:
        _check_float(out, shape, at)
    if alpha is None:
        alpha = 1.0 / math.sqrt(d)
    rc = load().fa_paged_scores(
        q.data_ptr(), lse.data_ptr(), k_pages.data_ptr(), block_table.data_ptr(), kv_len.data_ptr(),
        cu_q.data_ptr(), None if scores is None else scores.data_ptr(), out.data_ptr(), B, H, hk, T,
        max_q, d, ps, n, W, shape[2], qs, k_pages.stride(0), alpha, left, right, first,
        FA_BF16 if dtype is torch.bfloat16 else FA_FP16, torch._C._cuda_getCurrentRawStream(at))
    if rc != FA_OK:
        raise FaError(rc, "fa_paged_scores")
    return out


def paged_evict(k_pages, v_pages, scores, block_table, kv_len, dst_table, keep: int, first: int = 0,
                recent: int = 0, kept=None, scores_out=None, new_len=None, stream=None):
    """Cuts every sequence to its ``keep`` most important tokens per K/V head
    (the first ``first``, the last ``recent``, the others by ``scores``) and
    writes them, in their order, into the pages of ``dst_table``.  Returns
    (kept positions [B, H_kv, keep], their scores, new lengths); entries
    behind a new length are left as they were (-1 and 0 where they are
    allocated here).  ``new_len`` may be ``kv_len`` itself; ``scores_out`` is
    no part of ``scores``."""
    torch = _torch or _use_torch()
    at = scores.get_device()
    if stream is not None or (at >= 0 and at != torch._C._cuda_getDevice()):
        with _launch_on(scores.device, stream):
            return paged_evict(k_pages, v_pages, scores, block_table, kv_len, dst_table, keep, first,
                               recent, kept, scores_out, new_len)
    B, W = block_table.shape
    Wd = dst_table.shape[1]
    if not (-0x80000000 <= keep <= 0x7fffffff and -0x80000000 <= first <= 0x7fffffff
            and -0x80000000 <= recent <= 0x7fffffff):
        raise ValueError(_BEYOND_32)
    _check_paged(at, k_pages.dtype, k_pages, v_pages, block_table, kv_len, dst_table, (B, Wd))
    n, ps, hk, d = k_pages.shape
    L = scores.shape[2]
    _check_float(scores, (B, hk, L), at)
    room = (B, hk, max(keep, 0))
    if kept is None:
        kept = torch.full(room, -1, dtype=torch.int32, device=scores.device)
    else:
        _check_int(kept, room, at)
    if scores_out is None:
        scores_out = torch.zeros(room, dtype=torch.float32, device=scores.device)
    else:
        _check_float(scores_out, room, at)
    if new_len is None:
        new_len = torch.empty((B,), dtype=torch.int32, device=scores.device)
    else:
        _check_int(new_len, (B,), at)
    rc = load().fa_paged_evict(
        k_pages.data_ptr(), v_pages.data_ptr(), scores.data_ptr(), block_table.data_ptr(),
        kv_len.data_ptr(), dst_table.data_ptr(), kept.data_ptr(), scores_out.data_ptr(),
        new_len.data_ptr(), B, hk, d, ps, n, W, Wd, L, k_pages.stride(0), keep, first, recent,
        torch._C._cuda_getCurrentRawStream(at))
    if rc != FA_OK:
        raise FaError(rc, "fa_paged_evict")
    return kept, scores_out, new_len


def fa_selftest_wait_timeout(result, stream=None) -> int:
    """Direct call of the C entry point: a kernel whose bounded waits run
    out (no fault); result is a device uint32 tensor of 2 elements."""
    return load().fa_selftest_wait_timeout(_ptr(result), _stream(stream))


def fa_check_status(stream=None) -> int:
    return load().fa_check_status(_stream(stream))


def fa_status_detail() -> list[int]:
    out = (ctypes.c_uint32 * 4)()
    load().fa_status_detail(out)
    return list(out)


def fa_version() -> int:
    return load().fa_version()


def attention(q, k, v, causal: bool = False, alpha: float | None = None,
              out=None, lse=None, want_lse: bool = True, stream=None,
              pack_gqa: bool = False):
    """Convenience wrapper over ``fa_fwd`` for torch tensors on the GPU
    (``fa_fwd_gqa`` when K/V have fewer heads than Q; ``fa_fwd_gqa_packed``
    with ``pack_gqa``).

    Allocates O (and LSE) with torch when not given, launches, and raises
    FaError on a non-OK status.  Returns (O, LSE or None)."""
    import torch
    if q.dtype == torch.bfloat16:
        dt = FA_BF16
    elif q.dtype == torch.float16:
        dt = FA_FP16
    else:
        raise TypeError(f"unsupported dtype {q.dtype}")
    B, N, H, d = q.shape
    if alpha is None:
        alpha = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    H_kv = k.shape[2]
    if H_kv == H:
        rc = fa_fwd(q, k, v, out, lse, B, H, N, d, alpha, int(bool(causal)), dt, stream)
    else:
        call = fa_fwd_gqa_packed if pack_gqa else fa_fwd_gqa
        rc = call(q, k, v, out, lse, B, H, H_kv, N, d, alpha, int(bool(causal)), dt, stream)
    if rc != FA_OK:
        raise FaError(rc, "fa_fwd")
    return out, lse
