"""Host-side checks (no GPU): masked attention and the rotated append refuse outputs that share memory with what they
read or with one another."""
import pytest
import torch

import exact_attention_forward_fa_gb300 as fa
from tests.test_masked_host import A, INV, LAUNCH, M, _bwd, _fwd, _rappend, lib  # noqa: F401

# sizes of these calls' tensors in bytes: q, o, dq and dout 2 x 300 x 4 x 64 x 2, k, v, dk, dv half of it,
# lse 2 x 4 x 300 x 4, the plan's in fa_mask_plan_bytes; pages 4 x 2048 x 2
WQ, WK, LSE, POOL = 2 * 300 * 4 * 64 * 2, 2 * 300 * 2 * 64 * 2, 2 * 4 * 300 * 4, 4 * 2048 * 2


@pytest.mark.parametrize("lse", [A, A + 4, A + WQ - 4, A + M + WK - 4, A + 2 * M + 16, A + 3 * M, A + 3 * M + WQ - 4,
                                 A + 3 * M - LSE + 4, A + M - LSE + 4])
def test_forward_refuses_lse_in_a_tensor(lib, lse):  # noqa: F811
    assert _fwd(lib, lse=lse, plan=A + 5 * M) == INV


@pytest.mark.parametrize("kw", [dict(o=A + 5 * M), dict(o=A + 5 * M - 16), dict(lse=A + 5 * M), dict(lse=A + 6 * M),
                                dict(lse=A + 7 * M, sinks=A + 7 * M + 4), dict(o=A + 6 * M - WQ + 16)])
def test_forward_refuses_outputs_in_what_it_reads(lib, kw):  # noqa: F811
    kw = dict(dict(plan=A + 5 * M, slopes=A + 6 * M), **kw)
    assert _fwd(lib, **kw) == INV


@pytest.mark.parametrize("ds", [A, A + 4 * M, A + 3 * M + 8, A + 8 * M, A + 5 * M, A + 6 * M, A + 7 * M + WK - 4, A + 9 * M,
                                A + 10 * M, A + 11 * M - 4])
def test_backward_refuses_dsinks_in_a_tensor(lib, ds):  # noqa: F811
    assert _bwd(lib, lse=A + 8 * M, ws=A + 12 * M, plan=A + 9 * M, slopes=A + 11 * M, sinks=A + 10 * M, ds=ds) == INV


@pytest.mark.parametrize("kw", [dict(dq=A + 8 * M), dict(dk=A + 8 * M), dict(dv=A + 9 * M), dict(dq=A + 10 * M - 16)])
def test_backward_refuses_gradients_in_lse_or_plan(lib, kw):  # noqa: F811
    kw = dict(dict(lse=A + 8 * M, ws=A + 12 * M, plan=A + 9 * M, slopes=A + 10 * M), **kw)
    assert _bwd(lib, **kw) == INV


@pytest.mark.parametrize("kw", [dict(qo=A + 4 * M), dict(qo=A + 5 * M + POOL - 16), dict(k=A + 4 * M), dict(k=A + 5 * M - 16),
                                dict(v=A + 4 * M + POOL - 16), dict(v=A + 5 * M)])
def test_rotated_append_refuses_rows_in_the_pages(lib, kw):  # noqa: F811
    assert _rappend(lib, **dict(dict(kp=A + 4 * M, vp=A + 5 * M), **kw)) == INV


def test_neighbours_are_taken(lib):  # noqa: F811
    """What lies next to a tensor does not share memory with it."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the gpu tests")
    n = (lib.fa_mask_plan_bytes(2, 300) + 15) // 16 * 16
    assert _fwd(lib, lse=A + WQ, plan=A + M - n) in LAUNCH
    assert _fwd(lib, lse=A + 3 * M - LSE, plan=A + 3 * M + WQ) in LAUNCH
    # (plan, slopes, sinks, lse, dsinks and the workspace, one behind the other)
    at = A + 8 * M
    assert _bwd(lib, plan=at, slopes=at + n, sinks=at + n + 16, lse=at + n + 32, ds=at + n + 32 + LSE,
                ws=at + n + 48 + LSE) in LAUNCH
    assert _rappend(lib, kp=A + 4 * M, vp=A + 4 * M + POOL, qo=A + 4 * M + 2 * POOL, k=A + 4 * M - 3 * 256) in LAUNCH
    # K and V side by side in the pages of one pool
    assert _rappend(lib, kp=A + 4 * M, vp=A + 4 * M + 4096, pst=2 * 2048) in LAUNCH
