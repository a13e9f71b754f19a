"""The refusals of shared memory that are made once the device is known: the backward's workspace in what the call reads
or writes, a mask plan over its documents, the rotated append's queries in the pages, one pool for K and V.  Nothing is
launched, nothing written; all tensors are parts of one buffer, so that every range is memory of the process."""
import pytest
import torch

import exact_attention_forward_fa_gb300 as fa

pytestmark = pytest.mark.gpu


def test_backward_refuses_its_workspace_in_a_tensor(gpu_lib):
    B, N, H, Hk, d = 1, 256, 2, 1, 64
    g = torch.Generator("cuda").manual_seed(2)
    plan = fa.mask_plan(torch.tensor([[0, 100, 256]], dtype=torch.int32, device="cuda"), N)
    sizes = {"q": 2 * N * H * d, "k": 2 * N * d, "v": 2 * N * d, "o": 2 * N * H * d, "dout": 2 * N * H * d, "lse": 4 * H * N,
             "plan": plan.data.numel(), "sinks": 16, "dq": 2 * N * H * d, "dk": 2 * N * d, "dv": 2 * N * d, "dsinks": 16}
    ws_bytes = 4 * fa.bwd_workspace_floats(B, H, N)
    at, end = {}, 0
    for name, n in sizes.items():
        at[name] = end
        end += (n + 15) // 16 * 16
    buf = torch.zeros(end + 2 * ws_bytes, dtype=torch.uint8, device="cuda")
    buf[at["q"]:at["lse"]].view(torch.float16).copy_(0.1 * torch.randn((at["lse"] - at["q"]) // 2, generator=g, device="cuda"))
    buf[at["plan"]:at["plan"] + sizes["plan"]] = plan.data
    p = {name: buf.data_ptr() + x for name, x in at.items()}

    def call(ws):
        return gpu_lib.fa_bwd_masked(p["q"], p["k"], p["v"], p["o"], p["dout"], p["lse"], ws, p["plan"], None, p["sinks"],
                                     p["dq"], p["dk"], p["dv"], p["dsinks"], B, H, Hk, N, d, H * d, d, d, 0.125, fa.FA_FP16,
                                     torch.cuda.current_stream().cuda_stream)

    before = buf.clone()
    for name in sizes:
        assert call(p[name]) == fa.FA_ERR_INVALID_ARG, name
        if p[name] - ws_bytes + 16 >= buf.data_ptr():
            assert call(p[name] - ws_bytes + 16) == fa.FA_ERR_INVALID_ARG, name
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    assert call(buf.data_ptr() + end) == fa.FA_OK
    assert fa.fa_check_status() == fa.FA_OK


def test_plan_refuses_its_documents(gpu_lib):
    N = 300
    n = fa.fa_mask_plan_bytes(1, N)
    buf = torch.zeros(4 * n, dtype=torch.uint8, device="cuda")
    p = buf.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    buf[2 * n // 16 * 16:][:16] = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda").view(torch.uint8)
    docs = p + 2 * n // 16 * 16
    far = p + 3 * n // 16 * 16
    for args in ((docs, None, docs, None), (docs, None, docs - n + 16, None), (docs, far, far - 16, None),
                 (docs, None, p, p + 16), (docs, None, p, docs - 4 * N + 4), (docs, far, p, far)):
        assert gpu_lib.fa_mask_plan(*args, 1, N, 3, -1, 0, stream) == fa.FA_ERR_INVALID_ARG, args
    assert gpu_lib.fa_mask_plan(docs, None, p, far, 1, N, 3, -1, 0, stream) == fa.FA_OK
    assert fa.fa_check_status() == fa.FA_OK


def test_rotated_append_refuses_queries_in_the_pages(gpu_lib):
    ps, n, Hk, H, d, T = 16, 4, 2, 4, 64, 8
    pool = torch.zeros(2 * n, ps, Hk, d, dtype=torch.float16, device="cuda")
    k_pages, v_pages = pool[:n], pool[n:]
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    kv_len = torch.tensor([T], dtype=torch.int32, device="cuda")
    cu_q = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    w, _ = fa.rope_frequencies(d)
    q, k = torch.ones(T, H, d, dtype=torch.float16, device="cuda"), torch.ones(T, Hk, d, dtype=torch.float16, device="cuda")
    # the right pool's rows, taken for queries; K's pool for V's
    for args in ((pool.view(-1, H, d)[:T], k, k, k_pages, v_pages), (pool.view(-1, H, d)[-T:], k, k, k_pages, v_pages),
                 (q, k, k, k_pages, k_pages), (q, k, k, pool[:n], pool[n - 1:2 * n - 1])):
        with pytest.raises(fa.FaError) as e:
            fa.paged_rope_append(*args, table, kv_len, cu_q, w)
        assert e.value.code == fa.FA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert not pool.any()
    fa.paged_rope_append(q, k, k, k_pages, v_pages, table, kv_len, cu_q, w)
    assert fa.fa_check_status() == fa.FA_OK and pool.any()


def test_a_refused_plan_stays_as_it_was(gpu_lib):
    """A window that is refused leaves the plan's mask and what it says of its window."""
    N = 300
    docs = torch.tensor([[0, 120, 290]], dtype=torch.int32, device="cuda")
    plan = fa.mask_plan(docs, N, window=(17, 3))
    before = plan.data.clone()
    for window in ((-2, 0), (5, -3)):
        with pytest.raises(fa.FaError) as e:
            fa.mask_plan(docs, N, window=window, out=plan)
        assert e.value.code == fa.FA_ERR_INVALID_ARG and plan.window == (17, 3)
    torch.cuda.synchronize()
    assert torch.equal(plan.data, before)
    assert fa.mask_plan(docs, N, window=(-1, 0), out=plan) is plan and plan.window == (-1, 0)
