"""GPU checks of attention on a mask plan with several units a block: the records of units handed on, the slots and
parities that the next unit finds, with and without a bias, at both head dims, forward and backward.

576 units of two query tiles, 576 key tiles and 1152 query tiles for at most 152 SMs: four to eight a block, of all
lengths, among them units that see nothing (whole tiles of padding).  Some heads are compared with float64
(tolerances in test_masked_gpu.py and test_masked_bwd_gpu.py); all heads with calls of so few heads that no block takes
a second unit, which have to give the same bits: a unit's arithmetic does not depend on what its block did before."""
import math

import pytest
import torch

import exact_attention_forward_fa_gb300 as fa
from tests._masked import check_backward, check_forward, reference, slopes_of
from tests.test_masked_bwd_gpu import gradient
from tests.test_masked_gpu import make, pack

pytestmark = pytest.mark.gpu

B, N, H, HK = 2, 3001, 24, 12
G = H // HK
DOCS = [pack(N, [1, 300, 127, 900, 64, 700], 600), [0, 5, 1200, 1300, 2100, 2300, 2300]]
PREFIX = [[1, 200, 0, 500, 64, 0], [0, 1195, 10, 0, 200, 0]]


@pytest.mark.parametrize("left,right,prefix", [(-1, 0, None), (-1, -1, None), (700, 0, PREFIX)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_units_of_a_block(gpu_lib, d, bias, left, right, prefix):
    dt = "bf16" if bias == (d == 64) else "fp16"
    q, k, v, plan, seen = make(B, N, H, HK, d, dt, DOCS, prefix, left, right, seed=d + bias)
    do = gradient(q, DOCS, dt)
    # every head holds the largest value and gradient, which give the scale of fp16's gradients
    v[:, 1000, :, 3] = do[:, 1001, :, 5] = 8.0
    slopes = slopes_of(H) if bias else None

    def step(heads, kv, plan=plan):
        x = [t[:, :, s].contiguous() for t, s in ((q, heads), (k, kv), (v, kv), (do, heads))]
        sl = None if slopes is None else slopes[heads].contiguous()
        o, lse = fa.attention_masked(*x[:3], plan, slopes=sl)
        return (o, lse) + fa.attention_backward_masked(*x[:3], o, lse, x[3], plan, slopes=sl)[:3]

    o, lse, dq, dk, dv = step(slice(0, H), slice(0, HK))
    assert fa.fa_check_status() == fa.FA_OK
    for a in (0, 7, HK - 1):
        hs, ks = slice(a * G, a * G + G), slice(a, a + 1)
        sl = None if slopes is None else slopes[hs]
        r = reference(q[:, :, hs], k[:, :, ks], v[:, :, ks], seen, sl, None, 1 / math.sqrt(d), do[:, :, hs])
        check_forward(o[:, :, hs], lse[:, hs], r, dt, d, 1 / math.sqrt(d), sl)
        check_backward((dq[:, :, hs], dk[:, :, ks], dv[:, :, ks]), r, dt, d, sl)
    for a in range(HK):
        hs, ks = slice(a * G, a * G + G), slice(a, a + 1)
        few = step(hs, ks)             # 48 units, 48 key tiles, 96 query tiles
        for x, y in zip(few, (o[:, :, hs], lse[:, hs], dq[:, :, hs], dk[:, :, ks], dv[:, :, ks])):
            assert torch.equal(x, y)
