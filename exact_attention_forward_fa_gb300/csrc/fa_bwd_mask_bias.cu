// fa_bwd_mask_bias.cu -- the backward for a mask plan with a bias that depends on the
// distance: P = 2^(S c - beta |i - j| - LSE2); the bias has no gradient, so dS keeps its
// form.  Columns step by packed additions as in the forward.  Measured (GB300, fp16):
// 3 x 3001 tokens, 12 heads of 64 over 4, window 1000, both directions: 268 us (dK/dV 180,
// dQ 107, overlapping), bound by the elementwise warps (issue slots 40 to 43 %, tensor
// pipe 29 to 35 %).
#include "fa_bwd_launch.cuh"

namespace fa {

cudaError_t launch_bwd_mask_bias(const BwdLaunch &L) {
    if (L.d == 64)
        return L.bf16 ? launch_bwd_inst<64, false, true, false, false, true, true>(L)
                      : launch_bwd_inst<64, false, false, false, false, true, true>(L);
    return L.bf16 ? launch_bwd_inst<128, false, true, false, false, true, true>(L)
                  : launch_bwd_inst<128, false, false, false, false, true, true>(L);
}

}  // namespace fa
