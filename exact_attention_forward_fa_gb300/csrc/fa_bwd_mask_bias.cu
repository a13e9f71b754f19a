// fa_bwd_mask_bias.cu -- the backward for a mask plan with a bias that depends on the
// distance: P = 2^(S c - beta |i - j| - LSE2); the bias has no gradient, so dS keeps its
// form.  Columns step by packed additions, the dQ kernel's by the bias itself, from an FMA with
// -LSE2 on, the dK/dV kernel's by the distance, whose FMA with each column's -LSE2 rounds
// once.  Measured (GB300, fp16): 3 x 3001 tokens, 12 heads of 64 over 4, window 1000, both
// directions: 276 us (statistics 13, scale 6, dK/dV 181, dQ 106, overlapping), bound by the
// elementwise warps' step (dK/dV: about 4000 cycles a tile, 1090 of them tensor work, spills of
// 104 bytes stored and 120 loaded; issue slots 40 to 43 %, tensor pipe 28 to 35 %).
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
