// fa_bwd_mask_bias.cu -- the backward for a mask plan with a bias that depends on the
// distance.
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
