// fa_bwd_mask.cu -- the backward for the intervals of a mask plan (documents,
// prefixes, windows).
#include "fa_bwd_launch.cuh"

namespace fa {

cudaError_t launch_bwd_mask(const BwdLaunch &L) {
    if (L.d == 64)
        return L.bf16 ? launch_bwd_inst<64, false, true, false, false, true, false>(L)
                      : launch_bwd_inst<64, false, false, false, false, true, false>(L);
    return L.bf16 ? launch_bwd_inst<128, false, true, false, false, true, false>(L)
                  : launch_bwd_inst<128, false, false, false, false, true, false>(L);
}

}  // namespace fa
