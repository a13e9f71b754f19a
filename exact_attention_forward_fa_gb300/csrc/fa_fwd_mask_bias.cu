// The same with a bias that depends on the distance.
#include "fa_launch.cuh"

namespace fa {
cudaError_t launch_fwd_mask_bias(const FwdLaunch &L) {
    return L.d64 ? launch_fwd_ext_dispatch<64, 4>(L) : launch_fwd_ext_dispatch<128, 4>(L);
}
}  // namespace fa
