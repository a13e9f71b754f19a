// Attention over a paged cache with a bias that depends on the distance.
#include "fa_paged_launch.cuh"

namespace fa {
cudaError_t launch_fwd_paged_bias(const PagedFwdLaunch &L) {
    return L.d == 64 ? launch_fwd_paged_dispatch<64, true>(L) : launch_fwd_paged_dispatch<128, true>(L);
}
}  // namespace fa
