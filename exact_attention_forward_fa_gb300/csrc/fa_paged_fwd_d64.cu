// Attention over a paged cache, d = 64.
#include "fa_paged_launch.cuh"

namespace fa {
cudaError_t launch_fwd_paged_d64(const PagedFwdLaunch &L) {
    return launch_fwd_paged_dispatch<64>(L);
}
}  // namespace fa
