// Attention over a paged cache, d = 128.
#include "fa_paged_launch.cuh"

namespace fa {
cudaError_t launch_fwd_paged_d128(const PagedFwdLaunch &L) {
    return launch_fwd_paged_dispatch<128>(L);
}
}  // namespace fa
