// Attention over a paged cache, d = 128.
#include "fa_paged_launch.cuh"

namespace fa {
cudaError_t launch_fwd_paged_d128(const PagedFwdLaunch &L) {
    return L.bf16 ? launch_fwd_paged_inst<128, true>(L) : launch_fwd_paged_inst<128, false>(L);
}
}  // namespace fa
