// Attention over a paged cache, d = 64.
#include "fa_paged_launch.cuh"

namespace fa {
cudaError_t launch_fwd_paged_d64(const PagedFwdLaunch &L) {
    return L.bf16 ? launch_fwd_paged_inst<64, true>(L) : launch_fwd_paged_inst<64, false>(L);
}
}  // namespace fa
