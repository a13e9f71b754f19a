// Instantiations of the attention forward kernel with the intervals of a mask
// plan (documents, prefixes, windows).
#include "fa_launch.cuh"

namespace fa {
cudaError_t launch_fwd_mask(const FwdLaunch &L) {
    return L.d64 ? launch_fwd_ext_dispatch<64, 3>(L) : launch_fwd_ext_dispatch<128, 3>(L);
}
}  // namespace fa
