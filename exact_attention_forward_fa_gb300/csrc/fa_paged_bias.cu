// Attention over a paged cache with a bias that depends on the distance, S_ij = alpha
// q_i k_j - beta_h |p_i - j| for a row at place p_i.  Measured (GB300): 64 single tokens of
// 32 heads over 8 on up to 8192 cached ones (bf16, d 128) 172 us and the joining kernel 3.3, as without
// a bias (HBM, 6.3 TB/s; eight FMAs a key and thread); 24 sequences of 1 to 300 new tokens
// on up to 4096 (fp16) 101 to 103 us with the joining kernel (10; without a bias 92 with it),
// bound by each tile's chain and the code's footprint (d 128: spills of 184 bytes stored and 220 loaded).
#include "fa_paged_launch.cuh"

namespace fa {
cudaError_t launch_fwd_paged_bias(const PagedFwdLaunch &L) {
    return L.d == 64 ? launch_fwd_paged_dispatch<64, true>(L) : launch_fwd_paged_dispatch<128, true>(L);
}
}  // namespace fa
