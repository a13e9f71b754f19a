// The same with a bias that depends on the distance: S_ij = alpha q_i k_j - beta_h |i - j|.
// In a tile beside the diagonal one the bias is linear in the column: four packed pairs
// start at b0 + bs c and step by eight columns, one packed addition for two scores
// (6 % of a long document's time); on the diagonal tile |i - j| is formed for each.
// Measured (GB300, bf16): 16384 tokens, 16 heads of 128, causal: 710 to 748 us, 1470 to 1550
// TFLOP/s, bound as the forward without a bias.
#include "fa_launch.cuh"

namespace fa {
cudaError_t launch_fwd_mask_bias(const FwdLaunch &L) {
    return L.d64 ? launch_fwd_ext_dispatch<64, 4>(L) : launch_fwd_ext_dispatch<128, 4>(L);
}
}  // namespace fa
