// Instantiations of the attention forward kernel with the intervals of a mask
// plan (documents, prefixes, windows): O_i = sum_j P_ij v_j over j in [lo_i, hi_i).
//
// Only the key tiles that a pair of Q tiles sees are loaded (the plan's union of the rows'
// intervals), and only tiles that some row of a warp sees in part pay for a mask, as bits of the
// columns.  Bound by the tensor core and the softmax chain, at the ends of units by a
// step's latency.  Measured (GB300, bf16): 2 x 8192 tokens, 32 heads of 128 over 8,
// documents of 200 to 4000 tokens, causal: 237 to 241 us, 935 to 951 TFLOP/s of the visible pairs (83 %
// of the computed tiles' elements); one document 702 us, 1567; fp16, 4 x 4001, 32 heads
// of 64, prefixes: 286 us, 684.
#include "fa_launch.cuh"

namespace fa {
cudaError_t launch_fwd_mask(const FwdLaunch &L) {
    return L.d64 ? launch_fwd_ext_dispatch<64, 3>(L) : launch_fwd_ext_dispatch<128, 3>(L);
}
}  // namespace fa
