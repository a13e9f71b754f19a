// fa_bwd_mask.cu -- the backward for the intervals of a mask plan (documents,
// prefixes, windows): fa_bwd_kernel.cuh's three kernels over the plan's sorted query and
// key tiles, P and dS nonzero only where row i sees column j.  The kernels overlap at
// their ends: the dQ kernel reads nothing that the dK/dV kernel writes.  Measured (GB300,
// bf16): 2 x 8192 tokens, 32 heads of 128 over 8, documents of 200 to 4000, causal: 938 to 955
// us (statistics 47, HBM; dK/dV 465 and dQ 377, tensor pipe 69 and 62 %), 851 to 866 TFLOP/s of the
// visible pairs' five products, of which S and dP are formed twice.
#include "fa_bwd_launch.cuh"

namespace fa {

cudaError_t launch_bwd_mask(const BwdLaunch &L) {
    if (L.d == 64)
        return L.bf16 ? launch_bwd_inst<64, false, true, false, false, true, false>(L)
                      : launch_bwd_inst<64, false, false, false, false, true, false>(L);
    return L.bf16 ? launch_bwd_inst<128, false, true, false, false, true, false>(L)
                  : launch_bwd_inst<128, false, false, false, false, true, false>(L);
}

}  // namespace fa
