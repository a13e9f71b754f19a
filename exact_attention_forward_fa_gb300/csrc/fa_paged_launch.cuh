// fa_paged_launch.cuh -- launches the attention over a paged cache and the
// kernel that joins its parts.
#pragma once

#include "fa_paged_fwd_kernel.cuh"

namespace fa {

template <int D, bool kBF16, bool kNarrow>
cudaError_t launch_fwd_paged_inst(const PagedFwdLaunch &L) {
    using C = PagedCfg<D, kBF16, kNarrow>;
    auto kern = fa_paged_fwd_kernel<D, kBF16, kNarrow>;
    static unsigned long long configured = 0ull;   // bit per device id (< 64)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(C::SMEM_BYTES));
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&configured, bit, __ATOMIC_ACQ_REL);
    }
    kern<<<L.grid, C::NTHREADS, C::SMEM_BYTES, L.stream>>>(L.q, L.k, L.v, L.a, L.w, L.R, L.q_min);
    e = cudaGetLastError();
    if (e != cudaSuccess || L.grid == 1) return e;  // one share: nothing is cut
    // The joining kernel's CTAs are brought up while the attention's last ones
    // run; it waits for their results itself (griddepcontrol.wait).
    const int rows = 2 * L.R * L.a.group;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.grid, rows < 16 ? rows : 16);
    cfg.blockDim = dim3(256);
    cfg.stream = L.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_paged_combine_kernel<D, kBF16>, L.a, L.w, L.R);
}

template <int D>
cudaError_t launch_fwd_paged_dispatch(const PagedFwdLaunch &L) {
    if (L.R * L.a.group <= 32)
        return L.bf16 ? launch_fwd_paged_inst<D, true, true>(L) : launch_fwd_paged_inst<D, false, true>(L);
    return L.bf16 ? launch_fwd_paged_inst<D, true, false>(L) : launch_fwd_paged_inst<D, false, false>(L);
}

}  // namespace fa
