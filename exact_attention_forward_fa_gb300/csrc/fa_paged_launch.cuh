// fa_paged_launch.cuh -- launches the attention over a paged cache and the
// kernel that joins its parts.
#pragma once

#include <type_traits>

#include "fa_paged_combine.cuh"
#include "fa_paged_fwd_kernel.cuh"
#include "fa_paged_token_kernel.cuh"

namespace fa {

// kFew: the kernel for few rows, else the one for chunks; kBias: with a distance bias.
template <int D, bool kBF16, bool kFew, bool kBias>
cudaError_t launch_fwd_paged_inst(const PagedFwdLaunch &L) {
    using C = std::conditional_t<kFew, TokenCfg<D, kBF16>, PagedCfg<D, kBF16>>;
    void (*kern)(CUtensorMap, CUtensorMap, CUtensorMap, PagedArgs, PagedWork, int);
    if constexpr (kFew) kern = fa_paged_token_kernel<D, kBF16, kBias>;
    else kern = fa_paged_fwd_kernel<D, kBF16, kBias>;
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
    kern<<<L.grid, C::NTHREADS, C::SMEM_BYTES, L.stream>>>(L.q, L.k, L.v, L.a, L.w, L.R);
    e = cudaGetLastError();
    if (e != cudaSuccess || L.grid == 1) return e;  // one share: nothing is cut
    // The joining kernel is launched when every CTA of the attention is at its end
    // (their last statement lets it come), so that its launch overlaps their
    // teardown, nothing more; it waits for their results itself (griddepcontrol.wait).
    const int rows = (kFew ? 1 : 2) * L.R * L.a.group;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.grid, rows < 8 ? rows : 8);
    cfg.blockDim = dim3(256);
    cfg.stream = L.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_paged_combine_kernel<D, kBF16, kFew>, L.a, L.w, L.R);
}

// Up to kFewRows rows a tile: few rows against each K/V tile, bound by HBM.  64
// single tokens of 4 heads a group (4 rows) on up to 8192 188 us, one on 777 tokens 11.8,
// up to 4 rows of d = 64 with a window 60; the chunk kernel 197, 12.8 and 89 for the same.
template <int D, bool kBias = false>
cudaError_t launch_fwd_paged_dispatch(const PagedFwdLaunch &L) {
    if (L.R * L.a.group <= kFewRows)
        return L.bf16 ? launch_fwd_paged_inst<D, true, true, kBias>(L) : launch_fwd_paged_inst<D, false, true, kBias>(L);
    return L.bf16 ? launch_fwd_paged_inst<D, true, false, kBias>(L) : launch_fwd_paged_inst<D, false, false, kBias>(L);
}

}  // namespace fa
