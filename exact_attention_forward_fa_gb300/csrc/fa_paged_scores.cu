// fa_paged_scores.cu -- the attention weight that each cached token of a
// paged cache gets from the new tokens.
#include "fa_paged.cuh"

namespace fa {

template <bool kBF16>
__device__ __forceinline__ float to_f32(uint16_t x) {
    float lo, hi;
    unpack2<kBF16>(x, lo, hi);
    return lo;
}

// One warp per (sequence, K/V head, cached token): the rows that see it, one
// by one, in a fixed order.
template <int D, bool kBF16>
__global__ void __launch_bounds__(256) fa_paged_scores_kernel(const PagedScoresArgs g) {
    constexpr int E = D / 32;
    const PagedArgs &a = g.p;
    const int lane = threadIdx.x & 31;
    const int j = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int hk = blockIdx.y, b = blockIdx.z;
    const PagedSeq s = paged_seq(a.cu_q, a.kv_len, b, a.T, a.W, a.ps_log2);
    if (s.bad && lane == 0) report_bad_index(a.status, 1);
    if (s.n > g.L && lane == 0) report_bad_index(a.status, 3);
    if (j >= s.n || j >= g.L) return;
    const int page = paged_page(a.table + static_cast<long long>(b) * a.W, j, a.ps_log2, a.n_pages, a.status);
    const long long at = page * a.page_stride +
        (static_cast<long long>(j & ((1 << a.ps_log2) - 1)) * a.H_kv + hk) * D + lane * E;
    float k[E];
    for (int e = 0; e < E; ++e)
        k[e] = page < 0 ? 0.f : to_f32<kBF16>(reinterpret_cast<const uint16_t *>(a.k_pages)[at + e]);
    const int old = s.n - s.m;
    float sum = 0.f;
    for (int i = 0; i < s.m; ++i) {
        const int p = old + i;
        if (j >= paged_hi(p, s.n, a.wr) || (j < paged_lo(p, a.wl) && j >= a.first)) continue;
        for (int h = hk * a.group; h < (hk + 1) * a.group; ++h) {
            const uint16_t *qr = reinterpret_cast<const uint16_t *>(a.q) + (s.q0 + i) * a.q_stride + h * D + lane * E;
            float x = 0.f;
            for (int e = 0; e < E; ++e) x += to_f32<kBF16>(qr[e]) * k[e];
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            const float z = a.lse[static_cast<long long>(h) * a.T + s.q0 + i];
            if (z != -INFINITY) sum += exp2f(fmaf(x, a.scale_log2, -z * 1.44269504088896340736f));
        }
    }
    const long long w = (static_cast<long long>(b) * a.H_kv + hk) * g.L + j;
    if (lane == 0) g.out[w] = (g.in != nullptr && j < old ? g.in[w] : 0.f) + sum;
}

cudaError_t launch_paged_scores(const PagedScoresArgs &g, int d, bool bf16, int, cudaStream_t stream) {
    const long long most = min(static_cast<long long>(g.L), static_cast<long long>(g.p.W) << g.p.ps_log2);
    const dim3 grid(static_cast<unsigned>((most + 7) / 8), g.p.H_kv, g.p.B);
    if (d == 64)
        bf16 ? fa_paged_scores_kernel<64, true><<<grid, 256, 0, stream>>>(g)
             : fa_paged_scores_kernel<64, false><<<grid, 256, 0, stream>>>(g);
    else
        bf16 ? fa_paged_scores_kernel<128, true><<<grid, 256, 0, stream>>>(g)
             : fa_paged_scores_kernel<128, false><<<grid, 256, 0, stream>>>(g);
    return cudaGetLastError();
}

}  // namespace fa
