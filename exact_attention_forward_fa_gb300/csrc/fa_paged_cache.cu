// fa_paged_cache.cu -- the operators that move rows of a paged cache:
// fa_paged_append (new tokens into their pages) and fa_paged_evict (the
// tokens with the most accumulated attention weight into fresh pages).
#include "fa_paged.cuh"

namespace fa {

// ---------------------------------------------------------------------------
// Append.  pages[table[b][p / ps]][p % ps] = k[t], v[t] for every new token;
// pure copying: 2 x 2 x H_kv d elements read and as many written per token.
// One warp per token: its lanes copy the token's 16-byte vectors, all loads
// of a pass issued before the stores, and the loads of the first pass before
// the search for the token's sequence, whose latency they hide.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) fa_paged_append_kernel(const PagedAppendArgs a) {
    if (blockIdx.x == gridDim.x - 1)                     // the last block only checks
        return paged_check_seqs(a.cu_q, a.kv_len, a.B, a.T, a.W, a.ps_log2, a.status);
    const int lane = threadIdx.x & 31;
    const long long warp = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (warp >= a.T) return;
    const int t = static_cast<int>(warp);
    const uint4 *ks = reinterpret_cast<const uint4 *>(a.k) + static_cast<long long>(t) * (a.kv_stride / 8);
    const uint4 *vs = reinterpret_cast<const uint4 *>(a.v) + static_cast<long long>(t) * (a.kv_stride / 8);
    constexpr int U = 4;
    uint4 kr[U], vr[U];
    auto load = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * 32 + lane;
            if (i < a.row_vecs) {
                kr[u] = ks[i];
                vr[u] = vs[i];
            }
        }
    };
    load(0);
    const int b = paged_find_seq(a.cu_q, a.B, t);
    if (b < 0) return;                                   // behind the last sequence
    const PagedSeq s = paged_seq(a.cu_q, a.kv_len, b, a.T, a.W, a.ps_log2);
    const int p = s.n - s.m + (t - s.q0);
    if (p < 0 || p >= s.n) return;                       // more new tokens than the cache counts
    const int page = paged_page(a.table + static_cast<long long>(b) * a.W, p, a.ps_log2, a.n_pages,
                                a.status);
    if (page < 0) return;
    const long long at = static_cast<long long>(page) * (a.page_stride / 8) +
                         static_cast<long long>(p & ((1 << a.ps_log2) - 1)) * a.row_vecs;
    uint4 *kd = reinterpret_cast<uint4 *>(a.k_pages) + at;
    uint4 *vd = reinterpret_cast<uint4 *>(a.v_pages) + at;
    for (int i0 = 0;; ) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * 32 + lane;
            if (i < a.row_vecs) {
                kd[i] = kr[u];
                vd[i] = vr[u];
            }
        }
        i0 += U * 32;
        if (i0 >= a.row_vecs) break;
        load(i0);
    }
}

cudaError_t launch_paged_append(const PagedAppendArgs &a, cudaStream_t stream) {
    fa_paged_append_kernel<<<(a.T + 7) / 8 + 1, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Evict, first kernel: which tokens stay.  One CTA per (sequence, K/V head).
// Of n > keep cached tokens the first `first` and the last `recent` stay, and
// of the others the keep - first - recent with the largest score; equal
// scores go to the lower position, NaN ranks above +inf.  The k-th largest
// score is found by a radix select over an order-preserving 32-bit key, 8
// bits a pass; the kept positions are written in order.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);   // -0 equals +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;

__global__ void __launch_bounds__(kSelThreads) fa_paged_select_kernel(const PagedEvictArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t s_prefix, s_left;
    __shared__ int w_hi[32], w_eq[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.x, b = blockIdx.y;
    const long long cap = min(static_cast<long long>(a.W) << a.ps_log2, static_cast<long long>(a.L));
    const int n0 = a.kv_len[b];
    const int n = n0 < 0 ? 0 : static_cast<int>(min(static_cast<long long>(n0), cap));
    if (n != n0 && tid == 0) report_bad_index(a.status, 3);
    const long long bh = static_cast<long long>(b) * a.H_kv + h;
    const float *sc = a.scores + bh * a.L;
    int *kept = a.kept + bh * a.keep;
    float *so = a.scores_out ? a.scores_out + bh * a.keep : nullptr;
    const int len = min(n, a.keep);
    if (h == 0 && tid == 0) a.new_len[b] = len;
    if (n <= a.keep) {
        for (int j = tid; j < n; j += kSelThreads) {
            kept[j] = j;
            if (so) so[j] = sc[j];
        }
        return;
    }
    const int lo = a.first, hi = n - a.recent;            // the tokens that compete
    const uint32_t want = static_cast<uint32_t>(a.keep - a.first - a.recent);
    if (tid == 0) { s_prefix = 0; s_left = want; }
    // want = 0: a threshold above every key that competes
    for (int shift = 24; want != 0 && shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t prefix = s_prefix;
        const uint32_t above = shift == 24 ? 0u : (0xffffffffu << (shift + 8));
        for (int j = lo + tid; j < hi; j += kSelThreads) {
            const uint32_t k = score_key(sc[j]);
            if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l owns bins 255 - 8 l down to 248 - 8 l
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) { c[i] = hist[255 - 8 * lane - i]; sum += c[i]; }
            uint32_t before = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += v;
            }
            before -= sum;                                // keys above this lane's bins
            const uint32_t left = s_left;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (before < left && before + c[i] >= left) {
                    s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
                    s_left = left - before;
                }
                before += c[i];
            }
        }
        __syncthreads();
    }
    __syncthreads();
    const uint32_t thr = s_prefix;                        // the want-th largest key
    const uint32_t ties = want ? s_left : 0u;             // how many of its equals stay
    // every warp owns a run of whole 32-token groups
    const int groups = (n + 31) / 32, per = (groups + 31) / 32;
    const int g0 = min(groups, warp * per), g1 = min(groups, g0 + per);
    auto kind = [&](int j) __attribute__((always_inline)) -> int {   // 2 stays, 1 tie, 0 goes
        if (j >= n) return 0;
        if (j < lo || j >= hi) return 2;
        if (want == 0) return 0;
        const uint32_t k = score_key(sc[j]);
        return k > thr ? 2 : k == thr ? 1 : 0;
    };
    int c2 = 0, c1 = 0;
    for (int g = g0; g < g1; ++g) {
        const int k = kind(g * 32 + lane);
        c2 += __popc(__ballot_sync(0xffffffffu, k == 2));
        c1 += __popc(__ballot_sync(0xffffffffu, k == 1));
    }
    if (lane == 0) { w_hi[warp] = c2; w_eq[warp] = c1; }
    __syncthreads();
    int at = 0, eq = 0;                                   // stays and ties before this warp
    for (int w = 0; w < warp; ++w) { at += w_hi[w]; eq += w_eq[w]; }
    at += min(eq, static_cast<int>(ties));
    const unsigned below = (1u << lane) - 1u;
    for (int g = g0; g < g1; ++g) {
        const int j = g * 32 + lane;
        const int k = kind(j);
        const unsigned m1 = __ballot_sync(0xffffffffu, k == 1);
        const bool stay = k == 2 || (k == 1 && eq + __popc(m1 & below) < static_cast<int>(ties));
        const unsigned m = __ballot_sync(0xffffffffu, stay);
        if (stay) {
            const int r = at + __popc(m & below);
            kept[r] = j;
            if (so) so[r] = sc[j];
        }
        at += __popc(m);
        eq += __popc(m1);
    }
}

// Second kernel: row r of (b, h) in the fresh pages is the kept token's row.
// 16-byte vectors, one per thread and row; kRows rows per thread in flight.
constexpr int kMoveRows = 4;

template <int D>
__global__ void __launch_bounds__(256) fa_paged_move_kernel(const PagedEvictArgs a) {
    constexpr int V = D / 8;                              // vectors of a row
    constexpr int R = 256 / V;                            // rows per pass of the CTA
    const int h = blockIdx.y, b = blockIdx.z;
    const int n0 = a.kv_len[b];
    const long long cap = min(static_cast<long long>(a.W) << a.ps_log2, static_cast<long long>(a.L));
    const int len = n0 < 0 ? 0 : static_cast<int>(min(min(static_cast<long long>(n0), cap),
                                                      static_cast<long long>(a.keep)));
    const int c = threadIdx.x % V, r0 = blockIdx.x * (R * kMoveRows) + threadIdx.x / V;
    const int *kept = a.kept + (static_cast<long long>(b) * a.H_kv + h) * a.keep;
    const int mask = (1 << a.ps_log2) - 1;
    const uint4 *ks = reinterpret_cast<const uint4 *>(a.k_pages);
    const uint4 *vs = reinterpret_cast<const uint4 *>(a.v_pages);
    uint4 kr[kMoveRows], vr[kMoveRows];
    long long dst[kMoveRows];
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) {
        const int r = r0 + i * R;
        dst[i] = -1;
        if (r >= len) continue;
        const int j = kept[r];
        const int sp = paged_page(a.table + static_cast<long long>(b) * a.W, j, a.ps_log2, a.n_pages, a.status);
        const int dp = paged_page(a.dst_table + static_cast<long long>(b) * a.dst_W, r, a.ps_log2, a.n_pages,
                                  a.status);
        if (sp < 0 || dp < 0) continue;
        const long long src = static_cast<long long>(sp) * (a.page_stride / 8) +
                              (static_cast<long long>(j & mask) * a.H_kv + h) * V + c;
        dst[i] = static_cast<long long>(dp) * (a.page_stride / 8) +
                 (static_cast<long long>(r & mask) * a.H_kv + h) * V + c;
        kr[i] = ks[src];
        vr[i] = vs[src];
    }
#pragma unroll
    for (int i = 0; i < kMoveRows; ++i) {
        if (dst[i] < 0) continue;
        reinterpret_cast<uint4 *>(a.k_pages)[dst[i]] = kr[i];
        reinterpret_cast<uint4 *>(a.v_pages)[dst[i]] = vr[i];
    }
}

cudaError_t launch_paged_evict(const PagedEvictArgs &a, cudaStream_t stream) {
    fa_paged_select_kernel<<<dim3(a.H_kv, a.B), kSelThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int rows = (256 / (a.d / 8)) * kMoveRows;
    const dim3 grid((a.keep + rows - 1) / rows, a.H_kv, a.B);
    if (a.d == 64)
        fa_paged_move_kernel<64><<<grid, 256, 0, stream>>>(a);
    else
        fa_paged_move_kernel<128><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace fa
