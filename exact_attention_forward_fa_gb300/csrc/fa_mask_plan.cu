// fa_mask_plan.cu -- fa_mask_plan: the intervals and unit lists of fa_mask.cuh from
// documents' offsets on the device.  One launch; a training step makes it once for
// all layers.  Each token finds its document by bisection of the offsets; three
// further blocks a sequence sort the unit lists by their number of tiles (counting
// sort: which of two equally long units comes first may vary, no result depends on
// it).  Measured (GB300): 6 us for 2 x 8192 tokens (8 under the profiler, cold), the
// latency of the sorting blocks' dependent loads; it writes 16 bytes a token, 20 with the
// positions (which the torch wrapper always takes).
#include "fa_mask.cuh"
#include "fa_paged.cuh"

namespace fa {

namespace {

constexpr int kThreads = 256, kBuckets = 1024;

struct Docs {
    const int *at, *prefix;
    int D, N, wl, wr;

    __device__ __forceinline__ int offset(int k) const { return min(max(at[k], 0), N); }

    // Document [s, e) of token i and the end of its prefix; false outside.
    __device__ __forceinline__ bool find(int i, int &s, int &e, int &pe) const {
        int lo = 0, hi = D;                       // the last k with at[k] <= i
        if (at[0] > i) return false;
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (at[mid] <= i) lo = mid; else hi = mid - 1;
        }
        if (lo == D) return false;
        s = offset(lo);
        e = offset(lo + 1);
        if (i < s || i >= e) return false;        // (offsets that do not ascend)
        pe = prefix ? s + min(max(prefix[lo], 0), e - s) : s;
        return true;
    }
    // Written with min() so that no intermediate leaves [0, N] for any bound.
    __device__ __forceinline__ int2 keys(int i, int s, int e, int pe) const {
        const int lo = wl >= 0 ? max(s, i - min(wl, i)) : s;
        const int hi = wr >= 0 ? max(i + 1 + min(wr, e - 1 - i), pe) : e;
        return make_int2(lo, hi);
    }
    __device__ __forceinline__ int2 queries(int j, int s, int e, int pe) const {
        const int lo = wr >= 0 && j >= pe ? max(s, j - min(wr, j)) : s;
        const int hi = wl >= 0 ? j + 1 + min(wl, e - 1 - j) : e;
        return make_int2(lo, hi);
    }
    // Tiles that tokens [128 t, 128 t + 128) need: of keys, or of queries.
    template <bool kKeys>
    __device__ __forceinline__ int2 tiles(int t, int live_lo, int live_hi) const {
        const int r0 = max(t * 128, live_lo), r1 = min(t * 128 + 128, live_hi) - 1;
        if (r0 > r1) return make_int2(0, 0);
        int s, e, pe;
        int lo = 0, hi = 0;
        if (find(r0, s, e, pe)) lo = (kKeys ? keys(r0, s, e, pe) : queries(r0, s, e, pe)).x >> 7;
        if (find(r1, s, e, pe)) hi = ((kKeys ? keys(r1, s, e, pe) : queries(r1, s, e, pe)).y + 127) >> 7;
        return make_int2(lo, max(lo, hi));
    }
};

// Sorts units 0 .. n by cost(u), the longest first: out(u, place).
template <class Cost, class Out>
__device__ void sort_units(int n, int most, Cost &&cost, Out &&out) {
    __shared__ int count[kBuckets];
    for (int i = threadIdx.x; i < kBuckets; i += kThreads) count[i] = 0;
    __syncthreads();
    auto bucket = [&](int u) {
        return kBuckets - 1 - static_cast<int>(static_cast<long long>(min(cost(u), most)) * (kBuckets - 1) / most);
    };
    for (int u = threadIdx.x; u < n; u += kThreads) atomicAdd(&count[bucket(u)], 1);
    __syncthreads();
    // each thread's buckets, then the threads' sums over lanes and warps
    constexpr int kEach = kBuckets / kThreads;
    __shared__ int warp_sum[kThreads / 32];
    int c[kEach], mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        c[i] = count[threadIdx.x * kEach + i];
        mine += c[i];
    }
    const int lane = threadIdx.x & 31;
    int upto = mine;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, upto, w);
        if (lane >= w) upto += below;
    }
    if (lane == 31) warp_sum[threadIdx.x / 32] = upto;
    __syncthreads();
    int at = upto - mine;
    for (int w = 0; w < static_cast<int>(threadIdx.x) / 32; ++w) at += warp_sum[w];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        count[threadIdx.x * kEach + i] = at;
        at += c[i];
    }
    __syncthreads();
    for (int u = threadIdx.x; u < n; u += kThreads) out(u, atomicAdd(&count[bucket(u)], 1));
}

}  // namespace

__global__ void __launch_bounds__(kThreads) fa_mask_plan_kernel(const MaskPlanArgs a) {
    const int b = blockIdx.y;
    const Docs d{a.docs + static_cast<size_t>(b) * (a.D + 1), a.prefix ? a.prefix + static_cast<size_t>(b) * a.D : nullptr,
                 a.D, a.N, a.wl, a.wr};
    if (blockIdx.x >= 3) {                        // tokens
        const long long t = (blockIdx.x - 3ll) * kThreads + threadIdx.x;
        if (t >= a.N) return;
        const int i = static_cast<int>(t);
        int s = 0, e = 0, pe = 0;
        const bool in = d.find(i, s, e, pe);
        const size_t at = static_cast<size_t>(b) * a.N + i;
        const_cast<int2 *>(a.plan.rows)[at] = in ? d.keys(i, s, e, pe) : make_int2(0, 0);
        const_cast<int2 *>(a.plan.cols)[at] = in ? d.queries(i, s, e, pe) : make_int2(0, 0);
        if (a.positions) a.positions[at] = in ? i - s : 0;
        return;
    }
    const int live_lo = d.offset(0), live_hi = max(d.offset(a.D), d.offset(0));
    const int n_t = (a.N - 1) / 128 + 1, n_p = (n_t + 1) / 2;
    if (blockIdx.x == 0) {                        // pairs of query tiles
        if (threadIdx.x == 0) const_cast<int4 *>(a.plan.live)[b] = make_int4(live_lo, live_hi, 0, 0);
        // offsets that leave [0, N] or do not ascend, prefixes longer than their document
        for (int k = threadIdx.x; k <= a.D; k += kThreads) {
            const int x = d.at[k], y = d.at[min(k + 1, a.D)];
            if (x < 0 || x > a.N || y < x) report_bad_index(a.status, 4);
            else if (d.prefix && k < a.D && (d.prefix[k] < 0 || d.prefix[k] > y - x)) report_bad_index(a.status, 5);
        }
        auto ranges = [&](int p, int2 &x, int2 &y) {
            x = d.tiles<true>(2 * p, live_lo, live_hi);
            y = 2 * p + 1 < n_t ? d.tiles<true>(2 * p + 1, live_lo, live_hi) : make_int2(0, 0);
        };
        int4 *out = const_cast<int4 *>(a.plan.pairs) + static_cast<size_t>(b) * n_p * 2;
        sort_units(n_p, n_t, [&](int p) {
            int2 x, y;
            ranges(p, x, y);
            if (x.y <= x.x) return y.y - y.x;
            if (y.y <= y.x) return x.y - x.x;
            return max(x.y, y.y) - min(x.x, y.x);
        }, [&](int p, int place) {
            int2 x, y;
            ranges(p, x, y);
            out[2 * place] = make_int4(p, x.x, x.y, live_lo);
            out[2 * place + 1] = make_int4(0, y.x, y.y, live_hi);
        });
    } else if (blockIdx.x == 1) {                 // query tiles
        int4 *out = const_cast<int4 *>(a.plan.qtiles) + static_cast<size_t>(b) * n_t;
        sort_units(n_t, n_t, [&](int t) {
            const int2 x = d.tiles<true>(t, live_lo, live_hi);
            return x.y - x.x;
        }, [&](int t, int place) {
            const int2 x = d.tiles<true>(t, live_lo, live_hi);
            out[place] = make_int4(t, x.x, x.y, 0);
        });
    } else {                                      // key tiles
        int4 *out = const_cast<int4 *>(a.plan.ktiles) + static_cast<size_t>(b) * n_t;
        sort_units(n_t, n_t, [&](int t) {
            const int2 x = d.tiles<false>(t, live_lo, live_hi);
            return x.y - x.x;
        }, [&](int t, int place) {
            const int2 x = d.tiles<false>(t, live_lo, live_hi);
            out[place] = make_int4(t, x.x, x.y, 0);
        });
    }
}

cudaError_t launch_mask_plan(const MaskPlanArgs &a, cudaStream_t stream) {
    const dim3 grid(3u + static_cast<unsigned>((static_cast<long long>(a.N) + kThreads - 1) / kThreads),
                    static_cast<unsigned>(a.B));
    fa_mask_plan_kernel<<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace fa
