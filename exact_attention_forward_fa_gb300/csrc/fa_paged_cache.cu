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
// the search for the token's sequence, whose latency they hide.  64 single tokens
// of 8 heads of 128: 3.4 us, the latency of a launch and of three dependent loads;
// four chunks, 10240 tokens (84 MB in and out): 16.2 us, 5.2 TB/s.
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
    // The position as the caller's numbers have it: a length or an offset that is out
    // of range moves no token into the slot of another.
    const long long n = a.kv_len[b], at_p = n - a.cu_q[b + 1] + t;
    if (at_p < 0 || at_p >= min(n, static_cast<long long>(a.W) << a.ps_log2)) return;   // no slot
    const int p = static_cast<int>(at_p);
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
// Evict, the rows.
// ---------------------------------------------------------------------------
// Cached tokens of sequence b (as far as the table and the scores go).
__device__ __forceinline__ int evict_tokens(const PagedEvictArgs &a, int b) {
    // (2^31 - 2^20: indices past the end stay within 32 bits)
    const long long cap = min(min(static_cast<long long>(a.W) << a.ps_log2, static_cast<long long>(a.L)), 0x7ff00000ll);
    const int n0 = a.kv_len[b];
    return n0 < 0 ? 0 : static_cast<int>(min(static_cast<long long>(n0), cap));
}
__device__ __forceinline__ int evict_len(const PagedEvictArgs &a, int b) { return min(evict_tokens(a, b), a.keep); }

// Copies rows of (b, h) to the fresh pages: for i = first, first + step, ... below
// len (each call kThreads / V * kMoveRows of them) row_of(i, r, j) tells the row and
// the token that goes there.  V 16-byte vectors a row, one a thread; kMoveRows rows
// of K and V in flight per thread.  Where a row lies takes two dependent loads, its
// token and that token's page: those of the next rows are read while these are copied.
constexpr int kMoveRows = 4;

template <int D, int kThreads, class RowOf>
__device__ __forceinline__ void move_rows(const PagedEvictArgs &a, int b, int h, int first, int step, int len,
                                          RowOf &&row_of) {
    constexpr int V = D / 8, R = kThreads / V;
    const int c = threadIdx.x % V, r0 = threadIdx.x / V;
    const int mask = (1 << a.ps_log2) - 1;
    uint4 *kp = reinterpret_cast<uint4 *>(a.k_pages), *vp = reinterpret_cast<uint4 *>(a.v_pages);
    long long src[kMoveRows], dst[kMoveRows];             // in vectors; dst < 0: none
    auto find = [&](int at) __attribute__((always_inline)) {
        int j[kMoveRows], to[kMoveRows];
#pragma unroll
        for (int i = 0; i < kMoveRows; ++i) {
            j[i] = -1;
            to[i] = 0;
            if (at + r0 + i * R < len) row_of(at + r0 + i * R, to[i], j[i]);
        }
#pragma unroll
        for (int i = 0; i < kMoveRows; ++i) {
            const int r = to[i];
            dst[i] = -1;
            if (j[i] < 0) continue;
            const int sp = paged_page(a.table + static_cast<long long>(b) * a.W, j[i], a.ps_log2, a.n_pages, a.status);
            const int dp = paged_page(a.dst_table + static_cast<long long>(b) * a.dst_W, r, a.ps_log2, a.n_pages,
                                      a.status);
            if (sp < 0 || dp < 0) continue;
            src[i] = static_cast<long long>(sp) * (a.page_stride / 8) +
                     (static_cast<long long>(j[i] & mask) * a.H_kv + h) * V + c;
            dst[i] = static_cast<long long>(dp) * (a.page_stride / 8) +
                     (static_cast<long long>(r & mask) * a.H_kv + h) * V + c;
        }
    };
    if (first < len) find(first);
#pragma unroll 1
    for (int at = first; at < len; at += step) {
        uint4 kr[kMoveRows], vr[kMoveRows];
        long long to[kMoveRows];
#pragma unroll
        for (int i = 0; i < kMoveRows; ++i) {
            to[i] = dst[i];
            if (to[i] < 0) continue;
            kr[i] = kp[src[i]];
            vr[i] = vp[src[i]];
        }
        if (at + step < len) find(at + step);
#pragma unroll
        for (int i = 0; i < kMoveRows; ++i) {
            if (to[i] < 0) continue;
            kp[to[i]] = kr[i];
            vp[to[i]] = vr[i];
        }
    }
}

template <int D>
__global__ void __launch_bounds__(256) fa_paged_move_kernel(const PagedEvictArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");    // the kept positions
    const int h = blockIdx.y, b = blockIdx.z;
    constexpr int kRows = 256 / (D / 8) * kMoveRows;
    const int *kept = a.kept + (static_cast<long long>(b) * a.H_kv + h) * a.keep;
    move_rows<D, 256>(a, b, h, blockIdx.x * kRows, gridDim.x * kRows, evict_len(a, b),
                      [&](int i, int &r, int &j) { r = i; j = kept[i]; });
}

// ---------------------------------------------------------------------------
// Evict, which tokens stay.  One CTA per (sequence, K/V head).
// Of n > keep cached tokens the first `first` and the last `recent` stay, and
// of the others the keep - first - recent with the largest score; equal
// scores go to the lower position, NaN ranks above +inf.
//
// The want-th largest score is searched over an order-preserving 32-bit key by
// digits of 12 bits, from the first bit in which the keys differ, counted with
// shared-memory atomics.  The digits are wide so that a warp's keys spread over
// many bins: with 8 bits the first digit is little more than the exponent, and a
// warp's 32 additions go to a few addresses, one after the other.  Up to
// kSelStaged tokens the scores are read once and their keys kept in shared
// memory; longer caches are read again for each pass.
//
// What it takes is latency and issue slots, not bytes, so a pass does little more
// than read a key and compare.  Caches of 15400 tokens: 15 us (of which 5 read
// the scores, 2.5 a digit; it ends at the digit below which all keys of the bin stay);
// 23 with scores staged instead of keys (whose order is made anew in every pass) and
// places found by ballots, 26 reading the scores again for each digit, 40 with keys in
// registers and unrolled loops (their code comes from L2 once a launch), 56 with
// bins counted by ballots (a vote costs ~16 issue cycles).
//
// The kept positions are written in order: every thread owns a run of tokens (an
// odd number, so that a warp's reads of its runs fall into different banks) and
// counts those that stay and its ties; a scan over the threads gives their places.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t score_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);   // -0 equals +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024, kSelStaged = 49152;     // (192 KB)

// Inclusive sums over the block's threads (kSelThreads of them); `sums`: 32 words of
// shared memory, read by all when it returns.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    return v + __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0u);
}

// staged: the keys of the n tokens go to `held`.
__device__ __forceinline__ void select_tokens(const PagedEvictArgs &a, const bool staged, uint32_t *held) {
    __shared__ uint32_t hist[4096];                       // a digit's bins
    __shared__ uint32_t s_and, s_or, s_digit, s_left, s_all;
    __shared__ uint32_t sums[3][32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int h = blockIdx.x, b = blockIdx.y;
    const int n = evict_tokens(a, b);
    if (tid == 0 && n != a.kv_len[b]) report_bad_index(a.status, 3);
    const long long bh = static_cast<long long>(b) * a.H_kv + h;
    const float *sc = a.scores + bh * a.L;
    int *kept = a.kept + bh * a.keep;
    float *so = a.scores_out ? a.scores_out + bh * a.keep : nullptr;
    if (h == 0 && tid == 0 && a.new_len != a.kv_len) a.new_len[b] = min(n, a.keep);
    if (n <= a.keep) {
        for (int j = tid; j < n; j += kSelThreads) {
            kept[j] = j;
            if (so) so[j] = sc[j];
        }
        return;
    }
    const int lo = a.first, hi = n - a.recent;            // the tokens that compete
    const uint32_t want = static_cast<uint32_t>(a.keep - a.first - a.recent);
    // keys(j0, j1, step, f): f(j, key) for j = j0, j0 + step, ... below j1; the key
    // is 0 (less than any real one) where none competes
    auto keys = [&](int j0, int j1, int step, auto &&f) __attribute__((always_inline)) {
        if (staged) {
#pragma unroll 4
            for (int j = j0; j < j1; j += step) f(j, held[j]);
        } else {
#pragma unroll 4
            for (int j = j0; j < j1; j += step) f(j, j >= lo && j < hi ? score_key(sc[j]) : 0u);
        }
    };
    uint32_t all = ~0u, any = 0u;
    if (tid == 0) { s_and = ~0u; s_or = 0u; }
#pragma unroll 1
    for (int j0 = tid; j0 < n; j0 += 8 * kSelThreads) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = j0 + i * kSelThreads < n ? sc[j0 + i * kSelThreads] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + i * kSelThreads;
            const bool competes = j >= lo && j < hi;
            const uint32_t k = competes ? score_key(x[i]) : 0u;
            if (staged && j < n) held[j] = k;
            all &= competes ? k : ~0u;
            any |= k;
        }
    }
    __syncthreads();
    all = __reduce_and_sync(0xffffffffu, all);
    any = __reduce_or_sync(0xffffffffu, any);
    if (lane == 0) { atomicAnd(&s_and, all); atomicOr(&s_or, any); }
    for (int i = tid; i < 4096; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    int top = 32 - __clz(s_and ^ s_or);                   // bits to decide; the others are common
    uint32_t prefix = top == 32 ? 0u : (s_or >> top) << top, left = want;
#pragma unroll 1
    while (want != 0 && top > 0) {
        const int low = max(top - 12, 0), bins = 1 << (top - low);
        const uint32_t common = top == 32 ? 0u : ~0u << top;
        keys(tid, n, kSelThreads, [&](int, uint32_t k) __attribute__((always_inline)) {
            if (((k ^ prefix) & common) == 0u) atomicAdd(&hist[(k >> low) & (bins - 1)], 1u);
        });
        __syncthreads();
        // thread t sums bins 4095 - 4 t down to 4092 - 4 t; the digit is the bin
        // that holds the left-th key from the top
        uint32_t c[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = hist[4095 - 4 * tid - i];
            hist[4095 - 4 * tid - i] = 0;                 // (for the next digit)
            sum += c[i];
        }
        uint32_t above = block_scan(sum, sums[0]) - sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (above < left && above + c[i] >= left) {
                s_digit = static_cast<uint32_t>(4095 - 4 * tid - i);
                s_left = left - above;
                s_all = c[i] == left - above;             // all keys of the bin stay
            }
            above += c[i];
        }
        __syncthreads();
        left = s_left;
        prefix |= s_digit << low;
        top = low;
        if (s_all) break;
    }
    const uint32_t mask = top == 32 ? 0u : ~0u << top;    // (the bits below decide nothing)
    const uint32_t thr = prefix;                          // the want-th largest key
    const uint32_t ties = want ? left : 0u;               // how many of its equals stay
    // 2 stays, 1 tie, 0 goes
    auto rank = [&](int j, uint32_t k) __attribute__((always_inline)) -> int {
        if (j < lo || j >= hi) return 2;
        return want == 0 ? 0 : (k & mask) > thr ? 2 : (k & mask) == thr ? 1 : 0;
    };
    const int per = ((n + kSelThreads - 1) / kSelThreads) | 1;
    const int j0 = static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(tid) * per));
    const int j1 = min(n, j0 + per);
    uint32_t c2 = 0, c1 = 0;
    keys(j0, j1, 1, [&](int j, uint32_t k) __attribute__((always_inline)) {
        const int r = rank(j, k);
        c2 += r == 2;
        c1 += r == 1;
    });
    uint32_t eq = block_scan(c1, sums[1]) - c1;           // ties, and tokens that stay anyway, before this thread's
    uint32_t at = block_scan(c2, sums[2]) - c2 + min(eq, ties);
    keys(j0, j1, 1, [&](int j, uint32_t k) __attribute__((always_inline)) {
        const int r = rank(j, k);
        if (r == 2 || (r == 1 && eq < ties)) kept[at++] = j;
        eq += r == 1;
    });
    if (so) {
        __syncthreads();
#pragma unroll 4
        for (int r = tid; r < a.keep; r += kSelThreads) so[r] = sc[kept[r]];
    }
}

// D != 0: the CTA then moves the rows that it chose.  Those that stay anyway need not
// wait for the choice: CTAs of their own (z = 1) move the first and the last ones,
// or all of a short cache.  A CTA takes an SM's whole register file (1024 threads of 64),
// so these run on the SMs that no choosing CTA has, the others behind them.
template <int D>
__global__ void __launch_bounds__(kSelThreads) fa_paged_select_kernel(const PagedEvictArgs a, const bool staged) {
    extern __shared__ uint32_t held[];
    if constexpr (D == 0) {
        select_tokens(a, staged, held);
    } else {
        constexpr int kRows = kSelThreads / (D / 8) * kMoveRows;
        const int h = blockIdx.x, b = blockIdx.y, n = evict_tokens(a, b);
        if (blockIdx.z == 0) {
            select_tokens(a, staged, held);
            if (n <= a.keep) return;
            __syncthreads();                              // the kept positions are written
            const int *kept = a.kept + (static_cast<long long>(b) * a.H_kv + h) * a.keep + a.first;
            move_rows<D, kSelThreads>(a, b, h, 0, kRows, a.keep - a.first - a.recent,
                                      [&](int i, int &r, int &j) { r = a.first + i; j = kept[i]; });
        } else {
            const bool all = n <= a.keep;
            move_rows<D, kSelThreads>(a, b, h, 0, kRows, all ? n : a.first + a.recent, [&](int i, int &r, int &j) {
                const bool front = all || i < a.first;
                r = front ? i : a.keep - a.recent + (i - a.first);
                j = front ? i : n - a.recent + (i - a.first);
            });
        }
    }
}

template <int D>
static cudaError_t launch_select(const PagedEvictArgs &a, cudaStream_t stream) {
    static unsigned long long configured = 0ull;          // bit per device id (< 64)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & bit)) {
        e = cudaFuncSetAttribute(fa_paged_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelStaged * 4);
        if (e != cudaSuccess) return e;
        __atomic_fetch_or(&configured, bit, __ATOMIC_ACQ_REL);
    }
    const long long most = min(static_cast<long long>(a.W) << a.ps_log2, static_cast<long long>(a.L));
    const bool staged = most <= kSelStaged;
    fa_paged_select_kernel<D><<<dim3(a.H_kv, a.B, D ? 2 : 1), kSelThreads, staged ? most * 4 : 0, stream>>>(a, staged);
    return cudaGetLastError();
}

// With a (sequence, K/V head) for most of the SMs the CTA that selects also
// moves: short caches move while long ones still select (sixteen caches cut to
// 2048 tokens of 8 heads, 268 MB: 57 us, 4.7 TB/s; bound by HBM behind ~10 us of
// selection that nothing covers).  With few, moving is spread over the whole device
// by a kernel of its own, launched when the last selection ends (two caches cut to
// 512: 12.3 us, latency).  The border, two kernels against one, in us: caches of up to
// 2048 cut to 512, of up to 16384 cut to 2048 (d = 128) and of up to 6000 cut to 1024
// (d = 64), 8 heads:
//     16 pairs   11.3 / 14.4    22 / 43    13.3 / 18.4
//     64         15.5 / 15.5    43 / 48    17.5 / 18.5
//     96         19.4 / 17.5    55 / 53    21.7 / 20.0
//     128        24.6 / 21.6    65 / 61    27.5 / 22.6
//     152        26.6 / 24.7    74 / 76    28.9 / 27.1
//     256        42.5 / 38.9   119 / 108   46.8 / 42.0
static cudaError_t launch_evict_rows(const PagedEvictArgs &a, int sm_count, cudaStream_t stream) {
    if (static_cast<long long>(a.B) * a.H_kv * 3 >= 2ll * sm_count)
        return a.d == 64 ? launch_select<64>(a, stream) : launch_select<128>(a, stream);
    const cudaError_t e = launch_select<0>(a, stream);
    if (e != cudaSuccess) return e;
    const int rows = (256 / (a.d / 8)) * kMoveRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.keep + rows - 1) / rows, a.H_kv, a.B);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return a.d == 64 ? cudaLaunchKernelEx(&cfg, fa_paged_move_kernel<64>, a)
                     : cudaLaunchKernelEx(&cfg, fa_paged_move_kernel<128>, a);
}

// New lengths that replace kv_len itself: every CTA that selects or moves reads
// kv_len, so they are written when the last of these has ended.
__global__ void __launch_bounds__(256) fa_paged_len_kernel(const PagedEvictArgs a) {
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b < a.B) a.new_len[b] = evict_len(a, b);
}

cudaError_t launch_paged_evict(const PagedEvictArgs &a, int sm_count, cudaStream_t stream) {
    const cudaError_t e = launch_evict_rows(a, sm_count, stream);
    if (e != cudaSuccess || a.new_len != a.kv_len) return e;
    fa_paged_len_kernel<<<(a.B + 255) / 256, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace fa
