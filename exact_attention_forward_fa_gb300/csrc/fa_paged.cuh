// fa_paged.cuh -- the paged key/value cache: its argument record, the
// geometry of a sequence in it and the checks of what only the device can
// see (lengths, row offsets, page ids).
//
// K and V of all sequences lie in two pools of pages, [n_pages][page_size]
// [H_kv][d]; token p of sequence b is slot p % page_size of page
// table[b][p / page_size].  The new tokens of the call are rows cu_q[b] ..
// cu_q[b + 1] of the packed tensors; they are the last of the sequence's
// kv_len[b] cached tokens, so row cu_q[b] + i has position
// kv_len[b] - (cu_q[b + 1] - cu_q[b]) + i.
//
// Visible keys of the row at position p (the bottom-right diagonal of more keys
// than queries): j < kv_len, j <= p + wr (wr >= 0), and j >= p - wl (wl >= 0) or
// j < first -- a sliding window beside which the first tokens stay visible.
#pragma once

#include <cuda_runtime.h>

#include "fa_device.cuh"

namespace fa {

constexpr uint32_t kStatusBadIndex = 2;
constexpr uint32_t kRolePaged = 8;

struct PagedArgs {
    const void *q;                 // [T][H][d], q_stride elements between tokens
    const void *k_pages, *v_pages; // pools, page_stride elements between pages
    const int *table;              // [B][W]
    const int *kv_len;             // [B]
    const int *cu_q;               // [B + 1]
    void *o;                       // [T][H][d]
    float *lse;                    // [H][T] or nullptr
    uint32_t *status;
    long long q_stride, page_stride;
    int B, H, H_kv, group, T, W;
    int ps_log2, n_pages;
    int wl, wr, first;
    float scale_log2;              // alpha * log2(e)
};

// Records an index out of range (the access itself is skipped).
__device__ __forceinline__ void report_bad_index(uint32_t *status, uint32_t where) {
    if (atomicCAS(&status[0], kStatusOk, kStatusBadIndex) == kStatusOk) {
        status[1] = kRolePaged;
        status[2] = where;
        status[3] = blockIdx.x;
    }
}

// mbar_wait_warp for a warp whose answer is not urgent: it sleeps between its
// polls.  A polling warp takes issue slots and shared-memory bandwidth from
// the warps that work.
__device__ __forceinline__ bool mbar_wait_idle(uint32_t bar, uint32_t parity, const WaitCtx &w,
                                               uint32_t where) {
    bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
    const uint64_t t0 = globaltimer_ns();
    while (!ok) {
        __nanosleep(100);
        ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
        if (ok) break;
        const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
        if (late) report_timeout(w.abort_flag, w.status, w.role, where);
        if (__any_sync(0xffffffffu, late || *w.abort_flag != 0u)) return false;   // all lanes together
    }
    return true;
}

// Sequence b: its first packed row, its new tokens and its cached tokens,
// forced into the ranges that the buffers have; `bad` tells whether they
// were outside.
struct PagedSeq {
    int q0, m, n;
    bool bad;
};
__device__ __forceinline__ PagedSeq paged_seq(const int *cu_q, const int *kv_len, int b, int T,
                                              int W, int ps_log2) {
    const int c0 = cu_q[b], c1 = cu_q[b + 1], n0 = kv_len[b];
    const long long cap = static_cast<long long>(W) << ps_log2;
    PagedSeq s;
    s.q0 = min(max(c0, 0), T);
    s.m = min(max(c1, s.q0), T) - s.q0;
    s.n = n0 < 0 ? 0 : static_cast<int>(n0 < cap ? n0 : cap);
    s.bad = s.q0 != c0 || s.q0 + s.m != c1 || s.n != n0;
    return s;
}

// Reports sequences whose offsets or lengths are out of range; a whole block
// of a launch that otherwise looks sequences up row by row.
__device__ __forceinline__ void paged_check_seqs(const int *cu_q, const int *kv_len, int B, int T,
                                                 int W, int ps_log2, uint32_t *status) {
    for (int b = threadIdx.x; b < B; b += blockDim.x)
        if (paged_seq(cu_q, kv_len, b, T, W, ps_log2).bad) report_bad_index(status, 1);
}

// Visible keys of position p among n: [lo, hi) and [0, min(first, hi)).
// 64-bit sums: any window value is allowed.
__device__ __forceinline__ int paged_lo(int p, int wl) {
    const long long lo = wl >= 0 ? static_cast<long long>(p) - wl : 0;
    return lo > 0 ? static_cast<int>(lo) : 0;
}
__device__ __forceinline__ int paged_hi(int p, int n, int wr) {
    const long long hi = wr >= 0 ? static_cast<long long>(p) + wr + 1 : n;
    return hi < 0 ? 0 : hi < n ? static_cast<int>(hi) : n;
}

// A lane's part of a 128-token tile: TMA boxes of min(page_size, 128) slots by
// one 128-byte column chunk, kChunks chunks a row; lanes at and behind n_box
// have none.  row: the box's first token in the tile, c: its chunk.
template <int kChunks>
struct PagedBox {
    int box, n_box, row, c;
    __device__ __forceinline__ explicit PagedBox(int ps_log2) {
        const int lane = threadIdx.x & 31;
        box = min(1 << ps_log2, 128);
        n_box = (128 / box) * kChunks;
        row = (lane / kChunks) * box;
        c = lane % kChunks;
    }
    // Whether this lane has a box of tile j that holds tokens which a row sees,
    // [vlo, vhi) or [0, nf).  (Others are loaded from page n_pages: TMA gives zeros.)
    __device__ __forceinline__ bool needs(int j, int vlo, int vhi, int nf) const {
        const int tok = j * 128 + row;
        return (threadIdx.x & 31) < n_box && ((tok < vhi && tok + box > vlo) || tok < nf);
    }
};

// The page that holds token j of sequence b, or -1 (reported) for an id
// outside the pool.
__device__ __forceinline__ int paged_page(const int *table_b, int j, int ps_log2, int n_pages,
                                          uint32_t *status) {
    const int p = table_b[j >> ps_log2];
    if (static_cast<unsigned>(p) < static_cast<unsigned>(n_pages)) return p;
    report_bad_index(status, 2);
    return -1;
}

// The sequence of packed row t, by a 32-way search over cu_q (whole warp;
// t is the same in every lane): the last b in [0, B) with cu_q[b] <= t, or
// -1 when row t lies behind cu_q[B] (or before cu_q[0]).
__device__ __forceinline__ int paged_find_seq(const int *cu_q, int B, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, cnt = B + 1;                     // candidates cu_q[lo .. lo + cnt)
    if (cnt <= 0) return -1;
    while (cnt > 1) {
        const int step = (cnt + 31) / 32;
        const int i = lane * step;
        const bool le = i < cnt && cu_q[lo + i] <= t;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        if (m == 0) return -1;
        const int last = 31 - __clz(m);
        lo += last * step;
        cnt = min(step, cnt - last * step);
    }
    return (lo < B && cu_q[lo] <= t) ? lo : -1;
}

struct PagedAppendArgs {
    const void *k, *v;             // [T][H_kv][d], kv_stride elements between tokens
    void *k_pages, *v_pages;
    const int *table, *kv_len, *cu_q;
    uint32_t *status;
    long long kv_stride, page_stride;
    int B, T, W, ps_log2, n_pages;
    int row_vecs;                  // 16-byte vectors of one token, H_kv * d / 8
};
cudaError_t launch_paged_append(const PagedAppendArgs &a, cudaStream_t stream);

// What a unit costs beside its steps, in steps (fa_paged_share.cuh): in the kernel
// for few rows and in the one for chunks.
constexpr int kFewRows = 8, kUnitCostFew = 1, kUnitCostChunk = 3;

// The workspace of the attention: what the parts of cut units leave.
struct PagedWork {
    int *desc;          // [CTAs][8]: the cut unit that starts in a CTA's share
    float *lse;         // [2 * CTAs][2][128], log2 units
    float *o;           // [2 * CTAs][2][128][d], normalised
};
struct PagedFwdLaunch {
    CUtensorMap q;      // {d, H, T, 1}, box {64, group, R, 1}, 128-byte swizzle
    CUtensorMap k, v;   // {d, H_kv, page_size, n_pages}, box {64, 1, min(page_size, 128), 1}
    PagedArgs a;
    PagedWork w;
    int R;              // positions per Q tile
    int grid, d;
    bool bf16;
    cudaStream_t stream;
};
cudaError_t launch_fwd_paged_d64(const PagedFwdLaunch &L);
cudaError_t launch_fwd_paged_d128(const PagedFwdLaunch &L);

struct PagedScoresLaunch {
    CUtensorMap q, k;   // as in PagedFwdLaunch
    PagedArgs a;        // lse: read here
    const float *in;    // [B][H_kv][L] or nullptr
    float *out;         // [B][H_kv][L]
    int L;
    int R, grid, d;
    bool bf16;
    cudaStream_t stream;
};
cudaError_t launch_paged_scores(const PagedScoresLaunch &L);

struct PagedEvictArgs {
    void *k_pages, *v_pages;
    const float *scores;           // [B][H_kv][L]
    const int *table, *kv_len, *dst_table;
    int *kept;                     // [B][H_kv][keep]
    float *scores_out;             // [B][H_kv][keep] or nullptr
    int *new_len;                  // [B]
    uint32_t *status;
    long long page_stride;
    int B, H_kv, d, W, dst_W, ps_log2, n_pages, L;
    int keep, first, recent;
};
cudaError_t launch_paged_evict(const PagedEvictArgs &a, int sm_count, cudaStream_t stream);

}  // namespace fa
