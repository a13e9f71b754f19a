// fa_paged_share.cuh -- how the attention over a paged cache is dealt to the
// CTAs: units, their steps, every CTA's equal share of all steps, and the
// pieces that a share consists of.
//
// A unit is U positions of the new tokens of one (sequence, K/V head); its
// steps are the 128-key tiles that any of its rows sees, from the last to the
// first, the sliding window's first and then those of the first tokens.
// Lengths are known on the device only: every CTA adds up the cost of all
// units (a scan over the sequences by all its threads), takes the share
// [c Q, (c + 1) Q) of it, Q = ceil(total / CTAs), and walks it.  A unit costs its
// steps and, in front of them, kCost for its beginning and end, when the pipeline
// fills and drains (3 for chunks: 89 -> 85 us for 24 sequences of 1 to 300 new
// tokens; 1 for few rows: 184 -> 181 us for 64 single tokens; more is worse).
// Whole units are written to O; of a unit that a share's border cuts, each
// part leaves its normalised O and LSE in the workspace (at most two parts a
// CTA) and fa_paged_combine_kernel joins them in order.
#pragma once

#include "fa_paged.cuh"

namespace fa {

// One piece of a share, as posted in the ring.
struct __align__(16) PagedPiece {
    int qrow;           // packed row of tile L's first position; -1: no more pieces
    int nl, nh;         // positions in tiles L and H (nh = 0: one tile)
    int pos;            // cache position of tile L's first position
    int n, b, h;        // cached tokens, sequence, K/V head
    int hi, nw, T;      // one past the last key tile, steps in the window, all steps
    int t0, t1;         // this piece's steps
    int skip;           // steps that tile L does not see
    int slot;           // part in the workspace, or -1: the whole unit
    int vlo, vhi;       // keys of the window that any row sees
};
static_assert(sizeof(PagedPiece) == 64, "piece ring");

// The key tile of step t.
__device__ __forceinline__ int paged_tile(const PagedPiece &p, int t) {
    return t < p.nw ? p.hi - 1 - t : (p.T - 1) - t;
}

// Key tiles that rows at positions pa .. pb (of n cached tokens) see.
struct PagedTiles { int hi, nw, T; };
__device__ __forceinline__ PagedTiles paged_tiles(int pa, int pb, int n, int wl, int wr, int first) {
    const int khi = paged_hi(pb, n, wr);
    PagedTiles t;
    t.hi = (khi >> 7) + ((khi & 127) != 0);
    const int lo = min(paged_lo(pa, wl) >> 7, t.hi);
    const int f = min(first, khi);
    t.nw = t.hi - lo;
    t.T = max(1, t.nw + min((f >> 7) + ((f & 127) != 0), lo));   // an empty unit still writes O = 0
    return t;
}
// Cost of unit p of a sequence (U positions a unit).  Not inlined: the code
// before a CTA's first load comes from L2, line by line.
template <int kCost>
static __device__ __noinline__ int paged_unit_cost(int m, int n, int p, int U, int wl, int wr, int first) {
    const int i0 = p * U;
    return kCost + paged_tiles(n - m + i0, n - m + min(m, i0 + U) - 1, n, wl, wr, first).T;
}
__device__ __forceinline__ int paged_units(const PagedSeq &s, int U) {
    return static_cast<int>((static_cast<long long>(s.m) + U - 1) / U);
}
// Cost of all units of a sequence, by the whole warp.
template <int kCost>
__device__ __forceinline__ long long paged_seq_cost_warp(const PagedSeq &s, int U, const PagedArgs &a) {
    const int np = paged_units(s, U);
    long long sum = 0;
    for (int p = threadIdx.x & 31; p < np; p += 32) sum += paged_unit_cost<kCost>(s.m, s.n, p, U, a.wl, a.wr, a.first);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// A CTA's share [w0, w1) of the whole cost, in units of `quota`; its first unit
// belongs to sequence b or one behind it, whose units start at `at`.
struct PagedShare {
    long long w0, w1, quota, at, per;   // per: cost of one K/V head of sequence b
    int b;
    PagedSeq s;                         // sequence b
};

// Bytes of shared-memory scratch for paged_share.
constexpr uint32_t kShareScratch = 16 * 8 + 48;

// By the whole block (kThreads of them); ends with a barrier after which the
// scratch is free.
template <int kThreads, int kCost>
__device__ __forceinline__ PagedShare paged_share(const PagedArgs &a, int U, uint8_t *scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long *scan = reinterpret_cast<long long *>(scratch);          // [16]
    long long *found = scan + 16;                                      // at, per
    int *found_i = reinterpret_cast<int *>(found + 2);                 // b, q0, m, n
    // thread i owns sequences [i k, (i + 1) k)
    const int k = (a.B + kThreads - 1) / kThreads;
    long long mine = 0, per0 = 0;
    PagedSeq s0{0, 0, 0, false};
    for (int i = 0; i < k; ++i) {
        const int b = tid * k + i;
        PagedSeq s{0, 0, 0, false};
        if (b < a.B) s = paged_seq(a.cu_q, a.kv_len, b, a.T, a.W, a.ps_log2);
        if (s.bad && blockIdx.x == 0) report_bad_index(a.status, 1);
        const int np = paged_units(s, U);
        // a few units by the thread itself, many by its warp
        if (np <= 8)
            for (int p = 0; p < np; ++p) mine += paged_unit_cost<kCost>(s.m, s.n, p, U, a.wl, a.wr, a.first);
        for (unsigned big = __ballot_sync(0xffffffffu, np > 8); big != 0; big &= big - 1) {
            const int src = __ffs(big) - 1;
            PagedSeq t{0, __shfl_sync(0xffffffffu, s.m, src), __shfl_sync(0xffffffffu, s.n, src), false};
            const long long sum = paged_seq_cost_warp<kCost>(t, U, a);
            if (lane == src) mine += sum;
        }
        if (i == 0) { s0 = s; per0 = mine; }
    }
    mine *= a.H_kv;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long sums = lane < kThreads / 32 ? scan[lane] : 0;            // (every warp scans the warps' sums)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += v;
    }
    const long long total = __shfl_sync(0xffffffffu, sums, 31);
    const long long before = __shfl_sync(0xffffffffu, sums, warp == 0 ? 31 : warp - 1) - (warp == 0 ? total : 0);
    PagedShare sh;
    const unsigned G = gridDim.x;
    sh.quota = (total >> 31) == 0 ? static_cast<long long>((static_cast<unsigned>(total) + G - 1) / G)
                                  : (total + G - 1) / G;
    sh.w0 = blockIdx.x * sh.quota;
    sh.w1 = min(total, sh.w0 + sh.quota);
    const long long start = before + incl - mine;
    if (sh.w0 < sh.w1 && start <= sh.w0 && sh.w0 < start + mine) {
        found[0] = start;
        found[1] = per0;
        found_i[0] = tid * k;
        found_i[1] = s0.q0;
        found_i[2] = s0.m;
        found_i[3] = s0.n;
    }
    fence_proxy_async_smem();                              // the scratch may be TMA's next
    __syncthreads();
    sh.at = found[0];
    sh.per = found[1];
    sh.b = found_i[0];
    sh.s = PagedSeq{found_i[1], found_i[2], found_i[3], false};
    __syncthreads();
    return sh;
}

// The scheduler warp: the pieces of a share, in order, to post(piece) -> bool.
// kPair: units of two Q tiles of R positions (U = 2 R), otherwise of one.
// desc: this CTA's descriptor in the workspace.
template <bool kPair, int kCost, class Post>
__device__ __forceinline__ bool paged_walk(const PagedShare &sh, const PagedArgs &a, int R, int *desc, Post &&post) {
    const int lane = threadIdx.x & 31, U = kPair ? 2 * R : R;
    const long long w0 = sh.w0, w1 = sh.w1;
    if (lane == 0) desc[0] = 0;
    bool ok = true;
    if (w0 < w1) {
        int b = sh.b;
        long long at = sh.at, per = sh.per;            // cost before sequence b; of one K/V head
        PagedSeq s = sh.s;
        while (w0 >= at + per * a.H_kv && b + 1 < a.B) {
            at += per * a.H_kv;
            s = paged_seq(a.cu_q, a.kv_len, ++b, a.T, a.W, a.ps_log2);
            per = paged_seq_cost_warp<kCost>(s, U, a);
        }
        int h = 0;
        long long rem = w0 - at;                       // how far into this head's units
        if (rem >= per) {
            h = (rem >> 31) == 0 ? static_cast<unsigned>(rem) / static_cast<unsigned>(per)
                                 : static_cast<int>(rem / per);
            rem -= h * per;
        }
        int np = paged_units(s, U), p = 0;
        for (int p0 = 0; np > 1 && p0 < np; p0 += 32) {
            const long long mine_t =
                p0 + lane < np ? paged_unit_cost<kCost>(s.m, s.n, p0 + lane, U, a.wl, a.wr, a.first) : 0;
            long long inc = mine_t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, inc > rem);
            if (past != 0) {
                const int l = __ffs(past) - 1;
                p = p0 + l;
                rem -= __shfl_sync(0xffffffffu, inc - mine_t, l);
                break;
            }
            rem -= __shfl_sync(0xffffffffu, inc, 31);
        }
        int v0 = static_cast<int>(rem);                // where the share starts within the unit
        for (long long at_w = w0; ok && at_w < w1;) {
            PagedPiece pc;
            const int i0 = p * U, left = s.m - i0;
            pc.qrow = s.q0 + i0;
            pc.nl = min(left, R);
            pc.nh = kPair ? min(max(left - R, 0), R) : 0;
            pc.pos = s.n - s.m + i0;
            pc.n = s.n;
            pc.b = b;
            pc.h = h;
            const int last = pc.pos + pc.nl + pc.nh - 1;
            const PagedTiles tl = paged_tiles(pc.pos, last, s.n, a.wl, a.wr, a.first);
            pc.hi = tl.hi;
            pc.nw = tl.nw;
            pc.T = tl.T;
            pc.vlo = paged_lo(pc.pos, a.wl);
            pc.vhi = paged_hi(last, s.n, a.wr);
            const int khl = paged_hi(pc.pos + pc.nl - 1, s.n, a.wr);
            pc.skip = min(tl.T - 1, max(0, min(tl.nw, tl.hi - ((khl >> 7) + ((khl & 127) != 0)))));
            const int v1 = static_cast<int>(min(static_cast<long long>(tl.T) + kCost, v0 + (w1 - at_w)));
            pc.t0 = max(v0 - kCost, 0);
            pc.t1 = max(v1 - kCost, 0);
            const bool cont = pc.t1 < tl.T;
            pc.slot = pc.t0 > 0 ? 2 * static_cast<int>(blockIdx.x) : cont ? 2 * static_cast<int>(blockIdx.x) + 1 : -1;
            if (pc.t0 == 0 && pc.t1 > 0 && cont && lane == 0) {        // a cut unit that starts here
                desc[1] = pc.qrow;
                desc[2] = pc.nl;
                desc[3] = pc.nh;
                desc[4] = h;
                desc[0] = 1 + static_cast<int>((at_w - v0 + kCost + tl.T - 1) / sh.quota - blockIdx.x);   // its parts
            }
            if (pc.t1 > pc.t0) ok = post(pc);
            at_w += v1 - v0;
            v0 = 0;
            if (++p == np) {
                p = 0;
                if (++h == a.H_kv) {
                    h = 0;
                    do {
                        if (++b >= a.B) break;
                        s = paged_seq(a.cu_q, a.kv_len, b, a.T, a.W, a.ps_log2);
                        np = paged_units(s, U);
                    } while (np == 0);
                    if (b >= a.B) break;
                }
            }
        }
    }
    return ok;
}

// A TMA producer (whole warp), one of two.  The lanes of a warp issue their
// boxes one after the other, ~55 cycles each: with 16-token pages a K/V tile
// pair is 64 of them, which one warp could not issue in the time that HBM takes
// for the pair (2 x 32 KB: ~2900 cycles; 202 -> 172 us for 64 sequences of 4096
// at d = 128).
//   C::kByStep = false: warp 0 loads the Q tiles and K (even slots of the
//     ring), warp 1 V (odd slots).
//   C::kByStep: warp w loads K and V of the steps w, w + 2, ... of a piece into
//     a ring of its own (slots w * NRING ...), warp 0 the Q tiles.
// Whatever waits for a slot sees every phase of its barrier: a parity says only
// whether the last phase is complete, so a waiter that skipped one would pass
// a phase early.
template <class C, class Take>
__device__ __forceinline__ void paged_produce(const int wp, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                              const CUtensorMap &tm_v, const PagedArgs &a, const int R,
                                              const uint32_t base, Take &&take, const WaitCtx w) {
    const int lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return base + C::BAR_OFF + 8u * i; };
    constexpr int kStride = C::kByStep ? 2 : 1;        // between this warp's steps
    const uint32_t slot0 = C::kByStep ? wp * C::NRING : wp, slot1 = C::kByStep ? slot0 + C::NRING : C::NSTAGE;
    uint32_t qc = 0, pi = 0, slot = slot0, ph = 0;     // Q tiles, pieces; ring slot and its phase
    uint32_t qarmed = 0, qarmed_par = 0, armed = 0, armed_par = 0;
    bool ok = true;
    const PagedBox<C::NCH> bx(a.ps_log2);
    const uint32_t q_bytes = static_cast<uint32_t>(a.group * R) * 128u * C::NCH;
    // The page ids of a step are read PF steps ahead, and a piece's first
    // ones while the piece before it still loads: an id comes from L2 or
    // HBM, and a step may not wait for that.
    constexpr int PF = 4;
    auto page_of = [&](const PagedPiece &p, int t) __attribute__((always_inline)) -> int {
        if (t >= p.t1) return a.n_pages;
        const int j = paged_tile(p, t);
        return bx.needs(j, p.vlo, p.vhi, min(a.first, p.vhi))
                   ? a.table[static_cast<long long>(p.b) * a.W + ((j * 128 + bx.row) >> a.ps_log2)]
                   : a.n_pages;
    };
    const int skip = C::kByStep ? wp : 0;              // this warp's first step of a piece
    PagedPiece p, nx;
    int page[PF], page_n[PF];
    bool more = take(pi++, w, 31, p), more_n = false;
#pragma unroll
    for (int u = 0; u < PF; ++u) page[u] = more ? page_of(p, p.t0 + skip + u * kStride) : 0;
    while (ok && more) {
        for (int x = wp == 0 ? 0 : 2; x < (p.nh > 0 ? 2 : 1) && ok; ++x) {
            const uint32_t qs = qc % C::NQ, qph = (qc / C::NQ) & 1u;
            ok = mbar_wait_warp(bar(C::B_QEMPTY + qs), qph ^ 1u, w, 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(C::B_QFULL + qs), q_bytes);
            __syncwarp();
            if (lane < C::NCH)
                tma_load_4d(&tm_q, base + C::Q_OFF + qs * C::Q_BYTES + lane * C::Q_CHUNK,
                            bar(C::B_QFULL + qs), lane * 64, p.h * a.group, p.qrow + x * R, 0);
            qarmed |= 1u << qs;
            qarmed_par = (qarmed_par & ~(1u << qs)) | (qph << qs);
            ++qc;
        }
        bool ahead = false;                            // nx is taken
        auto look_ahead = [&]() __attribute__((always_inline)) {
            ahead = true;
            more_n = take(pi++, w, 31, nx);
#pragma unroll
            for (int u = 0; u < PF; ++u) page_n[u] = more_n ? page_of(nx, nx.t0 + skip + u * kStride) : 0;
        };
#pragma unroll 1
        for (int t = p.t0 + skip; t < p.t1 && ok; t += kStride) {
            const int j = paged_tile(p, t);
            int pg = page[0];
#pragma unroll
            for (int u = 0; u + 1 < PF; ++u) page[u] = page[u + 1];
            page[PF - 1] = page_of(p, t + PF * kStride);
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.n_pages)) {
                if (bx.needs(j, p.vlo, p.vhi, min(a.first, p.vhi))) report_bad_index(a.status, 2);
                pg = a.n_pages;                        // beyond the pool: zeros
            }
            const int row0 = (j * 128 + bx.row) & ((1 << a.ps_log2) - 1);
            const CUtensorMap *tm = C::kByStep || wp == 0 ? &tm_k : &tm_v;
#pragma unroll 1
            for (int v = 0; v < kStride; ++v, tm = &tm_v) {
                ok = mbar_wait_warp(bar(C::B_KVEMPTY + slot), ph ^ 1u, w, 2);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::B_KVFULL + slot), C::TILE_BYTES);
                __syncwarp();
                if (lane < bx.n_box)
                    tma_load_4d(tm, base + C::KV_OFF + slot * C::TILE_BYTES + bx.c * C::CHUNK_BYTES + bx.row * 128u,
                                bar(C::B_KVFULL + slot), bx.c * 64, p.h, row0, pg);
                armed |= 1u << slot;
                armed_par = (armed_par & ~(1u << slot)) | (ph << slot);
                slot += C::kByStep ? 1 : 2;
                if (slot >= slot1) { slot = slot0; ph ^= 1u; }
            }
            if (ok && !ahead) look_ahead();
        }
        if (ok && !ahead) look_ahead();
        p = nx;
        more = more_n;
#pragma unroll
        for (int u = 0; u < PF; ++u) page[u] = page_n[u];
    }
    // Every issued copy lands before the CTA may end (bounded).
    for (int s = 0; s < C::NSTAGE; ++s)
        if (armed & (1u << s)) mbar_wait_quiet(bar(C::B_KVFULL + s), (armed_par >> s) & 1u, 500000000ull);
    for (int q = 0; q < C::NQ; ++q)
        if (qarmed & (1u << q)) mbar_wait_quiet(bar(C::B_QFULL + q), (qarmed_par >> q) & 1u, 500000000ull);
    __syncwarp();
}

}  // namespace fa
