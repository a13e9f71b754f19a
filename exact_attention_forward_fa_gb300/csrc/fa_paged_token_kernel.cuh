// fa_paged_token_kernel.cuh -- attention over a paged cache for few rows
// (single tokens, drafts of two or three: at most 8 rows of R positions x g heads),
// on sm_103a.
//
// Such a call reads each K and V tile for a handful of rows: it is bound by
// HBM, 4 d bytes a key against 4 d g flops, and what counts is that no step's
// latency keeps loads from being issued.  Both products are formed transposed:
//     S^T = K Q^T   (128 keys x N rows; a TMEM lane, and a thread, is a key)
//     O^T = V^T P^T (d x N; a lane is an output column)
// so a tile of 128 keys has work for all 128 threads of a group -- an
// exponential a row each -- and the tensor core's N is 16 instead of 128.  (With rows as lanes one warp of four
// held all rows: 2000 cycles a step and group, 54 us for 32 caches of 32768 at
// d = 64 where HBM takes 39.)  P^T goes through shared memory, written in the
// swizzled layout that the product reads.
//
// Softmax.  A group keeps a reference r for each row (log2 units, in shared
// memory) and P = 2^(x - r).  r comes from the first tile that the row sees and
// moves only when a score exceeds it by more than 15 (P stays within fp16); a vote of
// the group's threads finds that out, and only then are maxima taken and O
// rescaled.  A thread sums the exponentials of its own keys; threads are added
// up once, at the end of a piece.  P is rounded to the 16-bit type, the operand that
// the tensor core takes at its full rate; O is normalised by the sum of the rounded
// terms, LSE is that of the FP32 ones.  O is then off by 0.0023 relative (bf16) and
// 0.0003 (fp16) where rounding O alone gives 0.0017 and 0.0002.
//
// Two groups of four warps take a piece's steps in turn, each with its own S^T
// (double-buffered), P^T, O^T and ring of K and V tiles; warps 8 and 9 load the
// rings, warps 10 and 11 issue the products, warp 12 walks the share
// (fa_paged_share.cuh).  At the end
// of a piece group 0 joins the two halves and writes O, or the part of a cut
// unit.
//
// Measured (32 heads over 8, d = 128, bf16): 64 sequences of up to 8192 tokens
// 180.5 us, 6.3 TB/s; two of 115831 and 125872 154 us, 6.4 TB/s; one of 777 11.5 us, all of it
// latency (launch, shares, first tiles, joining kernel).  d = 64, a K/V head for
// each of 16 heads, 1 to 4 new tokens, 32 caches of which the last 2047 and the first 4 are
// seen: 60 us, 4.5 TB/s: its steps pass at 1600 to 1700 cycles an SM, where HBM needs
// 1400 to 1500 for their 32 KB; the rest is the start, the joining kernel and, in every
// unit of 18 steps, one for the four first tokens.  The bytes in flight (192 KB an SM) cover HBM's latency; what is
// left of the longer ones are the ~6 us at the start and the ~4 us of the joining
// kernel.
//
// Waits are bounded, and a warp whose wait gave up keeps taking part in its
// group's barriers until a vote makes the whole group leave.
#pragma once

#include "fa_paged_share.cuh"

namespace fa {

template <int D, bool kBF16>
struct TokenCfg {
    static constexpr int NCH = D / 64;                    // 128-byte column chunks
    static constexpr uint32_t CHUNK_BYTES = 128u * 128u;
    static constexpr uint32_t TILE_BYTES = NCH * CHUNK_BYTES;
    // (32 rows of Q and P where the products read 16: what lies behind the K/V
    // tiles has to be as long as one of their chunks, see MMA_END)
    static constexpr uint32_t Q_CHUNK = 32u * 128u, Q_BYTES = NCH * Q_CHUNK;
    static constexpr uint32_t P_CHUNK = 32u * 128u, P_BYTES = 2 * P_CHUNK;   // [32 rows][128 keys]
    static constexpr int NSTAGE = D == 64 ? 12 : 6;
    static constexpr int NRING = NSTAGE / 2;              // slots of a group's ring: K and V of its steps in turn
    static constexpr bool kByStep = true;
    static constexpr int NQ = 2;
    static constexpr int NTHREADS = 416;
    static constexpr int RING = 2;
    static constexpr uint32_t KV_OFF = 0;
    static constexpr uint32_t Q_OFF = NSTAGE * TILE_BYTES;
    static constexpr uint32_t P_OFF = Q_OFF + NQ * Q_BYTES;
    static constexpr uint32_t R_OFF = P_OFF + 2 * P_BYTES;            // [2 groups][32] references (8 used)
    static constexpr uint32_t X_OFF = R_OFF + 2 * 32 * 4;             // group 1's LSE and 1 / l, the factors: [4][32]
    static constexpr uint32_t RED_OFF = X_OFF + 4 * 32 * 4;           // sums: [2 groups][2][4 warps][8]
    static constexpr uint32_t RING_OFF = RED_OFF + 2 * 64 * 4;
    static constexpr uint32_t BAR_OFF = RING_OFF + RING * 64;
    static constexpr int B_QFULL = 0, B_QEMPTY = NQ, B_KVFULL = 2 * NQ, B_KVEMPTY = B_KVFULL + NSTAGE,
                         B_SFULL = B_KVEMPTY + NSTAGE, B_SEMPTY = B_SFULL + 4, B_PFULL = B_SEMPTY + 4,
                         B_PEMPTY = B_PFULL + 2, B_OFULL = B_PEMPTY + 2, B_OEMPTY = B_OFULL + 2,
                         B_XFULL = B_OEMPTY + 2, B_XEMPTY = B_XFULL + 1, B_DONE = B_XEMPTY + 1,
                         B_PIECE = B_DONE + 2, B_FREE = B_PIECE + RING, NBAR = B_FREE + RING;
    // Arrivals that complete a phase: a group's four warps; both groups' last
    // product with a Q tile; producers, MMA issuers and the groups' warps.
    __device__ static uint32_t arrivals(int i) {
        return (i >= B_SEMPTY && i < B_PEMPTY) || i == B_OEMPTY || i == B_OEMPTY + 1 ? 4u
               : i >= B_QEMPTY && i < B_KVFULL ? 2u : i >= B_FREE ? 12u : 1u;
    }
    static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr uint32_t SMEM_BYTES = MISC_OFF + 16 + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
    // O^T's product has 128 rows, at d = 64 too: with the last V tile as A it reads
    // one chunk past the tiles, which must not lie outside shared memory.
    static constexpr uint32_t MMA_END = KV_OFF + (NSTAGE - 1) * TILE_BYTES + 2 * CHUNK_BYTES;
    static_assert(MMA_END <= MISC_OFF, "the last V tile's product stays in shared memory");
    static constexpr uint32_t TMEM_COLS = 256;
    __host__ __device__ static constexpr uint32_t col_s(int x, int buf) { return 64u * x + 32u * buf; }
    __host__ __device__ static constexpr uint32_t col_o(int x) { return 128u + 32u * x; }
    static constexpr float TAU = 8.0f;                    // a reference moves when its row's maximum grew by more
    static constexpr float CAP = 15.0f;                   // and has to when a P would pass 2^15
};

// TMEM: eight 32-bit columns of the warp's lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Adds (or takes the maximum of) v[n] over the 32 lanes of a warp, for every n:
// lane l gets that of v[l % kN].  9 exchanges for 8 values instead of 40.
template <int kN, bool kMax = false>
__device__ __forceinline__ float warp_reduce_transposed(float (&v)[kN]) {
    const int lane = threadIdx.x & 31;
    auto both = [](float x, float y) { return kMax ? fmaxf(x, y) : x + y; };
#pragma unroll
    for (int w = kN / 2; w > 0; w >>= 1) {
        const bool up = (lane & w) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = up ? v[i] : v[i + w];
            const float mine = up ? v[i + w] : v[i];
            v[i] = both(mine, __shfl_xor_sync(0xffffffffu, send, w));
        }
    }
#pragma unroll
    for (int w = kN; w < 32; w <<= 1) v[0] = both(v[0], __shfl_xor_sync(0xffffffffu, v[0], w));
    return v[0];
}

// Barrier of group x's 128 threads that tells whether any of them says so.
__device__ __forceinline__ bool group_any(int x, bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(v ? 1u : 0u), "r"(1 + x) : "memory");
    return r != 0;
}

// More rows are the chunk kernel's (fa_paged_launch.cuh): an instantiation of this
// one for 32 took 370 us for 64 sequences of four tokens on up to 8192 (16 rows) and
// 535 of eight (32 rows), where the chunk kernel takes 190, and 22 to 26 us for
// one sequence of 777 against 14: a thread's unrolled work on 32 rows, most of
// it at the beginning and end of a piece, comes from L2 each time.
template <int D, bool kBF16>
__global__ void __launch_bounds__(416, 1)
fa_paged_token_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const PagedArgs a, const PagedWork wk,
                      const int R) {
    using C = TokenCfg<D, kBF16>;
    constexpr int kN = kFewRows;                          // rows that the groups work on
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return base + C::BAR_OFF + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gbase + C::MISC_OFF);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + C::MISC_OFF + 4);
    PagedPiece *ring = reinterpret_cast<PagedPiece *>(gbase + C::RING_OFF);

    if (warp == 10) tmem_alloc(base + C::MISC_OFF, C::TMEM_COLS);
    if (tid == 0) *abort_flag = 0u;
    if (warp == 11) {
        for (int i = lane; i < C::NBAR; i += 32) mbar_init(bar(i), C::arrivals(i));
        fence_barrier_init();
    }
    if (tid == 8 * 32) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    tc_fence_before();
    const PagedShare share = paged_share<C::NTHREADS, kUnitCostFew>(a, R, gbase + C::KV_OFF);
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    auto take = [&](uint32_t i, const WaitCtx &w, uint32_t where, PagedPiece &p) __attribute__((always_inline)) -> bool {
        const uint32_t q = i % C::RING;
        if (!mbar_wait_warp(bar(C::B_PIECE + q), (i / C::RING) & 1u, w, where)) return false;
        p = ring[q];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_FREE + q));
        return p.qrow >= 0;
    };

    if (warp == 12) {
        // =================== scheduler (whole warp) ===================
        WaitCtx w{abort_flag, a.status, kRolePaged};
        uint32_t sent = 0;
        auto post = [&](const PagedPiece &p) __attribute__((always_inline)) -> bool {
            const uint32_t q = sent % C::RING;
            if (!mbar_wait_idle(bar(C::B_FREE + q), ((sent / C::RING) & 1u) ^ 1u, w, 30))
                return false;
            if (lane == 0) {
                ring[q] = p;
                mbar_arrive(bar(C::B_PIECE + q));
            }
            __syncwarp();
            ++sent;
            return true;
        };
        if (paged_walk<false, kUnitCostFew>(share, a, R, wk.desc + 8 * blockIdx.x, post)) {
            PagedPiece end{};
            end.qrow = -1;
            post(end);
        }
    } else if (warp == 8 || warp == 9) {
        paged_produce<C>(warp - 8, tm_q, tm_k, tm_v, a, R, base, take,
                         WaitCtx{abort_flag, a.status, kRoleProducer});
    } else if (warp >= 10) {
        // =================== MMA issuer of group x (whole warp) ===================
        // Step i of group x: S^T into its next buffer as soon as K is there,
        // a step ahead of O^T += V^T P^T.
        WaitCtx w{abort_flag, a.status, kRoleMma};
        const int x = __shfl_sync(0xffffffffu, warp - 10, 0);
        constexpr uint32_t idesc_s = idesc_f16(128, 16, kBF16, false, false);
        constexpr uint32_t idesc_o = idesc_f16(128, 16, kBF16, true, false);
        uint32_t kc = 0, vc = 1;                           // this group's next K and V tile, counted together
        uint32_t pc = 0, sc = 0, un = 0, pp = 0;           // pieces, S tiles, accumulators, P tiles so far
        bool ok = true;
        PagedPiece p;
        while (ok && take(pc, w, 32, p)) {
            const int ns = __shfl_sync(0xffffffffu, p.t1 - p.t0, 0);
            const uint32_t qs = pc % C::NQ;
            ok = mbar_wait_warp(bar(C::B_QFULL + qs), (pc / C::NQ) & 1u, w, 14);
            if (!ok) break;
            ++pc;
            if (x >= ns) {                                 // no step: its word on the Q tile is still due
                if (lane == 0) mbar_arrive(bar(C::B_QEMPTY + qs));
                __syncwarp();
            }
            // i: the step whose S^T is formed; its O^T follows one turn later
#pragma unroll 1
            for (int i = x; ok && i < ns + 2 && x < ns; i += 2) {
                if (i < ns) {
                    const uint32_t slot = x * C::NRING + kc % C::NRING;
                    const int buf = sc & 1u;
                    ok = mbar_wait_warp(bar(C::B_KVFULL + slot), (kc / C::NRING) & 1u, w, 13) &&
                         mbar_wait_warp(bar(C::B_SEMPTY + 2 * x + buf), ((sc >> 1) & 1u) ^ 1u, w, 15);
                    if (!ok) break;
                    ++sc;
                    kc += 2;
                    tc_fence_after();
                    const uint64_t kd = smem_desc_sw128(base + C::KV_OFF + slot * C::TILE_BYTES, 16u, 1024u);
                    const uint64_t qd = smem_desc_sw128(base + C::Q_OFF + qs * C::Q_BYTES, 16u, 1024u);
                    const uint32_t d_s = tbase + (x ? C::col_s(1, 0) : C::col_s(0, 0)) + (buf ? 32u : 0u);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t ko = ((kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32u) >> 4;
                        const uint32_t qo = ((kk >> 2) * C::Q_CHUNK + (kk & 3) * 32u) >> 4;
                        mma_ss_f16_elect(d_s, kd + ko, qd + qo, idesc_s, kk > 0 ? 1u : 0u);
                    }
                    mma_commit_elect(bar(C::B_SFULL + 2 * x + buf));
                    mma_commit_elect(bar(C::B_KVEMPTY + slot));
                    if (i + 2 >= ns) mma_commit_elect(bar(C::B_QEMPTY + qs));
                }
                if (i >= 2) {
                    const uint32_t slot = x * C::NRING + vc % C::NRING;
                    const bool begin = i < 4, end = i >= ns;
                    ok = mbar_wait_warp(bar(C::B_KVFULL + slot), (vc / C::NRING) & 1u, w, 10);
                    if (ok && begin) ok = mbar_wait_warp(bar(C::B_OEMPTY + x), (un & 1u) ^ 1u, w, 11);
                    if (ok) ok = mbar_wait_warp(bar(C::B_PFULL + x), pp & 1u, w, 12);
                    if (!ok) break;
                    ++pp;
                    vc += 2;
                    tc_fence_after();
                    // V as A, MN-major (at d = 64 the product's upper 64 lanes are
                    // whatever lies one chunk further; nobody reads them)
                    const uint64_t vd = smem_desc_sw128(base + C::KV_OFF + slot * C::TILE_BYTES, C::CHUNK_BYTES, 1024u);
                    const uint64_t pd = smem_desc_sw128(base + C::P_OFF + x * C::P_BYTES, 16u, 1024u);
                    const uint32_t d_o = tbase + (x ? C::col_o(1) : C::col_o(0));
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t po = ((kk >> 2) * C::P_CHUNK + (kk & 3) * 32u) >> 4;
                        mma_ss_f16_elect(d_o, vd + ((kk * 16 * 128u) >> 4), pd + po, idesc_o, (!begin || kk > 0) ? 1u : 0u);
                    }
                    mma_commit_elect(bar(C::B_KVEMPTY + slot));
                    mma_commit_elect(bar(C::B_PEMPTY + x));
                    if (end) {
                        mma_commit_elect(bar(C::B_OFULL + x));
                        ++un;
                    }
                }
            }
        }
        // Drain: every issued MMA completes before TMEM is released.
        mma_commit_elect(bar(C::B_DONE + x));
        mbar_wait_quiet(bar(C::B_DONE + x), 0, 500000000ull);
        __syncwarp();
    } else {
        // =================== group x: one key a thread, then one output column ===================
        const int x = warp >> 2, row = tid & 127, gwarp = warp & 3;
        const uint32_t lane_off = static_cast<uint32_t>(gwarp * 32) << 16;
        WaitCtx w{abort_flag, a.status, x ? kRoleSoftmax1 : kRoleSoftmax0};
        const float sl2 = a.scale_log2;
        float *ref = reinterpret_cast<float *>(gbase + C::R_OFF) + 32 * x;   // r of every row
        float *xch = reinterpret_cast<float *>(gbase + C::X_OFF);
        uint8_t *pbuf = gbase + C::P_OFF + x * C::P_BYTES;
        float *scratch = reinterpret_cast<float *>(pbuf);                    // while no product reads P
        // element (row n, this key) of P^T: chunk, then 128-byte rows whose
        // 16-byte parts are swizzled by the row
        uint8_t *pkey = pbuf + (row >> 6) * C::P_CHUNK;
        const uint32_t pcol = static_cast<uint32_t>(row & 63) * 2u;
        uint32_t pc = 0, sc = 0, pn = 0, un0 = 0, un1 = 0, nx = 0;   // pieces, steps (twice), accumulators, exchanges
        bool bad = false;
        PagedPiece p;
        for (;;) {
            const bool more = take(pc, w, 24, p);
            if (group_any(x, !more || bad)) break;
            ++pc;
            const int ns = p.t1 - p.t0;
            const int nr = p.nl * a.group;                                   // rows that exist
            const int nf = min(a.first, p.vhi);
            const int last = p.pos + p.nl - 1;
            // a tile [k0, k0 + 128) that every row sees whole: k0 + 128 <= all_hi, and
            // k0 >= all_lo or k0 + 128 <= all_f
            const int all_hi = paged_hi(p.pos, p.n, a.wr), all_lo = paged_lo(last, a.wl), all_f = min(a.first, all_hi);
            float le[kN], lr[kN];                                            // this thread's keys, per row
#pragma unroll
            for (int n = 0; n < kN; ++n) { le[n] = 0.f; lr[n] = 0.f; }
            uint32_t unseen = ~0u;                                           // rows without a reference yet
#pragma unroll 1
            for (int i = x; i < ns; i += 2) {
                const int k0 = paged_tile(p, p.t0 + i) * 128, kk = k0 + row;
                const int buf = sc & 1u;
                bad = !mbar_wait_warp(bar(C::B_SFULL + 2 * x + buf), (sc >> 1) & 1u, w, 20);
                ++sc;
                if (!((k0 >= p.vlo && k0 + 128 <= p.vhi) || k0 + 128 <= nf)) {
                    // a tile that the unit sees in part: its other V rows become 0
                    // (pn: this group's steps before this one)
                    const uint32_t vc = 2 * pn + 1, slot = x * C::NRING + vc % C::NRING;
                    bad = !mbar_wait_warp(bar(C::B_KVFULL + slot), (vc / C::NRING) & 1u, w, 22) || bad;
                    if (!bad && !((kk >= p.vlo && kk < p.vhi) || kk < nf)) {
                        uint8_t *vr = gbase + C::KV_OFF + slot * C::TILE_BYTES + row * 128;
#pragma unroll
                        for (int ch = 0; ch < C::NCH; ++ch)
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<uint4 *>(vr + ch * C::CHUNK_BYTES + q * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                tc_fence_after();
                uint32_t s[kN];
                const uint32_t tS = tbase + lane_off + C::col_s(0, 0) + 64u * x + 32u * buf;
                tmem_ld8(tS, s);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_SEMPTY + 2 * x + buf));
                // rows [ca, cb) see this key
                int ca = 0, cb = nr;
                if (!(k0 + 128 <= all_hi && (k0 >= all_lo || k0 + 128 <= all_f))) {
                    const long long ra = a.wr >= 0 ? static_cast<long long>(kk) - a.wr - p.pos : 0;
                    const long long rb = a.wl >= 0 && kk >= a.first ? static_cast<long long>(kk) + a.wl - p.pos + 1 : p.nl;
                    ca = static_cast<int>(min(max(ra, 0ll), static_cast<long long>(p.nl))) * a.group;
                    cb = kk < p.n ? static_cast<int>(min(max(rb, 0ll), static_cast<long long>(p.nl))) * a.group : 0;
                }
                // x - r; hidden scores are -inf, rows without a reference take r = 0
                bool big = false;
#pragma unroll
                for (int n4 = 0; n4 < kN; n4 += 4) {
                    if (n4 >= nr) continue;
                    const float4 r4 = *reinterpret_cast<const float4 *>(ref + n4);
                    const float rv[4] = {r4.x, r4.y, r4.z, r4.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = n4 + q;
                        const bool first_seen = (unseen & (1u << n)) != 0;
                        float v = fmaf(__uint_as_float(s[n]), sl2, first_seen ? 0.f : -rv[q]);
                        v = n >= ca && n < cb ? v : -INFINITY;
                        big |= v > C::CAP || (first_seen && v != -INFINITY);
                        s[n] = __float_as_uint(v);
                    }
                }
                // the last product has read P (its buffer is scratch until then)
                bad = !mbar_wait_warp(bar(C::B_PEMPTY + x), (pn & 1u) ^ 1u, w, 23) || bad;
                ++pn;
                if (group_any(x, big || bad)) {
                    // ---- new references: the rows' maxima over the tile ----
                    if (lane == 0) scratch[128 + gwarp] = bad ? 1.f : 0.f;
                    float m[kN];
#pragma unroll
                    for (int n = 0; n < kN; ++n) m[n] = n < nr ? __uint_as_float(s[n]) : -INFINITY;
                    const float top = warp_reduce_transposed<kN, true>(m);
                    if (lane < kN) scratch[gwarp * kN + lane] = top;
                    group_any(x, false);
                    bad = bad || scratch[128] + scratch[129] + scratch[130] + scratch[131] != 0.f;
                    bool moved = false;
                    float mine = 0.f;                                        // row `lane`'s new reference
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        m[n] = 1.f;
                        if (n >= nr) continue;
                        const bool first_seen = (unseen & (1u << n)) != 0;
                        const float o = first_seen ? 0.f : ref[n];
                        const float mx = fmaxf(fmaxf(scratch[n], scratch[kN + n]), fmaxf(scratch[2 * kN + n], scratch[3 * kN + n])) + o;
                        float rn = o, corr = 1.f;
                        if (first_seen) {
                            if (mx != -INFINITY) { rn = mx; unseen &= ~(1u << n); }
                        } else if (mx > o + C::TAU) {
                            rn = mx;
                            corr = ex2_approx(o - rn);
                            moved = true;
                        }
                        if (lane == n) mine = rn;
                        le[n] *= corr;
                        lr[n] *= corr;
                        s[n] = __float_as_uint(__uint_as_float(s[n]) + (o - rn));
                        m[n] = corr;
                    }
                    if (moved && !bad) {
                        // O^T's columns (lanes are output columns), all products done
                        const uint32_t tO = tbase + lane_off + C::col_o(0) + 32u * x;
                        uint32_t ov[kN];
                        tc_fence_after();
                        tmem_ld8(tO, ov);
                        tmem_ld_wait();
#pragma unroll
                        for (int n = 0; n < kN; ++n) ov[n] = __float_as_uint(__uint_as_float(ov[n]) * m[n]);
                        tmem_st8(tO, ov);
                        tmem_st_wait();
                        tc_fence_before();
                    }
                    group_any(x, false);                                     // all have read ref and scratch
                    if (gwarp == 0 && lane < nr) ref[lane] = mine;
                    group_any(x, false);
                    if (bad) break;
                }
#pragma unroll
                for (int n4 = 0; n4 < kN; n4 += 4) {
                    if (n4 >= nr) continue;
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        const int n = n4 + q;
                        const float e0 = ex2_approx(__uint_as_float(s[n])), e1 = ex2_approx(__uint_as_float(s[n + 1]));
                        const uint32_t pk = pack2<kBF16>(e0, e1);
                        le[n] += e0;
                        le[n + 1] += e1;
                        add_pair<kBF16>(lr[n], lr[n + 1], pk);
                        *reinterpret_cast<uint16_t *>(pkey + n * 128 + (pcol ^ ((n & 7) << 4))) = static_cast<uint16_t>(pk);
                        *reinterpret_cast<uint16_t *>(pkey + (n + 1) * 128 + (pcol ^ (((n + 1) & 7) << 4))) =
                            static_cast<uint16_t>(pk >> 16);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_PFULL + x));
            }
            const bool some = x < ns, joined = ns >= 2;
            // ---- row n's sums over all keys of the group, in thread n ----
            const float le_w = warp_reduce_transposed<kN>(le), lr_w = warp_reduce_transposed<kN>(lr);
            float *sums = reinterpret_cast<float *>(gbase + C::RED_OFF) + 64 * x;
            if (lane < kN) {
                sums[gwarp * kN + lane] = le_w;
                sums[(4 + gwarp) * kN + lane] = lr_w;
            }
            if (group_any(x, bad)) break;
            float lse2 = -INFINITY, inv = 0.f;                               // of row n = lane (warp 0)
            if (gwarp == 0 && some && lane < nr) {
                const float e = (sums[lane] + sums[kN + lane]) + (sums[2 * kN + lane] + sums[3 * kN + lane]);
                const float q = (sums[4 * kN + lane] + sums[5 * kN + lane]) + (sums[6 * kN + lane] + sums[7 * kN + lane]);
                if (!(e <= 0.f)) {                                           // (a NaN that the row sees stays one)
                    lse2 = ref[lane] + log2f(e);
                    inv = 1.f / q;
                }
            }
            if (x == 1) {
                if (joined) {
                    if (gwarp == 0) {
                        bad = !mbar_wait_warp(bar(C::B_XEMPTY), (nx & 1u) ^ 1u, w, 25);
                        xch[lane] = lse2;
                        xch[32 + lane] = inv;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::B_XFULL));
                    }
                    bad = !mbar_wait_warp(bar(C::B_OFULL + 1), un1 & 1u, w, 21) || bad;
                    ++nx;
                    ++un1;
                }
                ++un0;
                continue;
            }
            // ---- group 0: join the halves, write the rows ----
            float *fac = xch + 64;                                           // the rows' factors, [2][32]
            if (gwarp == 0) {
                float inv1 = 0.f;
                if (joined) {
                    bad = !mbar_wait_warp(bar(C::B_XFULL), nx & 1u, w, 26);
                    const float l1 = xch[lane], m = fmaxf(lse2, l1);
                    inv1 = xch[32 + lane];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_XEMPTY));
                    if (lse2 != -INFINITY || l1 != -INFINITY) {
                        const float w0 = ex2_approx(lse2 - m), w1 = ex2_approx(l1 - m), k = 1.f / (w0 + w1);
                        inv *= w0 * k;
                        inv1 *= w1 * k;
                        lse2 = m + log2f(w0 + w1);
                    }
                }
                fac[lane] = inv;
                fac[32 + lane] = inv1;
                if (lane < nr) {
                    if (p.slot >= 0) {
                        wk.lse[static_cast<size_t>(p.slot) * 256 + lane] = lse2;
                    } else if (a.lse != nullptr) {
                        const int tok = p.qrow + lane / a.group, qh = p.h * a.group + lane % a.group;
                        a.lse[static_cast<size_t>(qh) * a.T + tok] = lse2 * 0.69314718055994530942f;
                    }
                }
            }
            bad = !mbar_wait_warp(bar(C::B_OFULL), un0 & 1u, w, 21) || bad;
            if (joined) bad = !mbar_wait_warp(bar(C::B_OFULL + 1), un1 & 1u, w, 27) || bad;
            if (group_any(0, bad)) break;
            tc_fence_after();
            const uint32_t tO = tbase + lane_off + C::col_o(0);
            int tok = p.qrow, hd = 0;
            float *part = wk.o + static_cast<size_t>(max(p.slot, 0)) * 256 * D + row;
            uint16_t *out = reinterpret_cast<uint16_t *>(a.o) + static_cast<size_t>(p.h) * a.group * D + row;
            uint32_t o0[8], o1[8];
            tmem_ld8(tO, o0);
            tmem_ld8(tO + (C::col_o(1) - C::col_o(0)), o1);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {                                                 // the accumulators are read
                mbar_arrive(bar(C::B_OEMPTY));
                if (joined) mbar_arrive(bar(C::B_OEMPTY + 1));
            }
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                if (n >= nr || row >= D) continue;                           // (d = 64: lanes that hold nothing)
                float v = __uint_as_float(o0[n]) * fac[n];
                if (joined) v = fmaf(__uint_as_float(o1[n]), fac[32 + n], v);
                if (p.slot >= 0)
                    part[n * D] = v;
                else
                    out[(static_cast<size_t>(tok) * a.H + hd) * D] = static_cast<uint16_t>(pack2<kBF16>(v, 0.f));
                if (++hd == a.group) { hd = 0; ++tok; }
            }
            ++un0;
            if (joined) { ++un1; ++nx; }
        }
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if (warp == 10) {
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace fa
