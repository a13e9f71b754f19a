// fa_paged_fwd_kernel.cuh -- attention of new tokens over a paged cache on
// sm_103a (tcgen05 + TMA): more than 8 rows a Q tile (fewer: fa_paged_token_kernel.cuh).
//
// Rows.  The g = H / H_kv query heads of a K/V head share each Q tile: tile
// row p holds the tile's position p / g, head p % g, R positions a tile
// (R g <= 128), so one pass over a K/V head's pages serves the group.
//
// Units.  A unit is a pair of Q tiles (L, H) of one (sequence, K/V head), dealt
// to the CTAs in equal shares of steps (fa_paged_share.cuh).  A step is one
// 128-key tile:
//   * Two tiles: both softmax groups walk every step, each for its own tile
//     (the schedule of fa_fwd_kernel.cuh): 256 rows per K/V tile read.
//   * One tile (a short or a chunk's last one): the groups take the steps in turn,
//     each with an accumulator of its own, joined in TMEM at the end: one tile's
//     chain QK -> softmax -> PV is longer than its tensor work, and two of them
//     side by side overlap (1850 to 2300 cycles a step).
//
// P is rounded to the 16-bit type (fa_paged_token_kernel.cuh tells what that costs).
//
// Measured.  Bound by the tensor core and each tile's chain QK -> softmax -> PV,
// whose parts cannot overlap within a tile (S and P share their columns; at d = 128
// there are no others, at d = 64 128 columns lie idle): ~3400 cycles a step of two
// tiles, 2180 of them tensor work, as in the dense forward (~3090).  Three chunks of
// 1100 to 1200 tokens on caches of up to 14516 (32 heads over 8, d = 128): 548 us,
// 1305 TFLOP/s; 575 to 595 in long runs, under the power cap.  24 sequences with 1 to
// 300 new tokens on caches of up to 4096: 86 us, of which ~4 pass before a CTA's first
// scores, up to 10 go to the joining kernel's 152 cut units and its launch, and some
// to shares that count a step of one tile like one of two.  At d = 128 the epilogue of
// units with one tile spills (172 bytes: both groups' accumulators are held at once).
// Tried: an issuing warp for each Q tile (750 us for the chunks) and the issuer's
// loop unrolled for both tiles (608): both are code that pushes the softmax out
// of the instruction cache; shares in which a step of two tiles counts twice (the
// batch 99 us; by the cycles it is 3 : 2 to 5 : 3, and units had no cost of their own
// then).
//
// Warps: 0-3 and 4-7 the softmax groups, 8 and 11 the TMA producers of K and V
// (all lanes: one box of a page each), 9 the MMA issuer, 10 walks the share and
// posts its pieces in a ring that the others read.
//
// Code size.  Twelve warps run five different roles, and what their loops execute
// has to stay in the instruction cache: with two copies of the softmax step, four
// of each product and non-uniform descriptors every role ran at a third of its
// speed.  So there is one copy of each, and what differs between the two
// tiles and the two schedules is data.
//
// Pages.  A 128-key tile is 128 / page_size boxes (or part of one page).  A
// page that no row of the unit sees, or a bad id, is loaded from beyond the
// pool, which TMA fills with zeros.  In a tile that the unit sees in part, the
// rows of V outside are set to zero in shared memory before the product:
// their probabilities are 0, but 0 times a NaN left in a slot is not.
// Every mbarrier wait is bounded (fa_device.cuh).
#pragma once

#include "fa_paged_share.cuh"

namespace fa {

template <int D, bool kBF16>
struct PagedCfg {
    static constexpr int NCH = D / 64;                    // 128-byte column chunks
    static constexpr uint32_t CHUNK_BYTES = 128u * 128u;
    static constexpr uint32_t TILE_BYTES = NCH * CHUNK_BYTES;
    static constexpr int NSTAGE = D == 64 ? 8 : 4;
    static constexpr bool kByStep = false;                // K in the even slots, V in the odd ones
    static constexpr int NRING = NSTAGE;
    static constexpr int NQ = 3;
    static constexpr int QK_STEPS = D / 16, PV_STEPS = 8;
    static constexpr int NTHREADS = 384;
    static constexpr uint32_t REGS_LOW = 96, REGS_HIGH = 200;
    static_assert(128 * REGS_LOW + 256 * REGS_HIGH <= 384 * 168, "register budget");
    static constexpr int RING = 4;                        // pieces ahead
    static constexpr uint32_t Q_CHUNK = CHUNK_BYTES, Q_BYTES = TILE_BYTES;
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t KV_OFF = NQ * TILE_BYTES;
    static constexpr uint32_t X_OFF = KV_OFF + NSTAGE * TILE_BYTES;   // group H's LSE, 1 / l
    static constexpr uint32_t RING_OFF = X_OFF + 2 * 128 * 4;
    static constexpr uint32_t BAR_OFF = RING_OFF + RING * 64;
    static constexpr int B_QFULL = 0, B_QEMPTY = NQ, B_KVFULL = 2 * NQ, B_KVEMPTY = B_KVFULL + NSTAGE,
                         B_SFULL = B_KVEMPTY + NSTAGE, B_PFULL = B_SFULL + 2, B_OFULL = B_PFULL + 2,
                         B_OEMPTY = B_OFULL + 2, B_XFULL = B_OEMPTY + 2, B_XEMPTY = B_XFULL + 1,
                         B_MMADONE = B_XEMPTY + 1, B_PIECE = B_MMADONE + 1, B_FREE = B_PIECE + RING,
                         NBAR = B_FREE + RING;
    // Arrivals that complete a phase: a group's four warps; producers, MMA issuer
    // and the groups' warps.
    __device__ static uint32_t arrivals(int i) {
        return i == B_PFULL || i == B_PFULL + 1 || (i >= B_OEMPTY && i < B_MMADONE) ? 4u : i >= B_FREE ? 11u : 1u;
    }
    static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr uint32_t SMEM_BYTES = MISC_OFF + 16 + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
    static constexpr uint32_t TMEM_COLS = 512;
    __host__ __device__ static constexpr uint32_t col_s(int x) { return x ? 128u : 0u; }
    __host__ __device__ static constexpr uint32_t col_o(int x) { return 256u + (x ? D : 0u); }
    static constexpr uint32_t IDESC_QK = idesc_f16(128, 128, kBF16, false, false);
    static constexpr uint32_t IDESC_PV = idesc_f16(128, D, kBF16, false, true);
    // fa_fwd_kernel.cuh: the conditional rescale, tau in log2 units, and the
    // row sum up to which a tile's P against the old reference is kept: fp16's
    // largest number, so that no term of it becomes infinite.
    static constexpr float TAU = 8.0f, KEEP_SUM = 65504.0f;
};

template <int D, bool kBF16>
__global__ void __launch_bounds__(384, 1)
fa_paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const PagedArgs a, const PagedWork wk,
                    const int R) {
    using C = PagedCfg<D, kBF16>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return base + C::BAR_OFF + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gbase + C::MISC_OFF);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + C::MISC_OFF + 4);
    PagedPiece *ring = reinterpret_cast<PagedPiece *>(gbase + C::RING_OFF);

    // ---- prologue: TMEM (warp 9), barriers (thread 0), this CTA's share ----
    if (warp == 9) tmem_alloc(base + C::MISC_OFF, C::TMEM_COLS);
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
    // (the scratch lies in the K/V ring, which no copy uses yet)
    tc_fence_before();
    const PagedShare share = paged_share<C::NTHREADS, kUnitCostChunk>(a, 2 * R, gbase + C::KV_OFF);
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    // Reads piece number i (every role keeps its own count), whole warp; the
    // caller releases it.
    auto take = [&](uint32_t i, const WaitCtx &w, uint32_t where, PagedPiece &p) __attribute__((always_inline)) -> bool {
        const uint32_t q = i % C::RING;
        if (!mbar_wait_warp(bar(C::B_PIECE + q), (i / C::RING) & 1u, w, where)) return false;
        p = ring[q];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_FREE + q));
        return p.qrow >= 0;
    };

    if (warp >= 8) {
      regs_shrink<C::REGS_LOW>();
      if (warp == 10) {
        // =================== scheduler (whole warp) ===================
        WaitCtx w{abort_flag, a.status, kRolePaged};
        uint32_t np_out = 0;
        auto post = [&](const PagedPiece &p) __attribute__((always_inline)) -> bool {
            const uint32_t q = np_out % C::RING;
            if (!mbar_wait_idle(bar(C::B_FREE + q), ((np_out / C::RING) & 1u) ^ 1u, w, 30))
                return false;
            if (lane == 0) {
                ring[q] = p;
                mbar_arrive(bar(C::B_PIECE + q));
            }
            __syncwarp();
            ++np_out;
            return true;
        };
        if (paged_walk<true, kUnitCostChunk>(share, a, R, wk.desc + 8 * blockIdx.x, post)) {
            PagedPiece end{};
            end.qrow = -1;
            post(end);
        }
      } else if (warp != 9) {
        // =================== TMA producers (whole warps) ===================
        paged_produce<C>(warp == 11, tm_q, tm_k, tm_v, a, R, base, take,
                         WaitCtx{abort_flag, a.status, kRoleProducer});
      } else if (warp == 9) {
        // =================== MMA issuer (whole warp, one elected lane issues) ===================
        // Step i multiplies Q with its K tile, and P of step i - lag with that
        // step's V tile: with two Q tiles for both of them (lag 1), with one
        // for the group whose turn it is (lag 2).  Everything that a
        // descriptor depends on is kept warp-uniform (uniform()): tcgen05.mma
        // takes uniform registers.
        WaitCtx w{abort_flag, a.status, kRoleMma};
        auto uniform = [](int v) __attribute__((always_inline)) -> int { return __shfl_sync(0xffffffffu, v, 0); };
        uint32_t qs = 0, qph = 0, ks = 0, kph = 0, vs = 1, vph = 0, pi = 0;   // slots and their phases
        uint32_t un = 0, pp = 0;                           // bit x: phase of group x's accumulator, of its P
        bool ok = true;
        PagedPiece p;
        while (ok && take(pi, w, 32, p)) {
            ++pi;
            const int ns = uniform(p.t1 - p.t0);
            const bool one = uniform(p.nh) == 0;
            const int lag = one ? 2 : 1;
            const int s0l = one ? 0 : uniform(max(p.t0, p.skip) - p.t0);       // tile L's first step
            uint32_t q1 = qs + 1, q1ph = qph;              // tile H's slot
            if (q1 == C::NQ) { q1 = 0; q1ph ^= 1u; }
            // (an unused Q tile still has to land before its slot is released)
            if (s0l >= ns) ok = mbar_wait_warp(bar(C::B_QFULL + qs), qph, w, 15);
#pragma unroll 1
            for (int i = 0; i < ns + lag && ok; ++i) {
                const int iv = i - lag;
                bool v_here = false, k_here = false;       // (the second tile need not look again)
#pragma unroll 1
                for (int x = one ? i & 1 : 0; x < 2; ++x) {
                    const int s0 = one ? x : x ? 0 : s0l;
                    const uint32_t d_s = tbase + (x ? C::col_s(1) : C::col_s(0));
                    if (iv >= s0) {
                        const uint32_t d_o = tbase + (x ? C::col_o(1) : C::col_o(0));
                        const bool begin = iv == s0;
                        if (!v_here) ok = mbar_wait_warp(bar(C::B_KVFULL + vs), vph, w, 10);
                        v_here = true;
                        if (ok && begin) ok = mbar_wait_warp(bar(C::B_OEMPTY + x), ((un >> x) & 1u) ^ 1u, w, 11);
                        if (ok) ok = mbar_wait_warp(bar(C::B_PFULL + x), (pp >> x) & 1u, w, 12);
                        if (!ok) break;
                        pp ^= 1u << x;
                        tc_fence_after();
                        const uint64_t vd = smem_desc_sw128(base + C::KV_OFF + vs * C::TILE_BYTES, C::CHUNK_BYTES, 1024u);
#pragma unroll
                        for (int kk = 0; kk < C::PV_STEPS; ++kk)
                            mma_ts_f16_elect(d_o, d_s + kk * 8u, vd + ((kk * 16 * 128u) >> 4), C::IDESC_PV,
                                             (!begin || kk > 0) ? 1u : 0u);
                        if (iv + lag >= ns) {              // its last step
                            mma_commit_elect(bar(C::B_OFULL + x));
                            un ^= 1u << x;
                        }
                    }
                    if (i < ns && i >= s0) {
                        const uint32_t qx = one || x == 0 ? qs : q1, qxp = one || x == 0 ? qph : q1ph;
                        if (!k_here) ok = mbar_wait_warp(bar(C::B_KVFULL + ks), kph, w, 13);
                        k_here = true;
                        if (ok && i == s0) ok = mbar_wait_warp(bar(C::B_QFULL + qx), qxp, w, 14);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t qd = smem_desc_sw128(base + C::Q_OFF + qx * C::TILE_BYTES, 16u, 1024u);
                        const uint64_t kd = smem_desc_sw128(base + C::KV_OFF + ks * C::TILE_BYTES, 16u, 1024u);
#pragma unroll
                        for (int kk = 0; kk < C::QK_STEPS; ++kk) {
                            const uint32_t off = ((kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32u) >> 4;
                            mma_ss_f16_elect(d_s, qd + off, kd + off, C::IDESC_QK, kk > 0 ? 1u : 0u);
                        }
                        mma_commit_elect(bar(C::B_SFULL + x));
                    }
                    if (one) break;
                }
                if (!ok) break;
                if (i == ns - 1) {
                    mma_commit_elect(bar(C::B_QEMPTY + qs));
                    if (!one) mma_commit_elect(bar(C::B_QEMPTY + q1));
                }
                if (i < ns) {
                    mma_commit_elect(bar(C::B_KVEMPTY + ks));
                    ks += 2;
                    if (ks >= C::NSTAGE) { ks = 0; kph ^= 1u; }
                }
                if (iv >= 0) {
                    mma_commit_elect(bar(C::B_KVEMPTY + vs));
                    vs += 2;
                    if (vs >= C::NSTAGE) { vs = 1; vph ^= 1u; }
                }
            }
            qs = one ? qs + 1 : q1 + 1;
            qph = one ? qph : q1ph;
            if (qs == C::NQ) { qs = 0; qph ^= 1u; }
        }
        // Drain: every issued MMA completes before TMEM is released.
        mma_commit_elect(bar(C::B_MMADONE));
        mbar_wait_quiet(bar(C::B_MMADONE), 0, 500000000ull);
        __syncwarp();
      }
    } else {
        regs_grow<C::REGS_HIGH>();
        // =================== softmax group x ===================
        const int x = warp >> 2;
        const int row = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tbase + lane_off + C::col_s(x);
        const uint32_t tO = tbase + lane_off + C::col_o(x);
        WaitCtx w{abort_flag, a.status, x ? kRoleSoftmax1 : kRoleSoftmax0};
        const float sl2 = a.scale_log2;
        float *xch = reinterpret_cast<float *>(gbase + C::X_OFF);
        const bool v8ok = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
        uint32_t pi = 0, kv = 0, sph = 0;
        uint32_t un0 = 0, un1 = 0, nx = 0;                 // accumulator uses per group, exchanges
        bool ok = true;
        const int my_pos = row / a.group;                  // this row's position within a tile
        const int my_head = row - my_pos * a.group;
        PagedPiece p;
        while (ok && take(pi, w, 24, p)) {
            ++pi;
            const bool one = p.nh == 0;
            const int ns = p.t1 - p.t0;
            const int tile = one ? 0 : x;                  // the Q tile this group works on
            const int npos = tile ? p.nh : p.nl;
            const int s0 = one ? x : x ? 0 : max(p.t0, p.skip) - p.t0;   // its first step
            const int ds = one ? 2 : 1;
            const bool valid = my_pos < npos;
            const bool live_warp = __any_sync(0xffffffffu, valid);
            const int pos = p.pos + tile * R + my_pos;
            const int klo = paged_lo(pos, a.wl), khi = paged_hi(pos, p.n, a.wr), kf = min(a.first, khi);
            const int nf = min(a.first, p.vhi);            // first tokens that any row sees
            // r: reference point (log2 units); le: row sum of the FP32
            // exponentials (LSE); lr: of the same rounded as P (normalises O).
            // Rows that hold no token never ask for a new reference.
            float r = valid ? -INFINITY : 0.f, le = 0.f, lr = 0.f;
            for (int i = s0; i < ns; i += ds) {
                const int k0 = paged_tile(p, p.t0 + i) * 128;
                ok = mbar_wait(bar(C::B_SFULL + x), sph, w, 20);
                if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
                sph ^= 1;
                // ---- a tile that the unit sees in part: its other V rows become 0 ----
                if (!((k0 >= p.vlo && k0 + 128 <= p.vhi) || k0 + 128 <= nf)) {
                    const uint32_t idx = kv + 2 * i + 1, slot = idx % C::NSTAGE;
                    ok = mbar_wait(bar(C::B_KVFULL + slot), (idx / C::NSTAGE) & 1u, w, 22);
                    if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
                    const int kk = k0 + row;
                    if (!((kk >= p.vlo && kk < p.vhi) || kk < nf)) {
                        uint8_t *vr = gbase + C::KV_OFF + slot * C::TILE_BYTES + row * 128;
#pragma unroll
                        for (int ch = 0; ch < C::NCH; ++ch)
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<uint4 *>(vr + ch * C::CHUNK_BYTES + q * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (!live_warp) {
                    if (lane == 0) mbar_arrive(bar(C::B_PFULL + x));
                    continue;
                }
                tc_fence_after();
                uint32_t s[128];
                float *sf = reinterpret_cast<float *>(s);
                // visible columns: c < lim, and c >= llo or c < lf
                const int lim = valid ? khi - k0 : 128, llo = valid ? klo - k0 : 0, lf = kf - k0;
                const bool masked = __any_sync(0xffffffffu, lim < 128 || (llo > 0 && lf < 128));
                float rn = r, corr = 1.f;
                bool need = false;
                float2 e_a, e_b;
                uint32_t pk[64];
                const float2 c2 = make_float2(sl2, sl2);
                // P against the current reference first; the maximum only on the
                // first tile or when a row's sum got too large (fa_fwd_kernel.cuh)
                bool keep = __all_sync(0xffffffffu, r != -INFINITY);
#pragma unroll 1
                for (;;) {
                    tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                    tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                    tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&s[64]));
                    tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&s[96]));
                    tmem_ld_wait();
                    if (masked) {
#pragma unroll
                        for (int w32 = 0; w32 < 4; ++w32) {
                            // bit c of m: column 32 w32 + c is visible
                            auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
                            const uint32_t m = below(lim - 32 * w32) & (~below(llo - 32 * w32) | below(lf - 32 * w32));
#pragma unroll
                            for (int cc = 0; cc < 32; ++cc)
                                if (!(m & (1u << cc))) sf[32 * w32 + cc] = -INFINITY;
                        }
                    }
                    if (!keep) {
                        float m0 = sf[0], m1 = sf[1], m2 = sf[2], m3 = sf[3];
#pragma unroll
                        for (int cc = 4; cc < 128; cc += 8) {
                            m0 = max3(m0, sf[cc + 0], sf[cc + 4]);
                            m1 = max3(m1, sf[cc + 1], sf[cc + 5]);
                            m2 = max3(m2, sf[cc + 2], sf[cc + 6]);
                            m3 = max3(m3, sf[cc + 3], sf[cc + 7]);
                        }
                        const float bnew = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * sl2;
                        if (valid) {
                            if (r == -INFINITY) rn = bnew;
                            else { rn = (bnew > r + C::TAU) ? bnew : r; corr = ex2_approx(r - rn); }
                            need = (r != -INFINITY) && (rn != r);
                        }
                    }
                    const float rs = rn == -INFINITY ? 0.f : rn;
                    const float2 nr2 = make_float2(-rs, -rs);
                    e_a = make_float2(0.f, 0.f);
                    e_b = e_a;
#pragma unroll
                    for (int cc = 0; cc < 128; cc += 4) {
                        const float2 x01 = __ffma2_rn(make_float2(sf[cc + 0], sf[cc + 1]), c2, nr2);
                        const float2 x23 = __ffma2_rn(make_float2(sf[cc + 2], sf[cc + 3]), c2, nr2);
                        const float2 e01 = make_float2(ex2_approx(x01.x), ex2_approx(x01.y));
                        const float2 e23 = make_float2(ex2_approx(x23.x), ex2_approx(x23.y));
                        pk[cc / 2] = pack2<kBF16>(e01.x, e01.y);
                        pk[cc / 2 + 1] = pack2<kBF16>(e23.x, e23.y);
                        e_a = __fadd2_rn(e_a, e01);
                        e_b = __fadd2_rn(e_b, e23);
                    }
                    if (!keep) break;
                    const float ts = (e_a.x + e_a.y) + (e_b.x + e_b.y);
                    if (__all_sync(0xffffffffu, !valid || ts <= C::KEEP_SUM)) break;
                    keep = false;
                }
                tmem_st32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
                tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
                // ---- correction of O (its previous PV completed before S_FULL) ----
                if (__any_sync(0xffffffffu, need)) {
                    const float2 cc2 = make_float2(corr, corr);
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t ov[32];
                        tmem_ld32(tO + ch * 32, ov);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 32; q += 2) {
                            const float2 v2 = __fmul2_rn(
                                make_float2(__uint_as_float(ov[q]), __uint_as_float(ov[q + 1])), cc2);
                            ov[q] = __float_as_uint(v2.x);
                            ov[q + 1] = __float_as_uint(v2.y);
                        }
                        tmem_st32(tO + ch * 32, ov);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_PFULL + x));
                // ---- row sums, after P is published ----
                le = __fmaf_rn(le, corr, (e_a.x + e_a.y) + (e_b.x + e_b.y));
                float2 r_a = make_float2(0.f, 0.f), r_b = r_a;
#pragma unroll
                for (int q = 0; q < 64; q += 2) {
                    add_pair<kBF16>(r_a.x, r_a.y, pk[q]);
                    add_pair<kBF16>(r_b.x, r_b.y, pk[q + 1]);
                }
                lr = __fmaf_rn(lr, corr, (r_a.x + r_a.y) + (r_b.x + r_b.y));
                r = rn;
            }
            if (!ok) break;
            kv += 2 * ns;
            // ---- this group's normaliser and LSE (log2 units) ----
            const bool some = s0 < ns;
            const bool live = some && !(le <= 0.f);        // (a NaN that the row sees stays one)
            float inv = live ? 1.f / lr : 0.f;
            float lse2 = live ? r + log2f(le) : -INFINITY;
            const bool joined = one && ns >= 2;            // group H has a share of this tile
            if (one && x == 1) {
                if (joined) {
                    ok = mbar_wait_warp(bar(C::B_XEMPTY), (nx & 1u) ^ 1u, w, 25);
                    if (!ok) break;
                    xch[row] = lse2;
                    xch[128 + row] = inv;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::B_XFULL));
                    ++nx;
                    ++un1;
                }
                ++un0;
                continue;
            }
            const uint32_t my_un = x ? un1 : un0;
            if (some) {
                ok = mbar_wait_warp(bar(C::B_OFULL + x), my_un & 1u, w, 21);
                if (!ok) break;
            }
            float inv_h = 0.f;
            if (joined) {
                ok = mbar_wait_warp(bar(C::B_XFULL), nx & 1u, w, 26) &&
                     mbar_wait_warp(bar(C::B_OFULL + 1), un1 & 1u, w, 27);
                if (!ok) break;
                const float l_h = xch[row];
                const float m = fmaxf(lse2, l_h);
                if (lse2 != -INFINITY || l_h != -INFINITY) {
                    const float w_l = ex2_approx(lse2 - m), w_h = ex2_approx(l_h - m);
                    const float n2 = 1.f / (w_l + w_h);
                    inv *= w_l * n2;
                    inv_h = xch[128 + row] * w_h * n2;
                    lse2 = m + log2f(w_l + w_h);
                }
            }
            tc_fence_after();
            uint32_t ov[D];
            if (some && live_warp) {
#pragma unroll
                for (int ch = 0; ch < D / 32; ++ch)
                    tmem_ld32(tO + ch * 32, *reinterpret_cast<uint32_t(*)[32]>(&ov[ch * 32]));
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < D; ++q) ov[q] = __float_as_uint(__uint_as_float(ov[q]) * inv);
                if (joined) {
#pragma unroll
                    for (int ch = 0; ch < D / 32; ++ch) {
                        uint32_t oh[32];
                        tmem_ld32(tbase + lane_off + C::col_o(1) + ch * 32, oh);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            ov[ch * 32 + q] = __float_as_uint(
                                fmaf(__uint_as_float(oh[q]), inv_h, __uint_as_float(ov[ch * 32 + q])));
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < D; ++q) ov[q] = 0u;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (some) mbar_arrive(bar(C::B_OEMPTY + x));
                if (joined) {
                    mbar_arrive(bar(C::B_OEMPTY + 1));
                    mbar_arrive(bar(C::B_XEMPTY));
                }
            }
            if (one) {
                ++un0;
                if (joined) { ++un1; ++nx; }
            } else {
                un0 += max(p.t0, p.skip) - p.t0 < ns ? 1u : 0u;
                ++un1;
            }
            if (!valid) continue;
            if (p.slot >= 0) {
                // a part of the unit: normalised O and LSE to the workspace
                const size_t part = (static_cast<size_t>(p.slot) * 2 + tile) * 128 + row;
                wk.lse[part] = lse2;
                if (some) {
                    float *prow = wk.o + part * D;
#pragma unroll
                    for (int ch = 0; ch < D / 8; ++ch) st_global_v8(prow + 8 * ch, &ov[8 * ch]);
                }
                continue;
            }
            const int tok = p.qrow + tile * R + my_pos, qh = p.h * a.group + my_head;
            uint16_t *orow = reinterpret_cast<uint16_t *>(a.o) + (static_cast<size_t>(tok) * a.H + qh) * D;
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch) {
                uint32_t pk[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    pk[q] = pack2<kBF16>(__uint_as_float(ov[16 * ch + 2 * q]), __uint_as_float(ov[16 * ch + 2 * q + 1]));
                if (v8ok) {
                    st_global_v8(orow + 16 * ch, pk);
                } else {
                    reinterpret_cast<uint4 *>(orow)[2 * ch] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    reinterpret_cast<uint4 *>(orow)[2 * ch + 1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                }
            }
            if (a.lse != nullptr) a.lse[static_cast<size_t>(qh) * a.T + tok] = lse2 * 0.69314718055994530942f;
        }
    }

    // ---- teardown ----
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace fa
