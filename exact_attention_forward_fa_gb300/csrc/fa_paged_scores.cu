// fa_paged_scores.cu -- the attention weight that each cached token of a
// paged cache gets from the new tokens, on sm_103a (tcgen05 + TMA):
//     A[b][h][j] += sum_i exp(alpha q_i . k_j - LSE_i)
// over the rows i that see token j and the query heads of K/V head h.
//
// The sum runs over rows, so the product is formed transposed, S^T = K Q^T:
// a TMEM lane, and with it a thread, holds one cached token, its columns are
// the rows of a Q tile (R positions x g heads, packed as in
// fa_paged_fwd_kernel.cuh).  A token's sum then stays in one thread's
// registers from the first row to the last: no reduction between threads, no
// atomics, and the order of the terms is fixed.
//
// A unit is a pair of 128-token tiles of one (sequence, K/V head), one for
// each of the two groups of four warps; their K tiles stay while the Q tiles that
// see them stream past, so a Q tile that is read once serves 256 tokens.
//
// Two forms, by the rows of a Q tile (R positions x g heads).
//   * kN = 32, up to 32 rows (decoding: one token of up to 32 heads a group).
//     The product has N = 32, the kernel reads K at the rate of HBM: 51.9 us,
//     5.4 TB/s, for 32 sequences of up to 8192 tokens (8 K/V heads, d = 128);
//     launch and first tiles are ~6 us of it.  Small Q tiles leave room for six K tiles
//     instead of four: the bytes in flight.  Each group's S^T is
//     double-buffered.  A warp of its own (12) loads group 1's K tiles: a tile of
//     16-token pages is 16 boxes at ~80 cycles each, and a unit's two tiles come
//     from HBM in ~2900.
//   * kN = 128.  A group moves its K tile into TMEM once a unit, where the product
//     takes it as its A operand.  From shared memory K would be read again for
//     every Q tile, which with Q's own reads and writes and the log-sum-exps
//     (32 16-byte loads a warp and tile) fills its 128 bytes a clock: 100 us
//     against 94.5 (928 TFLOP/s) for chunks of 973 and 742 tokens on caches of
//     7947 and 5023 (32 heads over 8, d = 128).  TMEM then has room for three S^T
//     buffers, which the two groups take in turn.
//     A pair of tiles takes ~2000 cycles: 1090 of tensor work, 1024 of exponentials
//     (32 a clock and SM), each group's chain of waits, TMEM loads and
//     exponentials ~1900.  Sixteen warps (half of the columns each, sums joined
//     through TMEM) took 98 us, barriers looked at ahead of their waits 97.5.
//
// Units are dealt to the CTAs in turn, back and forth; warp 10 finds a unit's
// sequence by a prefix sum over 32 sequences at a time.  Warp 8 loads the K
// tiles (page ids a unit ahead) and the Q tiles, warp 11 puts the log-sum-exps
// of a Q tile's rows beside it, warp 9 issues the products.  Columns of other
// sequences (a Q tile reads past its sequence's end) are dropped by selection,
// never by multiplying with zero.  A row whose log-sum-exp is NaN counts as one that
// adds nothing, and a bit beside the log-sum-exps makes the tokens that see it NaN:
// hidden columns stay free of it, at one 16-byte load a tile (selecting the hidden
// exponents instead of the hidden scores parts the additions from the exponentials:
// 132 us instead of 88 for chunks).
// Columns of a Q tile that are no rows (group sizes that do not divide 128, short
// calls) hold zeros, and an infinite key times zero is NaN: where a key is not
// finite (held in TMEM, on its way there) or a sum became NaN (keys in shared
// memory) they are selected away too. Selecting them in every tile took 81 us
// instead of 50 for chunks of 3 heads a group at d = 64, 58.5 instead of 56.4 for 32
// single tokens.
#include "fa_paged.cuh"

namespace fa {

template <int D, bool kBF16, int kN>
struct ScoresCfg {
    static constexpr int NCH = D / 64;
    static constexpr uint32_t CHUNK_BYTES = 128u * 128u;
    static constexpr uint32_t TILE_BYTES = NCH * CHUNK_BYTES;
    static constexpr uint32_t Q_CHUNK = kN * 128u, Q_BYTES = NCH * Q_CHUNK;
    static constexpr int NK = (D == 64 ? 2 : 1) * (kN == 32 ? 6 : 4);   // K tiles in flight
    static constexpr int NQ = D == 64 && kN == 128 ? 5 : 3;             // Q tiles in flight
    static constexpr int NL = 3;                                        // and their LSEs (held longer)
    static constexpr int NKX = NK / 2;                                  // slots of a group's K ring
    static constexpr bool kTwo = kN == 32;                              // a K producer for each group
    static constexpr bool kHeld = kN == 128;                            // K tiles held in TMEM
    static constexpr int NS = kHeld ? 3 : 4;                            // S buffers
    static constexpr int NTHREADS = kTwo ? 416 : 384;
    static constexpr uint32_t REGS_LOW = 96, REGS_HIGH = 200;
    static constexpr int RING = 4;
    static constexpr uint32_t K_OFF = 0;
    static constexpr uint32_t Q_OFF = NK * TILE_BYTES;
    static constexpr uint32_t L_OFF = Q_OFF + NQ * Q_BYTES;             // [NL]: -LSE log2(e) of 128 columns, and
    static constexpr uint32_t L_SLOT = 128 * 4 + 16;                    // a bit for each that is NaN
    static constexpr uint32_t RING_OFF = L_OFF + NL * L_SLOT;
    static constexpr uint32_t BAR_OFF = RING_OFF + RING * 32;
    static constexpr int B_KFULL = 0, B_KEMPTY = NK, B_QFULL = 2 * NK, B_QEMPTY = B_QFULL + NQ,
                         B_LFULL = B_QEMPTY + NQ, B_LEMPTY = B_LFULL + NL, B_SFULL = B_LEMPTY + NL, B_SEMPTY = B_SFULL + NS, B_TFULL = B_SEMPTY + NS, B_MMADONE = B_TFULL + 2,
                         B_UNIT = B_MMADONE + 1, B_FREE = B_UNIT + RING, NBAR = B_FREE + RING;
    // Arrivals that complete a phase: LSEs read by the 8 group warps, S read and K
    // moved to TMEM by a group's, units taken by the producers, MMA issuer and groups.
    __device__ static uint32_t arrivals(int i) {
        return (kHeld && i >= B_KEMPTY && i < B_QFULL) ? 4u : i >= B_LEMPTY && i < B_SFULL ? 8u : i >= B_SEMPTY && i < B_MMADONE ? 4u
               : i >= B_FREE ? (kTwo ? 12u : 11u) : 1u;
    }
    static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr uint32_t SMEM_BYTES = MISC_OFF + 16 + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t COL_S = kHeld ? 128u : 0u;                // S buffers (K tile x: column 64 x)
};

struct __align__(16) ScoresUnit {
    int k0;             // first token of the pair; -1: no more units
    int n, q0, m;       // cached tokens, first packed row, new tokens
    int qa, qb;         // Q tiles that see any of the pair's tokens
    int b, h;
};
static_assert(sizeof(ScoresUnit) == 32, "unit ring");

template <int D, bool kBF16, int kN>
__global__ void __launch_bounds__(kN == 32 ? 416 : 384, 1)
fa_paged_scores_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const PagedArgs a, const float *in, float *out, const int L, const int R) {
    using C = ScoresCfg<D, kBF16, kN>;
    constexpr uint32_t idesc = idesc_f16(128, kN, kBF16, false, false);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return base + C::BAR_OFF + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gbase + C::MISC_OFF);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + C::MISC_OFF + 4);
    ScoresUnit *ring = reinterpret_cast<ScoresUnit *>(gbase + C::RING_OFF);

    if (warp == 9) tmem_alloc(base + C::MISC_OFF, C::TMEM_COLS);
    if (tid == 0) *abort_flag = 0u;
    if (warp == 11) {
        for (int i = lane; i < C::NBAR; i += 32) mbar_init(bar(i), C::arrivals(i));
        fence_barrier_init();
    }
    if (tid == 8 * 32) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
    }
    // The rows of the Q tiles that no box fills are columns of the product:
    // zeros there keep the scores finite, and a log-sum-exp of +inf their
    // terms zero.
    const int box_rows = R * a.group;
    for (int i = tid; i < C::NQ * C::NCH * (kN - box_rows) * 8; i += C::NTHREADS) {
        const int chunk = i / ((kN - box_rows) * 8), r = i % ((kN - box_rows) * 8);
        *reinterpret_cast<uint4 *>(gbase + C::Q_OFF + chunk * C::Q_CHUNK + box_rows * 128 + r * 16) =
            make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    auto take = [&](uint32_t i, const WaitCtx &w, uint32_t where, ScoresUnit &u) __attribute__((always_inline)) -> bool {
        const uint32_t q = i % C::RING;
        if (!mbar_wait_warp(bar(C::B_UNIT + q), (i / C::RING) & 1u, w, where)) return false;
        u = ring[q];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_FREE + q));
        return u.k0 >= 0;
    };

    if (warp >= 8) {
      if constexpr (!C::kTwo) regs_shrink<C::REGS_LOW>();
      if (warp == 10) {
        // =================== scheduler (whole warp) ===================
        WaitCtx w{abort_flag, a.status, kRolePaged};
        uint32_t sent = 0;
        bool ok = true;
        auto post = [&](const ScoresUnit &u) __attribute__((always_inline)) {
            const uint32_t q = sent % C::RING;
            ok = mbar_wait_idle(bar(C::B_FREE + q), ((sent / C::RING) & 1u) ^ 1u, w, 30);
            if (ok && lane == 0) {
                ring[q] = u;
                mbar_arrive(bar(C::B_UNIT + q));
            }
            __syncwarp();
            ++sent;
        };
        // lane l holds sequence b0 + l; units [first, end) of the window
        int b0 = -32;
        long long end = 0, incl = 0;
        PagedSeq s{0, 0, 0, false};
        long long u = blockIdx.x, st = 2ll * gridDim.x - 1 - 2ll * blockIdx.x;
        while (ok) {
            while (u >= end && b0 + 32 < a.B) {
                b0 += 32;
                s = PagedSeq{0, 0, 0, false};
                if (b0 + lane < a.B) s = paged_seq(a.cu_q, a.kv_len, b0 + lane, a.T, a.W, a.ps_log2);
                if (blockIdx.x == 0) {
                    if (s.bad) report_bad_index(a.status, 1);
                    if (s.n > L) report_bad_index(a.status, 3);
                }
                if (s.bad) s.m = 0;                       // what its rows would see is unknown: its weights stay
                incl = static_cast<long long>((min(s.n, L) + 255) >> 8) * a.H_kv;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                incl += end;
                end = __shfl_sync(0xffffffffu, incl, 31);
            }
            if (u >= end) break;
            const int l = __ffs(__ballot_sync(0xffffffffu, incl > u)) - 1;
            ScoresUnit o;
            o.n = __shfl_sync(0xffffffffu, s.n, l);
            o.q0 = __shfl_sync(0xffffffffu, s.q0, l);
            o.m = __shfl_sync(0xffffffffu, s.m, l);
            o.b = b0 + l;
            const int pairs = (min(o.n, L) + 255) >> 8;
            const long long r = u - (__shfl_sync(0xffffffffu, incl, l) - static_cast<long long>(pairs) * a.H_kv);
            o.h = static_cast<int>(r / pairs);
            o.k0 = static_cast<int>(r - static_cast<long long>(o.h) * pairs) * 256;
            // Q tiles t (positions [t R, t R + R) of the new tokens) that see a
            // token of [k0, k0 + 256): from the first whose last row reaches k0,
            // to the last whose first row's window still holds one
            const int old = o.n - o.m;
            const int tiles = (o.m + R - 1) / R;
            o.qa = 0;
            if (a.wr >= 0) {
                const long long need = static_cast<long long>(o.k0) - a.wr - old;   // first row with hi > k0
                o.qa = need <= 0 ? 0 : static_cast<int>(min(need / R, static_cast<long long>(tiles)));
            }
            o.qb = tiles;
            if (a.wl >= 0 && o.k0 >= a.first) {
                const long long last = static_cast<long long>(o.k0) + 255 + a.wl - old;   // last row with lo <= k0 + 255
                o.qb = last < 0 ? 0 : static_cast<int>(min(last / R + 1, static_cast<long long>(tiles)));
            }
            post(o);
            u += st;
            st = 2ll * gridDim.x - st;
        }
        if (ok) {
            ScoresUnit stop{};
            stop.k0 = -1;
            post(stop);
        }
      } else if (warp == 8 || warp == 12) {
        // =================== TMA producers (whole warps) ===================
        // K tile x of every unit for x in [xa, xb), each group's in a ring of its
        // own, and (warp 8) the Q tiles
        WaitCtx w{abort_flag, a.status, kRoleProducer};
        const int xa = warp == 12 ? 1 : 0, xb = warp == 12 || !C::kTwo ? 2 : 1;
        const PagedBox<C::NCH> bx(a.ps_log2);
        const uint32_t q_bytes = static_cast<uint32_t>(a.group * R) * 128u * C::NCH;
        uint32_t kc0 = 0, kc1 = 0, qc = 0, ui = 0;
        uint32_t qarmed = 0, qarmed_par = 0, armed = 0, armed_par = 0;
        bool ok = true;
        // page ids of a unit's tiles, read while the unit before it loads
        auto page_of = [&](const ScoresUnit &u, int x) __attribute__((always_inline)) -> int {
            const int j = (u.k0 >> 7) + x, vhi = paged_hi(u.n - 1, u.n, a.wr);
            if (u.qa >= u.qb || !bx.needs(j, paged_lo(u.n - u.m, a.wl), vhi, min(a.first, vhi))) return a.n_pages;
            return a.table[static_cast<long long>(u.b) * a.W + ((j * 128 + bx.row) >> a.ps_log2)];
        };
        ScoresUnit u, nx;
        bool more = take(ui++, w, 31, u);
        int page[2] = {0, 0};
        if (more) { page[0] = page_of(u, 0); page[1] = page_of(u, 1); }
        for (; ok && more; u = nx) {
            const int mine[2] = {page[0], page[1]};
            more = take(ui++, w, 31, nx);
            if (more) { page[0] = page_of(nx, 0); page[1] = page_of(nx, 1); }
            if (u.qa >= u.qb) continue;                   // no row sees the pair
            const int nk = u.k0 + 128 < min(u.n, L) ? 2 : 1;
#pragma unroll 1
            for (int x = xa; x < min(xb, nk) && ok; ++x) {
                const int j = (u.k0 >> 7) + x;
                int pg = x ? mine[1] : mine[0];
                if (static_cast<unsigned>(pg) >= static_cast<unsigned>(a.n_pages)) {
                    const int vhi = paged_hi(u.n - 1, u.n, a.wr);
                    if (bx.needs(j, paged_lo(u.n - u.m, a.wl), vhi, min(a.first, vhi))) report_bad_index(a.status, 2);
                    pg = a.n_pages;                       // beyond the pool: zeros
                }
                const uint32_t kc = x ? kc1 : kc0;
                const uint32_t slot = x * C::NKX + kc % C::NKX, ph = (kc / C::NKX) & 1u;
                ok = mbar_wait_warp(bar(C::B_KEMPTY + slot), ph ^ 1u, w, 2);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::B_KFULL + slot), C::TILE_BYTES);
                __syncwarp();
                if (lane < bx.n_box)
                    tma_load_4d(&tm_k, base + C::K_OFF + slot * C::TILE_BYTES + bx.c * C::CHUNK_BYTES + bx.row * 128u,
                                bar(C::B_KFULL + slot), bx.c * 64, u.h,
                                (j * 128 + bx.row) & ((1 << a.ps_log2) - 1), pg);
                armed |= 1u << slot;
                armed_par = (armed_par & ~(1u << slot)) | (ph << slot);
                if (x) ++kc1; else ++kc0;
            }
#pragma unroll 1
            for (int t = u.qa; t < u.qb && ok && warp == 8; ++t, ++qc) {
                const uint32_t slot = qc % C::NQ, ph = (qc / C::NQ) & 1u;
                ok = mbar_wait_warp(bar(C::B_QEMPTY + slot), ph ^ 1u, w, 1);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(bar(C::B_QFULL + slot), q_bytes);
                __syncwarp();
                if (lane < C::NCH)
                    tma_load_4d(&tm_q, base + C::Q_OFF + slot * C::Q_BYTES + lane * C::Q_CHUNK,
                                bar(C::B_QFULL + slot), lane * 64, u.h * a.group, u.q0 + t * R, 0);
                qarmed |= 1u << slot;
                qarmed_par = (qarmed_par & ~(1u << slot)) | (ph << slot);
            }
        }
        for (int s = 0; s < C::NK; ++s)
            if (armed & (1u << s)) mbar_wait_quiet(bar(C::B_KFULL + s), (armed_par >> s) & 1u, 500000000ull);
        for (int s = 0; s < C::NQ; ++s)
            if (qarmed & (1u << s)) mbar_wait_quiet(bar(C::B_QFULL + s), (qarmed_par >> s) & 1u, 500000000ull);
        __syncwarp();
      } else if (warp == 11) {
        // =================== log-sum-exps (whole warp) ===================
        // -LSE log2(e) of a Q tile's rows, -inf (a term of zero) for columns
        // that are none, rows that see nothing and NaN, whose bits follow; read a
        // tile ahead.
        WaitCtx w{abort_flag, a.status, kRoleProducer};
        uint32_t qc = 0, ui = 0;
        bool ok = true;
        constexpr int kEach = kN / 32;
        int pos[kEach], head[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            pos[i] = (lane + 32 * i) / a.group;
            head[i] = (lane + 32 * i) % a.group;
        }
        auto read = [&](const ScoresUnit &u, int t, float (&v)[kEach]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int row = t * R + pos[i];
                v[i] = -INFINITY;
                if (pos[i] < R && t < u.qb && row < u.m)
                    v[i] = a.lse[static_cast<size_t>(u.h * a.group + head[i]) * a.T + u.q0 + row];
            }
        };
        ScoresUnit u, nx;
        float val[kEach], val_n[kEach];
        bool more = take(ui++, w, 33, u);
        if (more) read(u, u.qa, val);
        while (ok && more) {
            more = take(ui++, w, 33, nx);
            if (more) read(nx, nx.qa, val_n);
            for (int t = u.qa; t < u.qb; ++t, ++qc) {
                const uint32_t slot = qc % C::NL, ph = (qc / C::NL) & 1u;
                float cur[kEach];
#pragma unroll
                for (int i = 0; i < kEach; ++i) cur[i] = val[i];
                read(u, t + 1, val);
                ok = mbar_wait_warp(bar(C::B_LEMPTY + slot), ph ^ 1u, w, 3);
                if (!ok) break;
                float *nl = reinterpret_cast<float *>(gbase + C::L_OFF + slot * C::L_SLOT);
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const bool nan = cur[i] != cur[i];
                    nl[lane + 32 * i] = cur[i] == -INFINITY || nan ? -INFINITY : cur[i] * -1.44269504088896340736f;
                    const unsigned bits = __ballot_sync(0xffffffffu, nan);
                    if (lane == i) reinterpret_cast<uint32_t *>(nl)[128 + i] = bits;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_LFULL + slot));
            }
            u = nx;
#pragma unroll
            for (int i = 0; i < kEach; ++i) val[i] = val_n[i];
        }
        __syncwarp();
      } else {
        // =================== MMA issuer (whole warp, one elected lane issues) ===================
        WaitCtx w{abort_flag, a.status, kRoleMma};
        auto uniform = [](int v) __attribute__((always_inline)) -> int { return __shfl_sync(0xffffffffu, v, 0); };
        uint32_t ks = 0, kph = 0, k1 = C::NKX, k1ph = 0, qs = 0, qph = 0, ui = 0;   // slots and their phases
        uint32_t sb = 0, sph = 0, tph = 0;                 // S buffer(s), their phases, bit x: phase of K tile x in TMEM
        bool ok = true;
        ScoresUnit u;
        while (ok && take(ui, w, 32, u)) {
            ++ui;
            const int tiles = uniform(u.qb - u.qa);
            if (tiles <= 0) continue;
            const int nk = uniform(u.k0 + 128 < min(u.n, L) ? 2 : 1);
#pragma unroll 1
            for (int t = 0; t < tiles && ok; ++t) {
                ok = mbar_wait_warp(bar(C::B_QFULL + qs), qph, w, 14);
                const uint64_t qd = smem_desc_sw128(base + C::Q_OFF + qs * C::Q_BYTES, 16u, 1024u);
#pragma unroll 1
                for (int x = 0; x < (C::kHeld ? 2 : nk) && ok; ++x) {
                    // held: the buffers in turn, and group 1's turn comes even if it has no tile
                    const uint32_t b = C::kHeld ? sb : 2 * x + ((sb >> x) & 1u);
                    if (t == 0 && x < nk)
                        ok = C::kHeld ? mbar_wait_warp(bar(C::B_TFULL + x), (tph >> x) & 1u, w, 13)
                                      : mbar_wait_warp(bar(C::B_KFULL + (x ? k1 : ks)), x ? k1ph : kph, w, 13);
                    if (ok) ok = mbar_wait_warp(bar(C::B_SEMPTY + b), ((sph >> b) & 1u) ^ 1u, w, 11);
                    if (!ok) break;
                    sph ^= 1u << b;
                    if (!C::kHeld) sb ^= 1u << x;
                    else if (++sb == C::NS) sb = 0;
                    tc_fence_after();
                    const uint32_t d_s = tbase + C::COL_S + 128u * b;
                    if constexpr (C::kHeld) {
                        if (x < nk) {
                            const uint32_t tK = tbase + 64u * x;
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t qo = ((kk >> 2) * C::Q_CHUNK + (kk & 3) * 32u) >> 4;
                                mma_ts_f16_elect(d_s, tK + kk * 8u, qd + qo, idesc, kk > 0 ? 1u : 0u);
                            }
                        }
                    } else {
                        const uint64_t kd = smem_desc_sw128(base + C::K_OFF + (x ? k1 : ks) * C::TILE_BYTES, 16u, 1024u);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t ko = ((kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32u) >> 4;
                            const uint32_t qo = ((kk >> 2) * C::Q_CHUNK + (kk & 3) * 32u) >> 4;
                            mma_ss_f16_elect(d_s, kd + ko, qd + qo, idesc, kk > 0 ? 1u : 0u);
                        }
                    }
                    mma_commit_elect(bar(C::B_SFULL + b));
                }
                if (!ok) break;
                mma_commit_elect(bar(C::B_QEMPTY + qs));
                if (++qs == C::NQ) { qs = 0; qph ^= 1u; }
            }
            if (!ok) break;
            tph ^= nk == 2 ? 3u : 1u;
            if (!C::kHeld) mma_commit_elect(bar(C::B_KEMPTY + ks));
            if (++ks == C::NKX) { ks = 0; kph ^= 1u; }
            if (nk == 2) {
                if (!C::kHeld) mma_commit_elect(bar(C::B_KEMPTY + k1));
                if (++k1 == C::NK) { k1 = C::NKX; k1ph ^= 1u; }
            }
        }
        mma_commit_elect(bar(C::B_MMADONE));
        mbar_wait_quiet(bar(C::B_MMADONE), 0, 500000000ull);
        __syncwarp();
      }
    } else {
        if constexpr (!C::kTwo) regs_grow<C::REGS_HIGH>();
        // =================== group x: one cached token a thread ===================
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        WaitCtx w{abort_flag, a.status, x ? kRoleSoftmax1 : kRoleSoftmax0};
        const float sl2 = a.scale_log2;
        const float2 c2 = make_float2(sl2, sl2);
        uint32_t ui = 0, ls = 0, lph = 0;                  // units; LSE slot and its phase
        uint32_t sb = C::kHeld ? x : 2 * x, sph = 0, kc = 0;   // S buffer and its phase; K tiles
        bool ok = true;
        ScoresUnit u;
        while (ok && take(ui, w, 24, u)) {
            ++ui;
            const int kk = u.k0 + x * 128 + row;                             // this thread's token
            const int end = min(u.n, L);                                     // no room for tokens behind it
            const bool none = u.k0 + x * 128 >= end;                         // the group has no tile of this unit
            const int old = u.n - u.m;
            const size_t at = (static_cast<size_t>(u.b) * a.H_kv + u.h) * L + kk;
            const float had = in != nullptr && kk < min(old, end) ? in[at] : 0.f;
            // rows [ra, rb) of the new tokens see this one
            const long long ra = a.wr >= 0 ? static_cast<long long>(kk) - a.wr - old : 0;
            const long long rb = a.wl >= 0 && kk >= a.first ? static_cast<long long>(kk) + a.wl - old + 1 : u.m;
            const int r0 = static_cast<int>(min(max(ra, 0ll), static_cast<long long>(u.m)));
            const int r1 = static_cast<int>(min(max(rb, 0ll), static_cast<long long>(u.m)));
            float sum = 0.f;
            // the next Q tile's LSEs and (if the group has a tile) scores are there
            auto arrived = [&]() __attribute__((always_inline)) -> bool {
                if (!mbar_wait_warp(bar(C::B_LFULL + ls), lph, w, 19)) return false;
                if (none && !C::kHeld) return true;
                if (!mbar_wait_warp(bar(C::B_SFULL + sb), sph, w, 20)) return false;
                tc_fence_after();
                return true;
            };
            bool odd = false;                              // (held) the key is not finite and there are columns that are none
            if (C::kHeld && !none && u.qa < u.qb) {
                // this token's key into TMEM (every product with the group's last one
                // is complete: its last scores are read)
                const uint32_t ks = x * C::NKX + kc % C::NKX;
                ok = mbar_wait_warp(bar(C::B_KFULL + ks), (kc / C::NKX) & 1u, w, 18);
                if (!ok) break;
                ++kc;
                const uint8_t *kr = gbase + C::K_OFF + ks * C::TILE_BYTES + row * 128;
                uint32_t top = 0u;                         // the largest magnitudes, in halves
#pragma unroll
                for (int ch = 0; ch < C::NCH; ++ch) {
                    uint32_t kw[32];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint4 v4 = *reinterpret_cast<const uint4 *>(kr + ch * C::CHUNK_BYTES + ((q ^ (row & 7)) << 4));
                        kw[4 * q] = v4.x; kw[4 * q + 1] = v4.y; kw[4 * q + 2] = v4.z; kw[4 * q + 3] = v4.w;
                    }
                    tmem_st32(tbase + lane_off + 64u * x + 32u * ch, kw);
                    if (box_rows != kN) {
#pragma unroll
                        for (int q = 0; q < 32; ++q) top = __vmaxu2(top, kw[q] & 0x7fff7fffu);
                    }
                }
                constexpr uint32_t kInf = kBF16 ? 0x7f80u : 0x7c00u;
                odd = max(top & 0xffffu, top >> 16) >= kInf;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::B_KEMPTY + ks));
                    mbar_arrive(bar(C::B_TFULL + x));
                }
            }
#pragma unroll 1
            for (int t = u.qa; t < u.qb; ++t) {
                ok = arrived();
                if (!ok) break;
                const uint32_t slot = ls, buf = sb;
                if (++ls == C::NL) { ls = 0; lph ^= 1u; }
                if (C::kHeld || !none) {
                    if (C::kHeld) sb += 2;
                    else sb ^= 1u;
                    if (C::kHeld ? sb >= C::NS : (sb & 1u) == 0) { if (C::kHeld) sb -= C::NS; sph ^= 1u; }
                }
                if (none) {
                    if (lane == 0) mbar_arrive(bar(C::B_LEMPTY + slot));
                    if (C::kHeld && lane == 0) mbar_arrive(bar(C::B_SEMPTY + buf));
                    continue;
                }
                uint32_t v[kN];
#pragma unroll
                for (int c = 0; c < kN; c += 32)
                    tmem_ld32(tbase + lane_off + C::COL_S + 128u * buf + c,
                              *reinterpret_cast<uint32_t(*)[32]>(&v[c]));
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_SEMPTY + buf));   // the scores are read
                // columns [ca, cb) see this token
                const int ca = min(max(r0 - t * R, 0), R) * a.group;
                const int cb = min(max(r1 - t * R, 0), R) * a.group;
                if (__any_sync(0xffffffffu, ca != 0 || cb != box_rows || odd)) {
                    // hidden columns: a score of -inf (what lies there may be anything;
                    // in a column that is none, an infinite key times its zeros)
#pragma unroll
                    for (int c = 0; c < kN; ++c)
                        if (c < ca || c >= cb) v[c] = 0xff800000u;
                }
                const float4 *l4 = reinterpret_cast<const float4 *>(gbase + C::L_OFF + slot * C::L_SLOT);
                uint4 nan = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (kN == 32) nan.x = reinterpret_cast<const uint32_t *>(l4)[128];
                else nan = reinterpret_cast<const uint4 *>(l4)[32];
                float2 e_a, e_b;
                float ts;
#pragma unroll 1
                for (bool again = false;; again = true) {
                    e_a = make_float2(0.f, 0.f);
                    e_b = e_a;
#pragma unroll
                    for (int c = 0; c < kN; c += 4) {
                        const float4 l = l4[c / 4];
                        const float2 x01 = __ffma2_rn(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])),
                                                      c2, make_float2(l.x, l.y));
                        const float2 x23 = __ffma2_rn(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])),
                                                      c2, make_float2(l.z, l.w));
                        e_a = __fadd2_rn(e_a, make_float2(ex2_approx(x01.x), ex2_approx(x01.y)));
                        e_b = __fadd2_rn(e_b, make_float2(ex2_approx(x23.x), ex2_approx(x23.y)));
                    }
                    ts = (e_a.x + e_a.y) + (e_b.x + e_b.y);
                    // (keys in shared memory) NaN, maybe of such a column: once more without them
                    if (C::kHeld || again || box_rows == kN || !__any_sync(0xffffffffu, ts != ts)) break;
#pragma unroll
                    for (int c = 0; c < kN; ++c)
                        if (c >= cb) v[c] = 0xff800000u;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_LEMPTY + slot));
                sum += ts;
                if ((nan.x | nan.y | nan.z | nan.w) != 0u) {
                    auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
                    auto sees = [&](int c) -> uint32_t { return below(cb - c) & ~below(ca - c); };
                    if ((nan.x & sees(0)) | (nan.y & sees(32)) | (nan.z & sees(64)) | (nan.w & sees(96)))
                        sum = __int_as_float(0x7fc00000);
                }
            }
            if (!ok) break;
            if (kk < end) out[at] = had + sum;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
}

template <int D, bool kBF16, int kN>
static cudaError_t launch_scores_inst(const PagedScoresLaunch &L) {
    using C = ScoresCfg<D, kBF16, kN>;
    auto kern = fa_paged_scores_kernel<D, kBF16, kN>;
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
    kern<<<L.grid, C::NTHREADS, C::SMEM_BYTES, L.stream>>>(L.q, L.k, L.a, L.in, L.out, L.L, L.R);
    return cudaGetLastError();
}

// Up to 32 rows a Q tile the narrow form: 64 sequences of 4 tokens on up to 8192 103 us
// (the other 154), of 8 tokens 103 (153), one of 4 tokens on 777 6.7 (8.2).
template <int D>
static cudaError_t launch_scores_dispatch(const PagedScoresLaunch &L) {
    if (L.R * L.a.group <= 32)
        return L.bf16 ? launch_scores_inst<D, true, 32>(L) : launch_scores_inst<D, false, 32>(L);
    return L.bf16 ? launch_scores_inst<D, true, 128>(L) : launch_scores_inst<D, false, 128>(L);
}

cudaError_t launch_paged_scores(const PagedScoresLaunch &L) {
    return L.d == 64 ? launch_scores_dispatch<64>(L) : launch_scores_dispatch<128>(L);
}

}  // namespace fa
