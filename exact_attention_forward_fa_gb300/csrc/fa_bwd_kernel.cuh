// fa_bwd_kernel.cuh -- gradients of exact attention (dQ, dK, dV) on sm_103a.
//
// "FlashAttention-3 on Hopper", ch. 7 (the backward pass):
//   sec. 7.1   S = alpha Q K^T, P = softmax(S) recomputed from the forward's
//              LSE as P = exp2(S alpha log2e - LSE log2e) (no running max:
//              the exponent is log P <= 0); dV = P^T dO; dP = dO V^T;
//              dS = P o (dP - D) with D_i = rowsum(dO_i o O_i);
//              dQ = alpha dS K; dK = alpha dS^T Q.
//   sec. 7.2   KV-parallel ownership for dK, dV (a CTA owns one key tile and
//              visits the query tiles; causal: from the diagonal on).  Of
//              the section's three ways to produce dQ across key tiles, this
//              file takes the first: a second, query-parallel kernel that
//              recomputes S and dP for its query tile and accumulates dQ in
//              TMEM.  On GB300 the KV-parallel kernel's TMEM is full with
//              S^T, dP^T, dV and dK at d = 128 (512 columns) and its shared
//              memory with K, V and two Q/dO stages, so a dQ accumulator or
//              an FP32 dQ staging tile has no room; the second kernel needs
//              no atomics, no FP32 workspace and gives identical bits on
//              every run.
//   sec. 7.3   the preprocessing pass computes D.
//
// Operand rings are per tensor, so the tile the MMA warp needs next lands in
// a slot freed well before (dQ kernel: K ring of 3, V ring of 2 at d = 128;
// dK/dV kernel: Q ring of 3, dO ring of 2).  The preprocess writes D and
// LSE*log2(e) into a workspace padded to whole 128-row tiles (padding: D = 0,
// LSE2 = +inf, which zero P), read by the elementwise warps through L1.
//
// Both main kernels: 320 threads -- warps 0-7 the elementwise group, warp 8
// the TMA producer, warp 9 the MMA issuer (converged warp, elected lane).
// The backward's elementwise work has no row reduction (P comes from LSE,
// dS is pointwise), so two warps share each TMEM lane quarter (one thread
// per tile row) and split the 128 columns: warp w takes lanes
// 32 (w mod 4) .. +31 and columns 64 (w / 4) .. +63.  All GEMMs are tcgen05.mma
// kind::f16 with FP32 accumulation in TMEM; P and dS are rounded to the
// input's 16-bit type for the GEMMs that consume them.  Every mbarrier wait
// is bounded and reports through the device status word.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_device.cuh"
#include "fa_mask.cuh"

namespace fa {

struct BwdArgs {
    const float *lse;      // [B][H][N], natural log, from the forward
    float *ws_d;           // [B][H][NP] D_i = rowsum(dO_i o O_i); 0 for n >= N
    float *ws_l;           // [B][H][NP] LSE_i log2(e); +inf for n >= N and empty rows
    const void *o;         // [B][N][H][d] forward output (preprocess only)
    const void *dout;      // [B][N][H][d] upstream gradient (preprocess only)
    void *dq, *dk, *dv;    // [B][N][H][d] outputs, input dtype
    uint32_t *status;
    int B, H, N;
    int n_t;               // 128-row tiles per sequence
    int NP;                // n_t * 128: padded row count of the workspace
    int n_units;           // B * H * n_t (dQ kernel: query tiles)
    int n_units_kv;        // B * (H / group) * n_t (dK/dV kernel: key tiles)
    int group;             // query heads per K/V head (>= 1); K/V are [B][N][H/group][d]
    float scale_log2;      // alpha * log2(e)
    float alpha;
    // Local window (kWin instantiations): key j is hidden from query i when
    // j > i + wr (wr >= 0) or j < i - wl (wl >= 0); -1 is no bound.  Causal
    // without a window: both main kernels take their units in the dynamic
    // order of the forward (make_bwd_unit), whose groups hold chunk heads;
    // chunk shares wl's storage (the two never meet in one launch).
    union {
        int wl;
        int chunk;
    };
    int wr;
    // Softcap c (kCap instantiations): the score is c tanh(alpha s / c),
    // t = tanh(sc_pre s) with sc_pre = alpha / c, in log2 units sc_post t
    // with sc_post = c log2(e); dS picks up the factor 1 - t^2.
    float sc_pre, sc_post;
    // Interval masks (kMask instantiations): the plan's lists and intervals;
    // kBias: the score loses slopes[h] |i - j|.  chunk as for causal units.
    MaskPlan plan;
    const float *slopes;
    // Interval masks in fp16 (kScale): V's tokens for the bound of dS, and the CTAs
    // that form it
    const void *v;
    long long v_stride;
    int parts;
    float *dsinks;         // 2^-e goes there (or NULL), for the sinks' gradient
};

// Visible keys [win_klo, win_khi) of query row i (0 <= i < N), and visible
// queries [win_qlo, win_qhi) of key row j (0 <= j < N), under (wl, wr).
// Written with min() so no intermediate leaves [0, N].
__device__ __forceinline__ int win_klo(int i, const BwdArgs &a) {
    return a.wl >= 0 ? i - min(a.wl, i) : 0;
}
__device__ __forceinline__ int win_khi(int i, const BwdArgs &a) {
    return a.wr >= 0 ? i + 1 + min(a.wr, a.N - 1 - i) : a.N;
}
__device__ __forceinline__ int win_qlo(int j, const BwdArgs &a) {
    return a.wr >= 0 ? j - min(a.wr, j) : 0;
}
__device__ __forceinline__ int win_qhi(int j, const BwdArgs &a) {
    return a.wl >= 0 ? j + 1 + min(a.wl, a.N - 1 - j) : a.N;
}
// 128-row tile range [lo, hi) covering rows [r_lo, r_hi) (r_hi > r_lo).
__device__ __forceinline__ int tile_lo(int r_lo) { return r_lo >> 7; }
__device__ __forceinline__ int tile_hi(int r_hi) { return (r_hi >> 7) + ((r_hi & 127) != 0); }

template <int D, bool kBF16>
struct BwdCfg {
    static_assert(D == 64 || D == 128, "head dim");
    static constexpr int NCH = D / 64;                   // 128-byte column chunks
    static constexpr uint32_t CHUNK = 128u * 128u;       // 128 rows x 128 B
    static constexpr uint32_t TILE = NCH * CHUNK;        // one 128 x D tile
    static constexpr int NTHREADS = 320;
    static constexpr int N_EW = 8;                        // elementwise warps
    static constexpr int CLC_DEPTH = 4;                   // causal: answers in flight
    static constexpr uint32_t TMEM_COLS = 512;
    // S = Q K^T style: both operands K-major, M = N = 128
    static constexpr uint32_t IDESC_SS = idesc_f16(128, 128, kBF16, false, false);
    // (.) x B with B MN-major, N = D (P V style)
    static constexpr uint32_t IDESC_ACC = idesc_f16(128, D, kBF16, false, true);
    static constexpr int QK_STEPS = D / 16;              // K = D in steps of 16
    static constexpr int ACC_STEPS = 128 / 16;           // K = 128 rows in steps of 16

    // ---- dQ kernel: Q, dO resident per unit; a K ring and a V ring ----
    static constexpr int KN = D == 128 ? 3 : 6, VN = D == 128 ? 2 : 5;
    static constexpr uint32_t DQ_Q_OFF = 0, DQ_DO_OFF = TILE, DQ_K_OFF = 2 * TILE,
                              DQ_V_OFF = DQ_K_OFF + KN * TILE;
    static constexpr uint32_t DQ_BAR_OFF = DQ_V_OFF + VN * TILE;
    static constexpr int DQB_QFULL = 0, DQB_QEMPTY = 1, DQB_SFULL = 2, DQB_DPFULL = 3,
                         DQB_SFREE = 4, DQB_DSFULL = 5 /* x2 */, DQB_DQFULL = 7,
                         DQB_DQEMPTY = 8, DQB_MMADONE = 9, DQB_KFULL = 10,
                         DQB_KEMPTY = DQB_KFULL + KN, DQB_VFULL = DQB_KEMPTY + KN,
                         DQB_VEMPTY = DQB_VFULL + VN,
                         // causal: the dynamic order's answers (see the kernel)
                         DQB_CLCFULL = DQB_VEMPTY + VN, DQB_UNIT = DQB_CLCFULL + 4,
                         DQB_CLCEMPTY = DQB_UNIT + 4, DQ_NBAR = DQB_CLCEMPTY + 4;
    static constexpr uint32_t DQ_MISC_OFF = DQ_BAR_OFF + DQ_NBAR * 8;
    static constexpr uint32_t DQ_CLC_OFF = (DQ_MISC_OFF + 16 + 15) & ~15u;   // 16-byte aligned
    static constexpr uint32_t DQ_UNIT_OFF = DQ_CLC_OFF + 4 * 16;
    static constexpr uint32_t DQ_REC_OFF = (DQ_UNIT_OFF + 4 * 4 + 15) & ~15u;   // interval masks: BwdRec per answer
    static constexpr uint32_t DQ_SMEM = DQ_REC_OFF + 4 * 32 + 1024;
    // TMEM: S [0,128), dP [128,256), dQ [256,256+D), dS0, dS1 (64 columns each)
    static constexpr uint32_t DQ_COL_S = 0, DQ_COL_DP = 128, DQ_COL_DQ = 256,
                              DQ_COL_DS = 256 + D;
    static_assert(DQ_COL_DS + 128 <= TMEM_COLS, "dQ kernel TMEM budget");

    // ---- dK/dV kernel: K, V resident per unit; a Q ring and a dO ring ----
    static constexpr int QN = D == 128 ? 3 : 6, DN = D == 128 ? 2 : 5;
    static constexpr uint32_t KV_K_OFF = 0, KV_V_OFF = TILE, KV_Q_OFF = 2 * TILE,
                              KV_DO_OFF = KV_Q_OFF + QN * TILE;
    static constexpr uint32_t KV_BAR_OFF = KV_DO_OFF + DN * TILE;
    static constexpr int KVB_KVFULL = 0, KVB_KVEMPTY = 1, KVB_STFULL = 2, KVB_DPTFULL = 3,
                         KVB_PFULL = 4, KVB_DSFULL = 5, KVB_ACCFULL = 6, KVB_ACCEMPTY = 7,
                         KVB_MMADONE = 8, KVB_QFULL = 9, KVB_QEMPTY = KVB_QFULL + QN,
                         KVB_DOFULL = KVB_QEMPTY + QN, KVB_DOEMPTY = KVB_DOFULL + DN,
                         KVB_STFULL1 = KVB_DOEMPTY + DN, KVB_PFULL1 = KVB_STFULL1 + 1,
                         // causal: the dynamic order's answers (see the kernel)
                         KVB_CLCFULL = KVB_PFULL1 + 1, KVB_UNIT = KVB_CLCFULL + 4,
                         KVB_CLCEMPTY = KVB_UNIT + 4, KV_NBAR = KVB_CLCEMPTY + 4;
    static constexpr uint32_t KV_MISC_OFF = KV_BAR_OFF + KV_NBAR * 8;
    static constexpr uint32_t KV_CLC_OFF = (KV_MISC_OFF + 16 + 15) & ~15u;   // 16-byte aligned
    static constexpr uint32_t KV_UNIT_OFF = KV_CLC_OFF + 4 * 16;
    static constexpr uint32_t KV_REC_OFF = (KV_UNIT_OFF + 4 * 4 + 15) & ~15u;   // interval masks: BwdRec per answer
    static constexpr uint32_t KV_SMEM = KV_REC_OFF + 4 * 32 + 1024;
    // TMEM: S^T [0,128) (P^T over its first 64), dP^T [128,256) (dS^T over
    // its first 64), dV [256,256+D), dK [256+D,256+2D); at d = 64 a second
    // S^T buffer [384,512), so the S^T of query tile i+2 is computed while
    // tile i+1's exponentials run (d = 128 fills TMEM with one).
    static constexpr uint32_t KV_COL_ST = 0, KV_COL_DPT = 128, KV_COL_DV = 256,
                              KV_COL_DK = 256 + D, KV_COL_ST1 = 256 + 2 * D;
    static constexpr bool KV_SDB = D == 64;
    static_assert(KV_COL_DK + D <= TMEM_COLS, "dK/dV kernel TMEM budget");
    static_assert(!KV_SDB || KV_COL_ST1 + 128 <= TMEM_COLS, "second S^T buffer");
    // S^T buffer and its full barrier for the n-th S^T tile of the CTA
    __host__ __device__ static constexpr uint32_t st_buf(uint32_t n) { return KV_SDB ? (n & 1u) : 0u; }
    __host__ __device__ static constexpr uint32_t st_col(uint32_t n) {
        return st_buf(n) ? KV_COL_ST1 : KV_COL_ST;
    }
    __host__ __device__ static constexpr int st_bar(uint32_t n) {
        return st_buf(n) ? KVB_STFULL1 : KVB_STFULL;
    }
    // parity of the n-th S^T tile's wait on its barrier (and on p_bar(n))
    __host__ __device__ static constexpr uint32_t st_par(uint32_t n) {
        return KV_SDB ? ((n >> 1) & 1u) : (n & 1u);
    }
    // "P^T of the n-th tile written", one barrier per S^T buffer.  With two
    // buffers, S^T of tile n+1 is ready before the MMA waits for P^T(n), so
    // an elementwise warp can finish tile n and arrive for tile n+1 while
    // another has not yet arrived for tile n.  On a single barrier counting
    // eight arrivals, that early arrival would complete tile n's phase
    // without the late warp; the MMA would then overwrite the late warp's
    // S^T buffer, whose barrier would advance two phases before that warp
    // waited on it (a lost phase: the wait never ends).  Per-buffer
    // barriers keep every phase to one tile.
    __host__ __device__ static constexpr int p_bar(uint32_t n) {
        return st_buf(n) ? KVB_PFULL1 : KVB_PFULL;
    }
    static_assert(DQ_SMEM <= 232448 && KV_SMEM <= 232448, "shared memory");
};

// Work unit: one 128-row tile (queries for dQ, keys for dK/dV) of one (b, h).
// Causal: the longest units first (dQ: the last query tiles; dK/dV: the
// first key tiles).
struct BwdUnit {
    int b, h, m;
    int lo, hi;     // interval masks: key (or query) tiles of the unit
};

// kWin: the window's loop bounds; longest-first when it has a right bound
// and no left one (the causal shape).  Longest-first orders are walked with
// unit_stride0's back-and-forth over the CTAs.
template <bool kCausal, bool kWin>
__device__ __forceinline__ bool bwd_longest_first(const BwdArgs &a) {
    return kWin ? (a.wl < 0 && a.wr >= 0) : kCausal;
}

// Interval masks: a unit as the producer reads it from the plan's lists (the dynamic
// order over tiles sorted longest first) and hands it on through shared memory.
struct BwdRec {
    int4 id;       // u (-1: no more units), b, h, tile
    int4 range;    // its tiles [x, y); z: the sequence has tokens outside documents
};
template <bool kKeyTiles>
__device__ __forceinline__ BwdRec bwd_rec(int u, const BwdArgs &a) {
    const int HH = kKeyTiles ? a.H / a.group : a.H;
    int i, bh;
    dynamic_order(u, a.B * HH, a.n_t, a.chunk, i, bh);
    const int b = bh / HH;
    const int4 *list = kKeyTiles ? a.plan.ktiles : a.plan.qtiles;
    const int4 rec = __ldg(list + static_cast<size_t>(b) * a.n_t + (a.n_t - 1 - i)), lv = __ldg(a.plan.live + b);
    return BwdRec{make_int4(u, b, bh - b * HH, rec.x), make_int4(rec.y, rec.z, lv.x > 0 || lv.y < a.N, 0)};
}
__device__ __forceinline__ BwdUnit bwd_unit(const BwdRec &r) {
    return BwdUnit{r.id.y, r.id.z, r.id.w, r.range.x, r.range.y};
}
__device__ __forceinline__ BwdRec read_bwd_rec(const uint8_t *slots, uint32_t q) {
    const volatile int *v = reinterpret_cast<const volatile int *>(slots) + 8 * q;
    return BwdRec{make_int4(v[0], v[1], v[2], v[3]), make_int4(v[4], v[5], v[6], v[7])};
}

template <bool kCausal, bool kKeyTiles, bool kWin = false>
__device__ __forceinline__ BwdUnit make_bwd_unit(int u, const BwdArgs &a) {
    BwdUnit U;
    const int HH = kKeyTiles ? a.H / a.group : a.H;     // K/V heads for key tiles
    const int BH = a.B * HH;
    U.lo = U.hi = 0;
    int bh;
    if (kCausal && !kWin) {
        // the forward's dynamic order (fa_fwd_kernel.cuh): unit i of a head
        // is its (i+1)-th longest; dQ: query tile i, dK/dV: key tile n_t-1-i
        int i;
        dynamic_order(u, BH, a.n_t, a.chunk, i, bh);
        U.m = kKeyTiles ? a.n_t - 1 - i : i;
    } else if (bwd_longest_first<kCausal, kWin>(a)) {
        const int k = u / BH;
        U.m = kKeyTiles ? k : a.n_t - 1 - k;
        bh = u % BH;
    } else {
        U.m = u % a.n_t;
        bh = u / a.n_t;
    }
    U.b = bh / HH;
    U.h = bh % HH;
    return U;
}

// x / y, in 32 bits where they suffice (a 64-bit division is a hundred instructions).
__device__ __forceinline__ long divide32(long x, int y) {
    return x >> 32 ? x / y : static_cast<long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}

// LSE in log2 units, as the main kernels take it; scale_undo gives back what e took off.
__device__ __forceinline__ float to_log2(float lse) { return __fmul_rn(lse, 1.4426950408889634f); }

// 2^-e for the e of a row whose LSE2 - e is given: the difference is e up to the rounding
// of LSE2 - e, a fourth at most while |LSE2| < 2^22 (beyond, FP32 scores mean little).
__device__ __forceinline__ float scale_undo(float lse, float lse2_less_e) {
    const float d = rintf(__fsub_rn(to_log2(lse), lse2_less_e));
    return d > 0.f && d <= 15.f ? __int_as_float((127 - static_cast<int>(d)) << 23) : 1.f;
}

// The larger of each half and the sizes of eight fp16 values, in packed pairs.
__device__ __forceinline__ uint32_t max_abs_f16(uint32_t m, const uint4 &x) {
    asm("{\n\t.reg .b32 a, b, c, d;\n\t"
        "and.b32 a, %1, 0x7fff7fff;\n\tand.b32 b, %2, 0x7fff7fff;\n\t"
        "and.b32 c, %3, 0x7fff7fff;\n\tand.b32 d, %4, 0x7fff7fff;\n\t"
        "max.f16x2 a, a, b;\n\tmax.f16x2 c, c, d;\n\tmax.f16x2 a, a, c;\n\tmax.f16x2 %0, %0, a;\n\t}"
        : "+r"(m) : "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w));
    return m;
}

// The maxima over a block of 256 threads, in all of them.
__device__ __forceinline__ float2 cta_max(float2 m, float2 (&warps)[8]) {
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, w));
        m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, w));
    }
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = make_float2(fmaxf(m.x, warps[w].x), fmaxf(m.y, warps[w].y));
    return m;
}

// ---------------------------------------------------------------------------
// Preprocess ("FlashAttention-3 on Hopper", sec. 7.1.2, 7.1.3 and 7.3):
//   ws_d[b][h][n] = sum_c dO[b][n][h][c] * O[b][n][h][c]   (FP32)
//   ws_l[b][h][n] = LSE[b][h][n] * log2(e)                  (+inf if empty)
// and the padding rows N <= n < NP get D = 0, LSE2 = +inf.  HBM-bound:
// reads 2 x 2 B per element.  A row of D elements is read by D/8 threads
// with 16-byte loads; each thread handles 4 rows per pass for memory
// parallelism.
// ---------------------------------------------------------------------------
// kMask: rows outside every document may hold anything; their D is 0.
//
// Interval masks in fp16 (kScale).  P and dS = P o (dP - D) are rounded to fp16 for the
// products that consume them, and fp16 is spaced by 2^-24 below 2^-14: P of long
// documents is there (1 / N), and dS falls with N, |dO| and |V| (dO of size 2^-10 and
// N = 4096: dQ off by 0.5 % in its norm).  So P and with it dS are formed 2^e times as
// large, e in [0, 15], with LSE2 - e in the place of LSE2 (no step of the tiles' loops),
// and the gradients are scaled back as they are stored.  P <= 1 and |dP - D| <= 2 d
// max|dO| max|V| (D is a mean of a row's dP): the largest e with 2^e times that below
// 65504 / 1.01.  This kernel forms the maxima a CTA (a NaN drops out, an infinity leaves e
// = 0); fa_bwd_scale_kernel joins them and writes LSE2 - e.  The maxima and e travel in
// dq (8 bytes a CTA and 4; a CTA's rows are 128 bytes of dq at least), which nobody writes
// before the dQ kernel: the dK/dV kernel's CTAs read e before they let that one begin, and
// it has e from LSE2 - e and the LSE.
template <int D, bool kBF16, bool kMask = false>
__global__ void __launch_bounds__(256)
fa_bwd_delta_kernel(const BwdArgs a) {
    constexpr bool kScale = kMask && !kBF16;
    constexpr int TPR = D / 8;                       // threads per row
    constexpr int RPW = 32 / TPR;                    // rows per warp pass
    const long n_rows = static_cast<long>(a.B) * a.N * a.H;
    const int lane = threadIdx.x & 31;
    const long warp_g = (static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const long n_warps = (static_cast<long>(gridDim.x) * blockDim.x) >> 5;
    const int sub = lane / TPR, part = lane % TPR;
    const uint4 *o4 = reinterpret_cast<const uint4 *>(a.o);
    const uint4 *d4 = reinterpret_cast<const uint4 *>(a.dout);
    uint32_t most_o = 0u, most_v = 0u;               // kScale: |dO|, |V|, as pairs
    for (long base = warp_g * RPW * 4; base < n_rows; base += n_warps * RPW * 4) {
        // row = (b * N + n) * H + h: the pass's first one
        const long bn0 = divide32(base, a.H);
        const int h0 = static_cast<int>(base - bn0 * a.H);
        const long b0 = divide32(bn0, a.N);
        const int n0 = static_cast<int>(bn0 - b0 * a.N);
        uint4 ov[4], dv[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const long row = base + r * RPW + sub;
            ov[r] = make_uint4(0u, 0u, 0u, 0u);
            dv[r] = ov[r];
            if (row < n_rows) {
                ov[r] = o4[row * TPR + part];
                dv[r] = d4[row * TPR + part];
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t ow[4] = {ov[r].x, ov[r].y, ov[r].z, ov[r].w};
            const uint32_t dw[4] = {dv[r].x, dv[r].y, dv[r].z, dv[r].w};
            float acc = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = fma_pair<kBF16>(acc, ow[i], dw[i]);
#pragma unroll
            for (int m = TPR / 2; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
            const long row = base + r * RPW + sub;
            if ((kScale || part == 0) && row < n_rows) {
                int h = h0 + r * RPW + sub, n = n0;      // (a few steps on: no division)
                long b = b0;
                while (h >= a.H) {
                    h -= a.H;
                    if (++n == a.N) {
                        n = 0;
                        ++b;
                    }
                }
                if constexpr (kMask) {
                    const int4 lv = __ldg(a.plan.live + b);
                    if (n < lv.x || n >= lv.y) acc = 0.f;
                    else if constexpr (kScale) most_o = max_abs_f16(most_o, dv[r]);
                }
                if (part == 0) a.ws_d[(b * a.H + h) * a.NP + n] = acc;
            }
        }
    }
    if constexpr (kMask) grid_launch_dependents();
    if constexpr (kScale) {
        // V's vectors within the documents, four in flight, then the CTA's maxima
        const int per = a.H / a.group * TPR;         // vectors of a token
        const long n_v = static_cast<long>(a.B) * a.N * per, step = n_warps * 32;
        const uint4 *v4 = reinterpret_cast<const uint4 *>(a.v);
        for (long idx = warp_g * 32 + lane; idx < n_v; idx += 4 * step) {
            uint4 x[4];
            long t[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const long i = idx + r * step;
                t[r] = i < n_v ? divide32(i, per) : -1;
                x[r] = t[r] < 0 ? make_uint4(0u, 0u, 0u, 0u) : v4[t[r] * (a.v_stride / 8) + (i - t[r] * per)];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (t[r] < 0) continue;
                const long b = divide32(t[r], a.N), n = t[r] - b * a.N;
                const int4 lv = __ldg(a.plan.live + b);
                if (n >= lv.x && n < lv.y) most_v = max_abs_f16(most_v, x[r]);
            }
        }
        __shared__ float2 most[8];
        float o0, o1, v0, v1;
        unpack2<false>(most_o, o0, o1);
        unpack2<false>(most_v, v0, v1);
        const float2 m = cta_max(make_float2(fmaxf(o0, o1), fmaxf(v0, v1)), most);
        if (threadIdx.x == 0) reinterpret_cast<float2 *>(a.dq)[blockIdx.x] = m;
    } else {
        const long n_pad = static_cast<long>(a.B) * a.H * a.NP;
        for (long idx = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; idx < n_pad;
             idx += static_cast<long>(gridDim.x) * blockDim.x) {
            const long bh = divide32(idx, a.NP), n = idx - bh * a.NP;
            float l2 = INFINITY;
            if (n < a.N) {
                const float l = a.lse[bh * a.N + n];
                l2 = l == -INFINITY ? INFINITY : to_log2(l);
            } else {
                a.ws_d[idx] = 0.f;
            }
            a.ws_l[idx] = l2;
        }
    }
}

// Joins the maxima (kScale, see above): e for the call, and LSE2 - e.  Measured (GB300, 4 x
// 4096 tokens, 32 heads of 64, documents of 256: 280 us, in bf16 259): V's pass 14 us, at HBM
// speed, this kernel 6; 2 x 8192, 32 heads of 128 over 8, of 1024: 478 and 470 together.
template <int D>
__global__ void __launch_bounds__(256) fa_bwd_scale_kernel(const BwdArgs a) {
    grid_launch_dependents();
    // four rows a thread, in one head: their LSE, an input, ahead of the wait
    const long n4 = static_cast<long>(a.B) * a.H * a.NP / 4, step = static_cast<long>(gridDim.x) * blockDim.x;
    long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
    float l[4];
    auto load = [&]() {
        const long bh = divide32(4 * i, a.NP);
        const int n = static_cast<int>(4 * i - bh * a.NP);
#pragma unroll
        for (int r = 0; r < 4; ++r) l[r] = n + r < a.N ? a.lse[bh * a.N + n + r] : -INFINITY;
        return n;
    };
    int n = i < n4 ? load() : 0;
    grid_wait();
    float2 *part = reinterpret_cast<float2 *>(a.dq);
    float2 m = make_float2(0.f, 0.f);
#pragma unroll 5
    for (int p = threadIdx.x; p < a.parts; p += blockDim.x) {
        const float2 x = part[p];
        m = make_float2(fmaxf(m.x, x.x), fmaxf(m.y, x.y));
    }
    __shared__ float2 most[8];
    m = cta_max(m, most);
    // 2^e 2 D m.x m.y <= 65504 / 1.01 = 2^15.985; infinities leave 0, zeros 15
    const float room = floorf((D == 64 ? 8.985f : 7.985f) - (log2f(m.x) + log2f(m.y)));
    const float e = room > 0.f ? fminf(room, 15.f) : 0.f;    // (a NaN: 0)
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *reinterpret_cast<int *>(part + a.parts) = static_cast<int>(e);
        if (a.dsinks != nullptr)
            for (int h = threadIdx.x; h < a.H; h += blockDim.x) a.dsinks[h] = exp2f(-e);
    }
    while (i < n4) {
        float w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            w[r] = l[r] == -INFINITY ? INFINITY : __fsub_rn(to_log2(l[r]), e);
            if (n + r >= a.N) a.ws_d[4 * i + r] = 0.f;
        }
        reinterpret_cast<float4 *>(a.ws_l)[i] = make_float4(w[0], w[1], w[2], w[3]);
        if ((i += step) < n4) n = load();
    }
}

// Shared helpers of the two main kernels -----------------------------------

// One TMA tile (128 rows x D, 128-byte swizzled chunks) of a [B][N][H][d] map.
template <int NCH>
__device__ __forceinline__ void load_tile(const CUtensorMap *m, uint32_t dst, uint32_t bar,
                                          int h, int row0, int b) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
        tma_load_4d(m, dst + c * 128u * 128u, bar, c * 64, h, row0, b);
}

// A ring of NS shared-memory slots filled and drained in order: item i
// lives in slot i % NS, in phase (i / NS) of that slot's barriers.
template <int NS>
struct Ring {
    __device__ static uint32_t slot(uint32_t i) { return i % NS; }
    __device__ static uint32_t phase(uint32_t i) { return (i / NS) & 1u; }
    // teardown: wait for the copy of the last item issued into each slot
    __device__ static void drain(uint32_t n_issued, uint32_t full0, const uint32_t full_bar_base) {
        for (uint32_t s = 0; s < NS && s < n_issued; ++s) {
            const uint32_t last = s + ((n_issued - 1 - s) / NS) * NS;
            mbar_wait_quiet(full_bar_base + 8u * (full0 + s), phase(last), 500000000ull);
        }
    }
};

// 16-bit A x B^T over the full K = D: both tiles K-major (S = Q K^T style).  kBatch:
// one election for four steps, or eight, instead of one each.  Interval masks at d = 64
// (4 x 4096, 12 heads over 4, both directions: 739 us with one each, 730); at d = 128 long documents
// lose 3 %, short ones nothing.
template <int D, bool kBatch = false>
__device__ __forceinline__ void gemm_ss_kmajor(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem,
                                               uint32_t idesc) {
    const uint64_t ad = smem_desc_sw128(a_smem, 16u, 1024u);
    const uint64_t bd = smem_desc_sw128(b_smem, 16u, 1024u);
    if constexpr (kBatch) {
#pragma unroll
        for (int kk = 0; kk < D / 16; kk += 4) {
            const uint32_t off = ((kk >> 2) * 128u * 128u) >> 4;
            mma_ss_f16_elect4<2, 2>(d_tmem, ad + off, bd + off, idesc, kk > 0 ? 1u : 0u);
        }
    } else {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * 128u * 128u + (kk & 3) * 32u) >> 4;
            mma_ss_f16_elect(d_tmem, ad + off, bd + off, idesc, kk > 0 ? 1u : 0u);
        }
    }
}

// D += A B with A (128 x 128, 16-bit) in TMEM and B (128 rows x D) an
// MN-major shared-memory tile (P V style).
template <bool kBatch = false>
__device__ __forceinline__ void gemm_ts_mn(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_smem,
                                           uint32_t idesc, bool accumulate) {
    const uint64_t bd = smem_desc_sw128(b_smem, 128u * 128u, 1024u);
    if constexpr (kBatch) {
        mma_ts_f16_elect8<8, 128>(d_tmem, a_tmem, bd, idesc, accumulate ? 1u : 0u);
    } else {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma_ts_f16_elect(d_tmem, a_tmem + kk * 8u, bd + ((kk * 2048u) >> 4), idesc,
                             (accumulate || kk > 0) ? 1u : 0u);
    }
}

// Whether tile t reaches outside the documents [live.x, live.y).
__device__ __forceinline__ bool tile_outside(int t, const int4 &live) {
    return t * 128 < live.x || t * 128 + 128 > live.y;
}

// Interval masks: a tile that does has these rows set to 0 in shared memory, by the eight elementwise warps (row
// `row` of the tile starting at token `first`, this thread's half of it), for
// products that weigh them with 0 (0 x NaN is not 0).
template <int NCH>
__device__ __forceinline__ void zero_outside(uint8_t *tile, int first, int row, int half, const int4 &live) {
    if (first + row < live.x || first + row >= live.y) {
        constexpr int PER = NCH == 2 ? 8 : 4;          // 16-byte vectors of this half
        uint8_t *at = tile + (NCH == 2 ? half * 128 * 128 : half * 64) + row * 128;
#pragma unroll
        for (int i = 0; i < PER; ++i) *reinterpret_cast<uint4 *>(at + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
}

// The rows' statistics, as the dK/dV kernel reads them.  Interval masks: it may begin
// while the kernel that writes them still runs, and the read-only path (ld.global.nc)
// is for data that nobody writes while a kernel runs; plain loads, which stay behind
// grid_wait()'s memory clobber.  (They cost 1 % on long documents at d = 64: 4 x 4096 tokens,
// 32 heads, bf16, 1080 us and 1091.)
template <bool kMask, class T>
__device__ __forceinline__ T ws_load(const T *p) {
    if constexpr (kMask) return *p;
    else return __ldg(p);
}

// Bits of the columns [lo, hi) of 32.
__device__ __forceinline__ uint32_t column_bits(int lo, int hi) {
    auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
    return below(hi) & ~below(lo);
}

// Distance bias -beta |i - j| of a tile row's columns c = 0, 1, ..., d0 = the row's
// token less the first column's.  In a tile beside the diagonal one it is linear,
// b0 + bs c.
struct BiasCols {
    float2 even, odd, step;     // columns (c, c + 1) and (c + 2, c + 3), four further on
    __device__ __forceinline__ BiasCols(float beta, float d0, bool before, float add) {
        const float bs = before ? beta : -beta, b0 = add - bs * d0;
        even = make_float2(b0, b0 + bs);
        odd = make_float2(__fmaf_rn(2.f, bs, b0), __fmaf_rn(3.f, bs, b0));
        step = make_float2(4.f * bs, 4.f * bs);
    }
    // in the order of the columns
    __device__ __forceinline__ float2 next(int c) {
        float2 &b = c & 2 ? odd : even;
        const float2 v = b;
        b = __fadd2_rn(b, step);
        return v;
    }
};

// Epilogue store: columns [col0, col0 + W) of one row, v * scale -> 16 bit.
template <int D, int W, bool kBF16>
__device__ __forceinline__ void store_cols(void *dst_base, const BwdArgs &a, int heads, int b,
                                           int h, int row, int col0, const uint32_t (&v)[W],
                                           float scale) {
    if (row >= a.N) return;
    uint16_t *dst = reinterpret_cast<uint16_t *>(dst_base) +
                    ((static_cast<size_t>(b) * a.N + row) * heads + h) * D + col0;
#pragma unroll
    for (int ch = 0; ch < W / 8; ++ch) {
        uint32_t pk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pk[i] = pack2<kBF16>(__uint_as_float(v[8 * ch + 2 * i]) * scale,
                                 __uint_as_float(v[8 * ch + 2 * i + 1]) * scale);
        reinterpret_cast<uint4 *>(dst)[ch] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
    }
}

// ---------------------------------------------------------------------------
// dQ kernel (query-parallel).  Per key tile t of the unit's query tile:
//   S(t) = Q K_t^T, dP(t) = dO V_t^T          (TMEM S, dP)
//   P = exp2(S c - LSE2), dS = P o (dP - D)   (elementwise group; P in
//                                              registers, dS -> TMEM dS[t%2])
//   dQ += dS(t) K_t                           (TMEM dQ; K_t MN-major)
// MMA order: S(0), dP(0), then for each t: [S consumed] S(t+1);
// [dS(t) ready] dP(t+1), dQ(t).  The exponentials of tile t+1 overlap dQ(t)
// and dP(t+1); dS is double-buffered so dQ(t) reads dS(t) while dS(t+1) is
// written.
// ---------------------------------------------------------------------------
template <int D, bool kCausal, bool kBF16, bool kWin = false, bool kCap = false, bool kMask = false,
          bool kBias = false>
__global__ void __launch_bounds__(320, 1)
fa_bwd_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                 const BwdArgs a) {
    using C = BwdCfg<D, kBF16>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool snake = bwd_longest_first<kCausal, kWin>(a);   // unit order (unit_stride0)
    auto bar = [&](int i) -> uint32_t { return base + C::DQ_BAR_OFF + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gbase + C::DQ_MISC_OFF);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + C::DQ_MISC_OFF + 4);
    // Causal without a window, interval masks: one CTA per unit, running CTAs take over those
    // not yet started (clc_try_cancel).  The producer asks for the next unit
    // once it has issued the current one's loads; the k-th answer goes to
    // slot k % CLC_DEPTH, the producer publishes its block index there (-1:
    // none left), and the MMA warp and the 8 elementwise warps read it.
    constexpr bool kDyn = (kCausal && !kWin) || kMask;
    constexpr bool kBatch = kMask && D == 64;               // (gemm_ss_kmajor)
    volatile int *unit_slot = reinterpret_cast<volatile int *>(gbase + C::DQ_UNIT_OFF);
    // key tiles [lo, hi) of query tile U.m, visited from hi - 1 down
    auto key_range = [&](const BwdUnit &U, int &lo, int &hi) {
        if constexpr (kMask) {
            lo = U.lo;
            hi = U.hi;
        } else if constexpr (kWin) {
            const int r0 = U.m * 128, r1 = min(a.N, r0 + 128) - 1;
            lo = tile_lo(win_klo(r0, a));
            hi = tile_hi(win_khi(r1, a));
        } else {
            lo = 0;
            hi = kCausal ? U.m + 1 : a.n_t;
        }
    };

    if (warp == 9) tmem_alloc(base + C::DQ_MISC_OFF, C::TMEM_COLS);
    if (tid == 0) {
        *abort_flag = 0u;
        mbar_init(bar(C::DQB_QFULL), 1);
        mbar_init(bar(C::DQB_QEMPTY), 1);
        mbar_init(bar(C::DQB_SFULL), 1);
        mbar_init(bar(C::DQB_DPFULL), 1);
        mbar_init(bar(C::DQB_SFREE), C::N_EW);
        mbar_init(bar(C::DQB_DSFULL + 0), C::N_EW);
        mbar_init(bar(C::DQB_DSFULL + 1), C::N_EW);
        mbar_init(bar(C::DQB_DQFULL), 1);
        mbar_init(bar(C::DQB_DQEMPTY), C::N_EW);
        mbar_init(bar(C::DQB_MMADONE), 1);
        for (int q = 0; kDyn && q < C::CLC_DEPTH; ++q) {
            mbar_init(bar(C::DQB_CLCFULL + q), 1);
            mbar_init(bar(C::DQB_UNIT + q), 1);
            mbar_init(bar(C::DQB_CLCEMPTY + q), 1 + C::N_EW);
        }
        for (int s = 0; s < C::KN; ++s) {
            mbar_init(bar(C::DQB_KFULL + s), 1);
            mbar_init(bar(C::DQB_KEMPTY + s), 1);
        }
        for (int s = 0; s < C::VN; ++s) {
            mbar_init(bar(C::DQB_VFULL + s), 1);
            mbar_init(bar(C::DQB_VEMPTY + s), 1);
        }
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    if (warp == 8) {
        // =================== TMA producer (one lane) ===================
        if (lane == 0) {
            WaitCtx w{abort_flag, a.status, kRoleProducer};
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            tma_prefetch_desc(&tm_do);
            using RK = Ring<C::KN>;
            using RV = Ring<C::VN>;
            uint32_t nk = 0, nv = 0;
            int qn = 0;
            bool ok = true;
            uint32_t kq = 0;                        // causal: requests issued
            bool clc_pending = false;               // a request without its answer
            auto next_dyn = [&]() __attribute__((always_inline)) -> int {
                if (!ok) return -1;
                const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
                ++kq;
                if (!mbar_wait(bar(C::DQB_CLCEMPTY + q), ph ^ 1u, w, 53)) { ok = false; return -1; }
                mbar_arrive_expect_tx(bar(C::DQB_CLCFULL + q), 16u);
                clc_try_cancel(base + C::DQ_CLC_OFF + 16u * q, bar(C::DQB_CLCFULL + q));
                clc_pending = true;
                if (!mbar_wait(bar(C::DQB_CLCFULL + q), ph, w, 54)) { ok = false; return -1; }
                clc_pending = false;
                const int nu = clc_block(base + C::DQ_CLC_OFF + 16u * q);
                unit_slot[q] = nu;
                mbar_arrive(bar(C::DQB_UNIT + q));    // release: the index is visible
                return nu;
            };
            // Interval masks: publishes unit u (-1: the end); the next one is asked for
            // ahead of this one's last tiles (fa_fwd_kernel.cuh).
            auto publish = [&](int u, BwdUnit &U) __attribute__((always_inline)) -> bool {
                const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
                BwdRec r{make_int4(-1, 0, 0, 0), make_int4(0, 0, 0, 0)};
                if (u >= 0) r = bwd_rec<false>(u, a);
                U = bwd_unit(r);
                ++kq;
                if (!mbar_wait(bar(C::DQB_CLCEMPTY + q), ph ^ 1u, w, 55)) { ok = false; return false; }
                int4 *slot_r = reinterpret_cast<int4 *>(gbase + C::DQ_REC_OFF) + 2 * q;
                slot_r[0] = r.id;
                slot_r[1] = r.range;
                mbar_arrive(bar(C::DQB_UNIT + q));      // release: the record is visible
                return u >= 0;
            };
            auto ask = [&]() __attribute__((always_inline)) {
                mbar_arrive_expect_tx(bar(C::DQB_CLCFULL), 16u);
                clc_try_cancel(base + C::DQ_CLC_OFF, bar(C::DQB_CLCFULL));
                clc_pending = true;
            };
            auto answer = [&]() __attribute__((always_inline)) -> int {
                if (!ok || !mbar_wait(bar(C::DQB_CLCFULL), (kq - 1) & 1u, w, 56)) { ok = false; return -1; }
                clc_pending = false;
                return clc_block(base + C::DQ_CLC_OFF);
            };
            for (int u = blockIdx.x, st = unit_stride0(snake); ok && (kMask || ((!kDyn || u >= 0) && u < a.n_units));
                     u = kMask ? answer() : kDyn ? next_dyn() : u + st, st = 2 * static_cast<int>(gridDim.x) - st) {
                BwdUnit U;
                if constexpr (kMask) {
                    if (!publish(u, U)) break;
                    if (U.lo >= U.hi) ask();
                } else {
                    U = make_bwd_unit<kCausal, false, kWin>(u, a);
                }
                if (kMask && U.lo >= U.hi) continue;         // sees nothing: dQ is 0
                ok = mbar_wait(bar(C::DQB_QEMPTY), (qn & 1) ^ 1, w, 50);
                if (!ok) break;
                mbar_arrive_expect_tx(bar(C::DQB_QFULL), 2 * C::TILE);
                load_tile<C::NCH>(&tm_q, base + C::DQ_Q_OFF, bar(C::DQB_QFULL), U.h, U.m * 128, U.b);
                load_tile<C::NCH>(&tm_do, base + C::DQ_DO_OFF, bar(C::DQB_QFULL), U.h, U.m * 128, U.b);
                ++qn;
                int klo_t, khi_t;
                key_range(U, klo_t, khi_t);
                const int T = khi_t - klo_t;
                for (int t = 0; ok && t < T; ++t) {
                    const int j = khi_t - 1 - t;
                    if (kMask && t == max(0, T - 2)) ask();
                    const uint32_t ks = RK::slot(nk), vs = RV::slot(nv);
                    ok = mbar_wait(bar(C::DQB_KEMPTY + ks), RK::phase(nk) ^ 1, w, 51);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(C::DQB_KFULL + ks), C::TILE);
                    load_tile<C::NCH>(&tm_k, base + C::DQ_K_OFF + ks * C::TILE, bar(C::DQB_KFULL + ks),
                                      U.h / a.group, j * 128, U.b);
                    ++nk;
                    ok = mbar_wait(bar(C::DQB_VEMPTY + vs), RV::phase(nv) ^ 1, w, 52);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(C::DQB_VFULL + vs), C::TILE);
                    load_tile<C::NCH>(&tm_v, base + C::DQ_V_OFF + vs * C::TILE, bar(C::DQB_VFULL + vs),
                                      U.h / a.group, j * 128, U.b);
                    ++nv;
                }
            }
            if (kMask && clc_pending)
                mbar_wait_quiet(bar(C::DQB_CLCFULL), (kq - 1) & 1u, 500000000ull);
            else if (kDyn && clc_pending)
                mbar_wait_quiet(bar(C::DQB_CLCFULL + (kq - 1) % C::CLC_DEPTH),
                                ((kq - 1) / C::CLC_DEPTH) & 1u, 500000000ull);
            RK::drain(nk, C::DQB_KFULL, base + C::DQ_BAR_OFF);
            RV::drain(nv, C::DQB_VFULL, base + C::DQ_BAR_OFF);
            if (qn > 0) mbar_wait_quiet(bar(C::DQB_QFULL), (qn - 1) & 1, 500000000ull);
        }
        __syncwarp();
    } else if (warp == 9) {
        // =================== MMA issuer ===================
        WaitCtx w{abort_flag, a.status, kRoleMma};
        using RK = Ring<C::KN>;
        using RV = Ring<C::VN>;
        uint32_t k0 = 0;                    // K and V items of earlier units
        uint32_t qph = 0, sfree_ph = 0, ds_ph0 = 0, ds_ph1 = 0, dqe_ph = 0;
        bool ok = true;
        auto k_tile = [&](uint32_t i) { return base + C::DQ_K_OFF + RK::slot(i) * C::TILE; };
        auto v_tile = [&](uint32_t i) { return base + C::DQ_V_OFF + RV::slot(i) * C::TILE; };
        auto wait_k = [&](uint32_t i) {
            return mbar_wait_warp(bar(C::DQB_KFULL + RK::slot(i)), RK::phase(i), w, 61);
        };
        auto wait_v = [&](uint32_t i) {
            return mbar_wait_warp(bar(C::DQB_VFULL + RV::slot(i)), RV::phase(i), w, 62);
        };
        uint32_t kq = 0;                            // causal: answers read
        auto next_dyn = [&]() __attribute__((always_inline)) -> int {
            if (!ok) return -1;
            const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
            ++kq;
            if (!mbar_wait_warp(bar(C::DQB_UNIT + q), ph, w, 64)) { ok = false; return -1; }
            const int nu = unit_slot[q];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::DQB_CLCEMPTY + q));
            return nu;
        };
        auto next_rec = [&](BwdUnit &U) __attribute__((always_inline)) -> int {
            if (!ok) return -1;
            const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
            ++kq;
            if (!mbar_wait_warp(bar(C::DQB_UNIT + q), ph, w, 66)) { ok = false; return -1; }
            const BwdRec r = read_bwd_rec(gbase + C::DQ_REC_OFF, q);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::DQB_CLCEMPTY + q));
            U = bwd_unit(r);
            return r.id.x;
        };
        BwdUnit U;
        for (int u = kMask ? next_rec(U) : static_cast<int>(blockIdx.x), st = unit_stride0(snake);
                 ok && (!kDyn || u >= 0) && u < a.n_units;
                 u = kMask ? next_rec(U) : kDyn ? next_dyn() : u + st, st = 2 * static_cast<int>(gridDim.x) - st) {
            if constexpr (!kMask) U = make_bwd_unit<kCausal, false, kWin>(u, a);
            int klo_t, khi_t;
            key_range(U, klo_t, khi_t);
            const int T = khi_t - klo_t;
            if (kMask && T <= 0) continue;
            ok = mbar_wait_warp(bar(C::DQB_QFULL), qph, w, 60);
            if (!ok) break;
            qph ^= 1;
            // S(0), dP(0)
            ok = wait_k(k0) && wait_v(k0);
            if (!ok) break;
            tc_fence_after();
            gemm_ss_kmajor<D, kBatch>(tbase + C::DQ_COL_S, base + C::DQ_Q_OFF, k_tile(k0), C::IDESC_SS);
            mma_commit_elect(bar(C::DQB_SFULL));
            gemm_ss_kmajor<D, kBatch>(tbase + C::DQ_COL_DP, base + C::DQ_DO_OFF, v_tile(k0), C::IDESC_SS);
            mma_commit_elect(bar(C::DQB_DPFULL));
            mma_commit_elect(bar(C::DQB_VEMPTY + RV::slot(k0)));
            if (T == 1) mma_commit_elect(bar(C::DQB_QEMPTY));
            for (int t = 0; ok && t < T; ++t) {
                const uint32_t it = k0 + t;          // item index of tile t in both rings
                // ---- S(t+1) once S(t) has been read ----
                ok = mbar_wait_warp(bar(C::DQB_SFREE), sfree_ph, w, 63);
                if (!ok) break;
                sfree_ph ^= 1;
                if (t + 1 < T) {
                    ok = wait_k(it + 1);
                    if (!ok) break;
                    tc_fence_after();
                    gemm_ss_kmajor<D, kBatch>(tbase + C::DQ_COL_S, base + C::DQ_Q_OFF, k_tile(it + 1), C::IDESC_SS);
                    mma_commit_elect(bar(C::DQB_SFULL));
                }
                // ---- dS(t) ready: dP(t+1), then dQ += dS(t) K(t) ----
                const int b2 = t & 1;
                ok = mbar_wait_warp(bar(C::DQB_DSFULL + b2), b2 ? ds_ph1 : ds_ph0, w, 65);
                if (!ok) break;
                if (b2) ds_ph1 ^= 1; else ds_ph0 ^= 1;
                if (t + 1 < T) {
                    ok = wait_v(it + 1);
                    if (!ok) break;
                    tc_fence_after();
                    gemm_ss_kmajor<D, kBatch>(tbase + C::DQ_COL_DP, base + C::DQ_DO_OFF, v_tile(it + 1), C::IDESC_SS);
                    mma_commit_elect(bar(C::DQB_DPFULL));
                    mma_commit_elect(bar(C::DQB_VEMPTY + RV::slot(it + 1)));
                    if (t + 2 == T) mma_commit_elect(bar(C::DQB_QEMPTY));   // last use of Q, dO
                }
                if (t == 0) {
                    ok = mbar_wait_warp(bar(C::DQB_DQEMPTY), dqe_ph ^ 1, w, 67);
                    if (!ok) break;
                    dqe_ph ^= 1;
                }
                tc_fence_after();
                gemm_ts_mn<kBatch>(tbase + C::DQ_COL_DQ, tbase + C::DQ_COL_DS + b2 * 64u, k_tile(it),
                           C::IDESC_ACC, t > 0);
                mma_commit_elect(bar(C::DQB_KEMPTY + RK::slot(it)));
            }
            if (!ok) break;
            mma_commit_elect(bar(C::DQB_DQFULL));
            k0 += T;
        }
        mma_commit_elect(bar(C::DQB_MMADONE));
        mbar_wait_quiet(bar(C::DQB_MMADONE), 0, 500000000ull);
        __syncwarp();
    } else {
        // =================== elementwise group (warps 0-7) ===================
        const int quarter = warp & 3, half = warp >> 2;
        const int row = quarter * 32 + lane;                 // TMEM lane == tile row
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const int col0 = half * 64;                          // this warp's key columns
        WaitCtx w{abort_flag, a.status, kRoleSoftmax0};
        const float sl2 = a.scale_log2;
        uint32_t sph = 0, dpph = 0, dqph = 0;
        uint32_t kt = 0;                            // interval masks: K tiles of the units so far
        bool ok = true;
        uint32_t kq = 0;                            // causal: answers read
        auto next_dyn = [&]() __attribute__((always_inline)) -> int {
            if (!ok) return -1;
            const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
            ++kq;
            ok = mbar_wait(bar(C::DQB_UNIT + q), ph, w, 73);
            if (__any_sync(0xffffffffu, !ok)) { ok = false; return -1; }
            const int nu = unit_slot[q];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::DQB_CLCEMPTY + q));
            return nu;
        };
        // Interval masks: the next unit's record, and this row's keys and statistics in
        // it, are read before the stores of the unit at hand.
        BwdRec rec_n{};
        int2 vis_n = make_int2(0, 0);
        float lse2_n = 0.f, drow_n = 0.f, beta_n = 0.f;
        auto fetch = [&]() __attribute__((always_inline)) -> int {
            const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
            ++kq;
            ok = mbar_wait(bar(C::DQB_UNIT + q), ph, w, 73);
            if (__any_sync(0xffffffffu, !ok)) { ok = false; return -1; }
            rec_n = read_bwd_rec(gbase + C::DQ_REC_OFF, q);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::DQB_CLCEMPTY + q));
            if (rec_n.id.x < 0) return -1;
            const int n = rec_n.id.w * 128 + row;
            const size_t at = (static_cast<size_t>(rec_n.id.y) * a.H + rec_n.id.z) * a.NP + n;
            vis_n = n < a.N ? __ldg(a.plan.rows + static_cast<size_t>(rec_n.id.y) * a.N + n) : make_int2(0, 0);
            lse2_n = __ldg(a.ws_l + at);
            drow_n = __ldg(a.ws_d + at);
            if constexpr (kBias) beta_n = __ldg(a.slopes + rec_n.id.z) * 1.44269504088896340736f;
            return rec_n.id.x;
        };
        for (int u = kMask ? fetch() : static_cast<int>(blockIdx.x), st = unit_stride0(snake);
                 ok && (!kDyn || u >= 0) && u < a.n_units;
                 u = kMask ? u : kDyn ? next_dyn() : u + st, st = 2 * static_cast<int>(gridDim.x) - st) {
            BwdUnit U;
            const bool padded = rec_n.range.z != 0;
            const int2 vis = vis_n;
            if constexpr (kMask) U = bwd_unit(rec_n);
            else U = make_bwd_unit<kCausal, false, kWin>(u, a);
            int klo_t, khi_t;
            key_range(U, klo_t, khi_t);
            const int T = khi_t - klo_t;
            const int grow = U.m * 128 + row;
            if (kMask && T <= 0) {                           // no row of the tile sees a key
                u = fetch();
                if (grow < a.N) {
                    uint4 *z = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.dq) +
                               ((static_cast<size_t>(U.b) * a.N + grow) * a.H + U.h) * D + half * (D / 2));
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) z[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                continue;
            }
            // this row's visible keys (rows past N: any range; their P is 0)
            int klo_r = 0, khi_r = a.N;
            float beta = 0.f;                                // the bias a key of distance, log2 units
            if constexpr (kMask) {
                klo_r = vis.x;
                khi_r = vis.y;
                if constexpr (kBias) beta = beta_n;
            } else if constexpr (kWin) {
                const int gr = min(grow, a.N - 1);
                klo_r = win_klo(gr, a);
                khi_r = win_khi(gr, a);
            }
            // log2-domain LSE of this row (+inf for rows beyond N and empty
            // rows: their P is 0) and D of this row, from the workspace
            const size_t widx = (static_cast<size_t>(U.b) * a.H + U.h) * a.NP + grow;
            const float lse2 = kMask ? lse2_n : a.ws_l[widx], drow = kMask ? drow_n : a.ws_d[widx];
            const float2 c2 = kCap ? make_float2(a.sc_post, a.sc_post) : make_float2(sl2, sl2);
            const float2 nl2 = make_float2(-lse2, -lse2);
            const float2 nd2 = make_float2(-drow, -drow);
            for (int t = 0; t < T; ++t) {
                const int j = khi_t - 1 - t;
                // ---- P(t) = exp2(S c - LSE2) from S(t) ----
                ok = mbar_wait(bar(C::DQB_SFULL), sph, w, 70);
                if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
                sph ^= 1;
                tc_fence_after();
                uint32_t sv[64];
                const uint32_t tS = tbase + lane_off + C::DQ_COL_S + col0;
                tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::DQB_SFREE));
                int lim = min(128, a.N - j * 128) - col0;        // keys beyond N
                if (kCausal) lim = min(lim, grow - j * 128 + 1 - col0);
                int llo = 0;                                     // window: first visible
                if constexpr (kWin || kMask) {
                    lim = min(lim, khi_r - j * 128 - col0);
                    llo = klo_r - j * 128 - col0;
                }
                float *pf = reinterpret_cast<float *>(sv);
                // interval masks: the visible columns, whether every row of the warp sees
                // them all, whether hidden ones may hold anything
                uint32_t seen[2] = {~0u, ~0u};
                bool whole = true, edge = false;
                if constexpr (kMask) {
                    whole = __all_sync(0xffffffffu, lim >= 64 && llo <= 0) && !(kBias && j == U.m);
                    if (!whole) {
                        seen[0] = column_bits(llo, lim);
                        seen[1] = column_bits(llo - 32, lim - 32);
                    }
                }
                if constexpr (kMask) {
                    if (padded) {
                        const int4 live = __ldg(a.plan.live + U.b);
                        const bool outside = tile_outside(j, live);
                        edge = outside || tile_outside(U.m, live);
                        // (S(t) has been formed, dQ(t) waits for dS(t): K rows may change)
                        if (outside)
                            zero_outside<C::NCH>(gbase + C::DQ_K_OFF + ((kt + t) % C::KN) * C::TILE, j * 128, row, half,
                                                 live);
                    }
                }
                if constexpr (kCap) {
                    // keep t = tanh(alpha s / c); P comes from t in the dS step
#pragma unroll
                    for (int c = 0; c < 64; ++c) pf[c] = tanh_approx(pf[c] * a.sc_pre);
                } else if constexpr (kMask) {
                    const float d0 = static_cast<float>(grow - j * 128 - col0);
                    if (whole) {
                        BiasCols bc(beta, d0, j < U.m, -lse2);
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const float2 x = __ffma2_rn(make_float2(pf[c], pf[c + 1]), c2, kBias ? bc.next(c) : nl2);
                            pf[c] = ex2_approx(x.x);
                            pf[c + 1] = ex2_approx(x.y);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 64; ++c) {
                            const float x = __fmaf_rn(pf[c], sl2, kBias ? __fmaf_rn(-beta, fabsf(d0 - c), -lse2) : -lse2);
                            pf[c] = (seen[c >> 5] & (1u << (c & 31))) ? ex2_approx(x) : 0.f;
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const float2 x = __ffma2_rn(make_float2(pf[c], pf[c + 1]), c2, nl2);
                        pf[c] = (c < lim && (!kWin || c >= llo)) ? ex2_approx(x.x) : 0.f;
                        pf[c + 1] = (c + 1 < lim && (!kWin || c + 1 >= llo)) ? ex2_approx(x.y) : 0.f;
                    }
                }
                // ---- dS(t) = P o (dP - D) -> TMEM dS[t%2] ----
                ok = mbar_wait(bar(C::DQB_DPFULL), dpph, w, 71);
                if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
                dpph ^= 1;
                tc_fence_after();
                uint32_t dp[64];
                const uint32_t tDP = tbase + lane_off + C::DQ_COL_DP + col0;
                tmem_ld32(tDP, *reinterpret_cast<uint32_t(*)[32]>(&dp[0]));
                tmem_ld32(tDP + 32, *reinterpret_cast<uint32_t(*)[32]>(&dp[32]));
                tmem_ld_wait();
                if constexpr (kMask) {
                    if (edge) {                  // dP of a row or key outside may be NaN
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!(seen[c >> 5] & (1u << (c & 31)))) dp[c] = 0u;
                    }
                }
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float2 g = __fadd2_rn(
                        make_float2(__uint_as_float(dp[i]), __uint_as_float(dp[i + 1])), nd2);
                    float2 pp = make_float2(pf[i], pf[i + 1]);
                    if constexpr (kCap) {
                        // P = 2^(t c log2(e) - LSE2), and dS/du = 1 - t^2
                        const float2 x = __ffma2_rn(pp, c2, nl2);
                        const float2 dt = __ffma2_rn(make_float2(-pp.x, -pp.y), pp,
                                                     make_float2(1.f, 1.f));
                        pp.x = (i < lim && (!kWin || i >= llo)) ? ex2_approx(x.x) * dt.x : 0.f;
                        pp.y = (i + 1 < lim && (!kWin || i + 1 >= llo)) ? ex2_approx(x.y) * dt.y : 0.f;
                    }
                    const float2 ds = __fmul2_rn(pp, g);
                    pk[i / 2] = pack2<kBF16>(ds.x, ds.y);
                }
                tmem_st32(tbase + lane_off + C::DQ_COL_DS + (t & 1) * 64u + half * 32, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::DQB_DSFULL + (t & 1)));
            }
            if (!ok) break;
            kt += static_cast<uint32_t>(T);
            if constexpr (kMask) {
                u = fetch();
                if (!ok) break;
            }
            // ---- epilogue: dQ * alpha -> global (this warp's half of the columns) ----
            float out_scale = a.alpha;
            if constexpr (kMask && !kBF16)
                if (grow < a.N)
                    out_scale *= scale_undo(__ldg(a.lse + (static_cast<size_t>(U.b) * a.H + U.h) * a.N + grow), lse2);
            ok = mbar_wait(bar(C::DQB_DQFULL), dqph, w, 72);
            if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
            dqph ^= 1;
            tc_fence_after();
            constexpr int W = D / 2;
            uint32_t dq[W];
#pragma unroll
            for (int ch = 0; ch < W / 32; ++ch)
                tmem_ld32(tbase + lane_off + C::DQ_COL_DQ + half * W + ch * 32,
                          *reinterpret_cast<uint32_t(*)[32]>(&dq[ch * 32]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::DQB_DQEMPTY));
            store_cols<D, W, kBF16>(a.dq, a, a.H, U.b, U.h, grow, half * W, dq, out_scale);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
    // Interval masks: this grid may have begun before the dK/dV kernel's end, and what
    // follows it on the stream waits for this one alone.
    if constexpr (kMask) grid_wait();
}

// ---------------------------------------------------------------------------
// dK/dV kernel (key-parallel).  The unit's key tile K, V stays in shared
// memory; per query tile i (causal: i from the diagonal on):
//   G1  S^T(i) = K Q_i^T,   G2  dP^T(i) = V dO_i^T        (TMEM S^T, dP^T)
//   P^T = exp2(S^T c - LSE2[q]) -> 16 bit over S^T        (elementwise)
//   G3  dV += P^T dO_i                                     (dO_i MN-major)
//   dS^T = P^T o (dP^T - D[q]) -> 16 bit over dP^T         (elementwise)
//   G4  dK += dS^T Q_i                                     (Q_i MN-major)
// MMA order per tile: G3(i), G1(i+1), G4(i), G2(i+1), so the exponentials
// of tile i+1 overlap G4(i) and G2(i+1), and dS(i+1) overlaps G3(i+1) and
// G1(i+2).  The 16-bit P^T and dS^T of the query columns [64h, 64h+64)
// (h: the warp's column half) go to TMEM columns 32 + 32h .. +32 of the
// S^T / dP^T regions, which that warp has itself read, so the two warps of
// a lane quarter need no barrier; G3 and G4 read their A operand from
// column 32.  Q_i and dO_i come through separate rings (Q is held until G4,
// dO until G3); LSE2 and D of the query columns are read from the padded
// workspace through L1 (the producer prefetches them, and the elementwise
// warps touch the next tile's sectors a tile ahead).
// ---------------------------------------------------------------------------
template <int D, bool kCausal, bool kBF16, bool kWin = false, bool kCap = false, bool kMask = false,
          bool kBias = false>
__global__ void __launch_bounds__(320, 1)
fa_bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                   const BwdArgs a) {
    using C = BwdCfg<D, kBF16>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool snake = bwd_longest_first<kCausal, kWin>(a);   // unit order (unit_stride0)
    auto bar = [&](int i) -> uint32_t { return base + C::KV_BAR_OFF + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gbase + C::KV_MISC_OFF);
    volatile uint32_t *abort_flag = reinterpret_cast<volatile uint32_t *>(gbase + C::KV_MISC_OFF + 4);
    constexpr bool kScale = kMask && !kBF16;                // (fa_bwd_delta_kernel)
    volatile int *scale_slot = reinterpret_cast<volatile int *>(gbase + C::KV_MISC_OFF + 8);   // its e
    // Causal without a window, interval masks: one CTA per unit, running CTAs take over those
    // not yet started (clc_try_cancel).  The producer asks for the next unit
    // once it has issued the current one's loads; the k-th answer goes to
    // slot k % CLC_DEPTH, the producer publishes its block index there (-1:
    // none left), and the MMA warp and the 8 elementwise warps read it.
    constexpr bool kDyn = (kCausal && !kWin) || kMask;
    constexpr bool kBatch = kMask && D == 64;               // (gemm_ss_kmajor)
    volatile int *unit_slot = reinterpret_cast<volatile int *>(gbase + C::KV_UNIT_OFF);
    // query tiles [lo, hi) that see key tile U.m
    auto query_range = [&](const BwdUnit &U, int &lo, int &hi) {
        if constexpr (kMask) {
            lo = U.lo;
            hi = U.hi;
        } else if constexpr (kWin) {
            const int k0 = U.m * 128, k1 = min(a.N, k0 + 128) - 1;
            lo = tile_lo(win_qlo(k0, a));
            hi = tile_hi(win_qhi(k1, a));
        } else {
            lo = kCausal ? U.m : 0;
            hi = a.n_t;
        }
    };
    using RQ = Ring<C::QN>;
    using RO = Ring<C::DN>;
    auto q_tile = [&](uint32_t i) { return base + C::KV_Q_OFF + RQ::slot(i) * C::TILE; };
    auto do_tile = [&](uint32_t i) { return base + C::KV_DO_OFF + RO::slot(i) * C::TILE; };

    if (warp == 9) tmem_alloc(base + C::KV_MISC_OFF, C::TMEM_COLS);
    if (tid == 0) {
        *abort_flag = 0u;
        mbar_init(bar(C::KVB_KVFULL), 1);
        mbar_init(bar(C::KVB_KVEMPTY), 1);
        mbar_init(bar(C::KVB_STFULL), 1);
        mbar_init(bar(C::KVB_STFULL1), 1);
        mbar_init(bar(C::KVB_DPTFULL), 1);
        mbar_init(bar(C::KVB_PFULL), C::N_EW);
        mbar_init(bar(C::KVB_PFULL1), C::N_EW);
        mbar_init(bar(C::KVB_DSFULL), C::N_EW);
        mbar_init(bar(C::KVB_ACCFULL), 1);
        mbar_init(bar(C::KVB_ACCEMPTY), C::N_EW);
        mbar_init(bar(C::KVB_MMADONE), 1);
        for (int q = 0; kDyn && q < C::CLC_DEPTH; ++q) {
            mbar_init(bar(C::KVB_CLCFULL + q), 1);
            mbar_init(bar(C::KVB_UNIT + q), 1);
            mbar_init(bar(C::KVB_CLCEMPTY + q), 1 + C::N_EW);
        }
        for (int s = 0; s < C::QN; ++s) {
            mbar_init(bar(C::KVB_QFULL + s), 1);
            mbar_init(bar(C::KVB_QEMPTY + s), 1);
        }
        for (int s = 0; s < C::DN; ++s) {
            mbar_init(bar(C::KVB_DOFULL + s), 1);
            mbar_init(bar(C::KVB_DOEMPTY + s), 1);
        }
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;

    if (warp == 8) {
        // =================== TMA producer (one lane) ===================
        if (lane == 0) {
            WaitCtx w{abort_flag, a.status, kRoleProducer};
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            tma_prefetch_desc(&tm_do);
            uint32_t nq = 0, n_qc = 0, n_dc = 0;     // tiles; Q and dO copies issued
            int kvn = 0;
            bool ok = true;
            uint32_t kq = 0;                        // causal: requests issued
            bool clc_pending = false;               // a request without its answer
            auto next_dyn = [&]() __attribute__((always_inline)) -> int {
                if (!ok) return -1;
                const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
                ++kq;
                if (!mbar_wait(bar(C::KVB_CLCEMPTY + q), ph ^ 1u, w, 83)) { ok = false; return -1; }
                mbar_arrive_expect_tx(bar(C::KVB_CLCFULL + q), 16u);
                clc_try_cancel(base + C::KV_CLC_OFF + 16u * q, bar(C::KVB_CLCFULL + q));
                clc_pending = true;
                if (!mbar_wait(bar(C::KVB_CLCFULL + q), ph, w, 84)) { ok = false; return -1; }
                clc_pending = false;
                const int nu = clc_block(base + C::KV_CLC_OFF + 16u * q);
                unit_slot[q] = nu;
                mbar_arrive(bar(C::KVB_UNIT + q));    // release: the index is visible
                return nu;
            };
            // Interval masks: publishes unit u (-1: the end); the next one is asked for
            // ahead of this one's last tiles (fa_fwd_kernel.cuh).
            auto publish = [&](int u, BwdUnit &U) __attribute__((always_inline)) -> bool {
                const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
                BwdRec r{make_int4(-1, 0, 0, 0), make_int4(0, 0, 0, 0)};
                if (u >= 0) r = bwd_rec<true>(u, a);
                U = bwd_unit(r);
                ++kq;
                if (!mbar_wait(bar(C::KVB_CLCEMPTY + q), ph ^ 1u, w, 55)) { ok = false; return false; }
                int4 *slot_r = reinterpret_cast<int4 *>(gbase + C::KV_REC_OFF) + 2 * q;
                slot_r[0] = r.id;
                slot_r[1] = r.range;
                mbar_arrive(bar(C::KVB_UNIT + q));      // release: the record is visible
                return u >= 0;
            };
            auto ask = [&]() __attribute__((always_inline)) {
                mbar_arrive_expect_tx(bar(C::KVB_CLCFULL), 16u);
                clc_try_cancel(base + C::KV_CLC_OFF, bar(C::KVB_CLCFULL));
                clc_pending = true;
            };
            auto answer = [&]() __attribute__((always_inline)) -> int {
                if (!ok || !mbar_wait(bar(C::KVB_CLCFULL), (kq - 1) & 1u, w, 56)) { ok = false; return -1; }
                clc_pending = false;
                return clc_block(base + C::KV_CLC_OFF);
            };
            for (int u = blockIdx.x, st = unit_stride0(snake); ok && (kMask || ((!kDyn || u >= 0) && u < a.n_units_kv));
                     u = kMask ? answer() : kDyn ? next_dyn() : u + st, st = 2 * static_cast<int>(gridDim.x) - st) {
                BwdUnit U;
                if constexpr (kMask) {
                    if (!publish(u, U)) break;
                    if (U.lo >= U.hi) ask();
                } else {
                    U = make_bwd_unit<kCausal, true, kWin>(u, a);
                }
                if (kMask && U.lo >= U.hi) continue;         // nobody sees it: dK = dV = 0
                ok = mbar_wait(bar(C::KVB_KVEMPTY), (kvn & 1) ^ 1, w, 80);
                if (!ok) break;
                mbar_arrive_expect_tx(bar(C::KVB_KVFULL), 2 * C::TILE);
                load_tile<C::NCH>(&tm_k, base + C::KV_K_OFF, bar(C::KVB_KVFULL), U.h, U.m * 128, U.b);
                load_tile<C::NCH>(&tm_v, base + C::KV_V_OFF, bar(C::KVB_KVFULL), U.h, U.m * 128, U.b);
                ++kvn;
                if (kMask && kvn == 1) {
                    grid_wait();                             // (the first rows' statistics)
                    if constexpr (kScale) {
                        // e, ahead of the first Q tile, behind which the stores read it;
                        // then dq may be written (below)
                        *scale_slot =
                            *reinterpret_cast<const volatile int *>(reinterpret_cast<const float2 *>(a.dq) + a.parts);
                        grid_launch_dependents();
                    }
                }
                int qlo_t, qhi_t;
                query_range(U, qlo_t, qhi_t);
                // the query heads of this K/V head, each over its query tiles
                for (int k = 0, hq = U.h * a.group, i = qlo_t; ok && k < a.group * (qhi_t - qlo_t);
                     ++k, ++nq, i = i + 1 < qhi_t ? i + 1 : qlo_t, hq += i == qlo_t ? 1 : 0) {
                    if (kMask && k == max(0, a.group * (qhi_t - qlo_t) - 2)) ask();
                    const size_t wrow = (static_cast<size_t>(U.b) * a.H + hq) * a.NP;
                    // the elementwise warps read LSE2 and D of these 128
                    // columns: 2 x 512 B, four 128-byte lines each.  Measured:
                    // at d = 128 (little L1 next to 225 KB of shared memory)
                    // the lines are gone again by the time they are read; at
                    // d = 64 they stay (causal d = 64 +6 %).
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        asm volatile("prefetch.global.L1 [%0];" :: "l"(a.ws_l + wrow + i * 128 + l * 32));
                        asm volatile("prefetch.global.L1 [%0];" :: "l"(a.ws_d + wrow + i * 128 + l * 32));
                    }
                    ok = mbar_wait(bar(C::KVB_QEMPTY + RQ::slot(nq)), RQ::phase(nq) ^ 1, w, 81);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(C::KVB_QFULL + RQ::slot(nq)), C::TILE);
                    load_tile<C::NCH>(&tm_q, q_tile(nq), bar(C::KVB_QFULL + RQ::slot(nq)), hq, i * 128, U.b);
                    ++n_qc;
                    ok = mbar_wait(bar(C::KVB_DOEMPTY + RO::slot(nq)), RO::phase(nq) ^ 1, w, 82);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(C::KVB_DOFULL + RO::slot(nq)), C::TILE);
                    load_tile<C::NCH>(&tm_do, do_tile(nq), bar(C::KVB_DOFULL + RO::slot(nq)), hq, i * 128, U.b);
                    ++n_dc;
                }
            }
            if (kMask && clc_pending)
                mbar_wait_quiet(bar(C::KVB_CLCFULL), (kq - 1) & 1u, 500000000ull);
            else if (kDyn && clc_pending)
                mbar_wait_quiet(bar(C::KVB_CLCFULL + (kq - 1) % C::CLC_DEPTH),
                                ((kq - 1) / C::CLC_DEPTH) & 1u, 500000000ull);
            RQ::drain(n_qc, C::KVB_QFULL, base + C::KV_BAR_OFF);
            RO::drain(n_dc, C::KVB_DOFULL, base + C::KV_BAR_OFF);
            if (kvn > 0) mbar_wait_quiet(bar(C::KVB_KVFULL), (kvn - 1) & 1, 500000000ull);
        }
        __syncwarp();
    } else if (warp == 9) {
        // =================== MMA issuer ===================
        WaitCtx w{abort_flag, a.status, kRoleMma};
        uint32_t q_item = 0, kvph = 0, dsph = 0, accph = 0;
        bool ok = true;
        auto wait_q = [&](uint32_t i) {
            return mbar_wait_warp(bar(C::KVB_QFULL + RQ::slot(i)), RQ::phase(i), w, 91);
        };
        auto wait_do = [&](uint32_t i) {
            return mbar_wait_warp(bar(C::KVB_DOFULL + RO::slot(i)), RO::phase(i), w, 96);
        };
        uint32_t kq = 0;                            // causal: answers read
        auto next_dyn = [&]() __attribute__((always_inline)) -> int {
            if (!ok) return -1;
            const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
            ++kq;
            if (!mbar_wait_warp(bar(C::KVB_UNIT + q), ph, w, 94)) { ok = false; return -1; }
            const int nu = unit_slot[q];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::KVB_CLCEMPTY + q));
            return nu;
        };
        auto next_rec = [&](BwdUnit &U) __attribute__((always_inline)) -> int {
            if (!ok) return -1;
            const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
            ++kq;
            if (!mbar_wait_warp(bar(C::KVB_UNIT + q), ph, w, 66)) { ok = false; return -1; }
            const BwdRec r = read_bwd_rec(gbase + C::KV_REC_OFF, q);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::KVB_CLCEMPTY + q));
            U = bwd_unit(r);
            return r.id.x;
        };
        BwdUnit U;
        for (int u = kMask ? next_rec(U) : static_cast<int>(blockIdx.x), st = unit_stride0(snake);
                 ok && (!kDyn || u >= 0) && u < a.n_units_kv;
                 u = kMask ? next_rec(U) : kDyn ? next_dyn() : u + st, st = 2 * static_cast<int>(gridDim.x) - st) {
            if constexpr (!kMask) U = make_bwd_unit<kCausal, true, kWin>(u, a);
            int qlo_t, qhi_t;
            query_range(U, qlo_t, qhi_t);
            const int Ti = a.group * (qhi_t - qlo_t);    // query tiles of all the group's heads
            if (kMask && Ti <= 0) continue;
            ok = mbar_wait_warp(bar(C::KVB_KVFULL), kvph, w, 90);
            if (!ok) break;
            kvph ^= 1;
            // q_item counts the CTA's query tiles, and so its S^T tiles
            auto g1 = [&](uint32_t i) __attribute__((always_inline)) -> bool {
                if (!wait_q(i)) return false;
                tc_fence_after();
                gemm_ss_kmajor<D, kBatch>(tbase + C::st_col(i), base + C::KV_K_OFF, q_tile(i), C::IDESC_SS);
                mma_commit_elect(bar(C::st_bar(i)));
                return true;
            };
            ok = g1(q_item);
            if (!ok) break;
            ok = wait_do(q_item);
            if (!ok) break;
            tc_fence_after();
            gemm_ss_kmajor<D, kBatch>(tbase + C::KV_COL_DPT, base + C::KV_V_OFF, do_tile(q_item), C::IDESC_SS);
            mma_commit_elect(bar(C::KVB_DPTFULL));
            if (C::KV_SDB && Ti > 1) {               // the second buffer starts one tile ahead
                ok = g1(q_item + 1);
                if (!ok) break;
            }
            for (int k = 0; ok && k < Ti; ++k) {
                const uint32_t ic = q_item + k, in = ic + 1;
                const bool more = k + 1 < Ti;
                // ---- G3: dV += P^T dO_i (P^T at columns 32..95 of S^T) ----
                ok = mbar_wait_warp(bar(C::p_bar(ic)), C::st_par(ic), w, 92);
                if (ok && k == 0) ok = mbar_wait_warp(bar(C::KVB_ACCEMPTY), accph ^ 1, w, 93);
                if (!ok) break;
                if (k == 0) accph ^= 1;
                tc_fence_after();
                gemm_ts_mn<kBatch>(tbase + C::KV_COL_DV, tbase + C::st_col(ic) + 32, do_tile(ic), C::IDESC_ACC,
                           k > 0);
                mma_commit_elect(bar(C::KVB_DOEMPTY + RO::slot(ic)));
                // ---- G1 into the S^T buffer G3 has just read: tile i+2
                //      (two buffers) or i+1 (one) ----
                if (C::KV_SDB ? k + 2 < Ti : more) {
                    ok = g1(C::KV_SDB ? ic + 2 : in);
                    if (!ok) break;
                }
                // ---- G4: dK += dS^T Q_i (dS^T at columns 32..95 of dP^T) ----
                ok = mbar_wait_warp(bar(C::KVB_DSFULL), dsph, w, 95);
                if (!ok) break;
                dsph ^= 1;
                tc_fence_after();
                gemm_ts_mn<kBatch>(tbase + C::KV_COL_DK, tbase + C::KV_COL_DPT + 32, q_tile(ic), C::IDESC_ACC,
                           k > 0);
                mma_commit_elect(bar(C::KVB_QEMPTY + RQ::slot(ic)));
                // ---- G2(i+1) ----
                if (more) {
                    ok = wait_do(in);
                    if (!ok) break;
                    tc_fence_after();
                    gemm_ss_kmajor<D, kBatch>(tbase + C::KV_COL_DPT, base + C::KV_V_OFF, do_tile(in), C::IDESC_SS);
                    mma_commit_elect(bar(C::KVB_DPTFULL));
                }
            }
            if (!ok) break;
            mma_commit_elect(bar(C::KVB_ACCFULL));
            mma_commit_elect(bar(C::KVB_KVEMPTY));
            q_item += Ti;
        }
        mma_commit_elect(bar(C::KVB_MMADONE));
        mbar_wait_quiet(bar(C::KVB_MMADONE), 0, 500000000ull);
        __syncwarp();
    } else {
        // =================== elementwise group (warps 0-7) ===================
        if constexpr (kMask) {
            // This grid may have begun before the statistics' kernel ended: nothing of the
            // workspace is read ahead of this wait (ws_load).  Once it has ended, and every
            // CTA of this grid has begun (or been taken over), the dQ kernel's may begin on
            // SMs that run out of key tiles; it reads nothing that this one writes.  (kScale:
            // the producer says so, once it has read e from dq.)
            grid_wait();
            if (!kScale && warp == 0) grid_launch_dependents();
        }
        const int quarter = warp & 3, half = warp >> 2;
        const int row = quarter * 32 + lane;                 // key row of the tile
        const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
        const int col0 = half * 64;                          // this warp's query columns
        WaitCtx w{abort_flag, a.status, kRoleSoftmax0};
        const float sl2 = kCap ? a.sc_post : a.scale_log2;
        const float2 c2 = make_float2(sl2, sl2);
        uint32_t stn = 0, dpph = 0, accph = 0;    // stn: S^T tiles of this CTA so far
        bool ok = true;
        uint32_t kq = 0;                            // causal: answers read
        auto next_dyn = [&]() __attribute__((always_inline)) -> int {
            if (!ok) return -1;
            const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
            ++kq;
            ok = mbar_wait(bar(C::KVB_UNIT + q), ph, w, 103);
            if (__any_sync(0xffffffffu, !ok)) { ok = false; return -1; }
            const int nu = unit_slot[q];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::KVB_CLCEMPTY + q));
            return nu;
        };
        // Interval masks: the next unit's record, and this key's queries in it, are read
        // before the stores of the unit at hand.
        BwdRec rec_n{};
        int2 vis_n = make_int2(0, 0);
        auto fetch = [&]() __attribute__((always_inline)) -> int {
            const uint32_t q = kq % C::CLC_DEPTH, ph = (kq / C::CLC_DEPTH) & 1u;
            ++kq;
            ok = mbar_wait(bar(C::KVB_UNIT + q), ph, w, 103);
            if (__any_sync(0xffffffffu, !ok)) { ok = false; return -1; }
            rec_n = read_bwd_rec(gbase + C::KV_REC_OFF, q);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::KVB_CLCEMPTY + q));
            if (rec_n.id.x < 0) return -1;
            const int n = rec_n.id.w * 128 + row;
            vis_n = n < a.N ? __ldg(a.plan.cols + static_cast<size_t>(rec_n.id.y) * a.N + n) : make_int2(0, 0);
            return rec_n.id.x;
        };
        for (int u = kMask ? fetch() : static_cast<int>(blockIdx.x), st = unit_stride0(snake);
                 ok && (!kDyn || u >= 0) && u < a.n_units_kv;
                 u = kMask ? u : kDyn ? next_dyn() : u + st, st = 2 * static_cast<int>(gridDim.x) - st) {
            BwdUnit U;
            const bool padded = rec_n.range.z != 0;
            const int2 vis = vis_n;
            if constexpr (kMask) U = bwd_unit(rec_n);
            else U = make_bwd_unit<kCausal, true, kWin>(u, a);
            int i0, qhi_t;
            query_range(U, i0, qhi_t);
            const int Ti = qhi_t - i0;
            const int krow = U.m * 128 + row;
            if (kMask && Ti <= 0) {
                u = fetch();
                if (krow < a.N) {
                    const size_t at = ((static_cast<size_t>(U.b) * a.N + krow) * (a.H / a.group) + U.h) * D + half * (D / 2);
                    uint4 *zk = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.dk) + at);
                    uint4 *zv = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.dv) + at);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        zk[i] = make_uint4(0u, 0u, 0u, 0u);
                        zv[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                continue;
            }
            // this key row's visible queries (rows past N: any range)
            int qlo_r = 0, qhi_r = a.N;
            if constexpr (kMask) {
                qlo_r = vis.x;
                qhi_r = vis.y;
            } else if constexpr (kWin) {
                const int kr = min(krow, a.N - 1);
                qlo_r = win_qlo(kr, a);
                qhi_r = win_qhi(kr, a);
            }
            // LSE2 and D of a query tile are read below as broadcast loads
            // through L1, one per four columns, each feeding the next step of
            // a dependent loop.  At d = 128 the first read of each 32-byte
            // sector missed L1 and waited for L2 there (measured: 1 miss per
            // line, the producer's prefetch notwithstanding), so during tile k
            // lanes 0-7 load one word of each of the 8 sectors of tile k+1's
            // LSE2 [col0, col0+64) and lanes 8-15 those of D.  The word is
            // read only at the next tile (into `touched_sum`, which a store
            // the host rules out keeps alive), when the load has long landed.
            // Not with a softcap: its registers are spent (the loads spilled).
            float touched = 0.f, touched_sum = 0.f;
            // query head of the group, then its query tile
            for (int k = 0, hq = U.h * a.group, i = i0; k < a.group * Ti;
                 ++k, i = i + 1 < qhi_t ? i + 1 : i0, hq += i == i0 ? 1 : 0) {
                const size_t wrow = (static_cast<size_t>(U.b) * a.H + hq) * a.NP;
                const float4 *lse4 = reinterpret_cast<const float4 *>(a.ws_l + wrow + i * 128 + col0);
                const float4 *dd4 = reinterpret_cast<const float4 *>(a.ws_d + wrow + i * 128 + col0);
                touched_sum += touched;
                if (!kCap && k + 1 < a.group * Ti && lane < 16) {
                    const int i1 = i + 1 < qhi_t ? i + 1 : i0, hq1 = i1 == i0 ? hq + 1 : hq;
                    const size_t w1 = (static_cast<size_t>(U.b) * a.H + hq1) * a.NP + i1 * 128 + col0 +
                                      (lane & 7) * 8;
                    touched = ws_load<kMask>((lane < 8 ? a.ws_l : a.ws_d) + w1);
                }
                // this tile's LSE2, loaded before the wait for S^T so the
                // loads overlap it (D stays in the loop: 64 more registers
                // would spill under the 168 a thread has with ten warps; with
                // a softcap LSE2 is needed again in the dS step, so there it
                // stays in the loops too)
                float4 lse_v[16];
                if constexpr (!kCap) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) lse_v[c] = ws_load<kMask>(lse4 + c);
                }
                // ---- P^T = exp2(S^T c - LSE2[q]) ----
                ok = mbar_wait(bar(C::st_bar(stn)), C::st_par(stn), w, 100);
                if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
                tc_fence_after();
                uint32_t sv[64];
                const uint32_t tST = tbase + lane_off + C::st_col(stn);
                const int pbar = C::p_bar(stn);
                bool edge = false;               // interval masks: hidden columns may hold anything
                if constexpr (kMask) {
                    // a query tile that reaches outside the documents: its Q (S^T has been
                    // formed) and dO rows there become 0; dP^T, which may read them
                    // meanwhile, is masked in those columns
                    if (padded) {
                        const int4 live = __ldg(a.plan.live + U.b);
                        const bool outside = tile_outside(i, live);
                        edge = outside || tile_outside(U.m, live);
                        if (outside) {
                            ok = mbar_wait(bar(C::KVB_DOFULL + RO::slot(stn)), RO::phase(stn), w, 104);
                            if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
                            zero_outside<C::NCH>(gbase + C::KV_Q_OFF + RQ::slot(stn) * C::TILE, i * 128, row, half, live);
                            zero_outside<C::NCH>(gbase + C::KV_DO_OFF + RO::slot(stn) * C::TILE, i * 128, row, half, live);
                        }
                    }
                }
                ++stn;
                tmem_ld32(tST + col0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                tmem_ld32(tST + col0 + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                tmem_ld_wait();
                // causal: query column q sees this key row iff krow <= q
                int lo = (kCausal ? krow - i * 128 : 0) - col0;         // first visible column
                int hi = 1 << 30;                                       // one past the last
                if constexpr (kWin || kMask) {
                    lo = qlo_r - i * 128 - col0;
                    hi = qhi_r - i * 128 - col0;
                }
                // interval masks: as in the dQ kernel
                uint32_t seen[2] = {~0u, ~0u};
                bool whole = true;
                float beta = 0.f;
                const float d0 = static_cast<float>(krow - i * 128 - col0);
                if constexpr (kMask) {
                    whole = __all_sync(0xffffffffu, lo <= 0 && hi >= 64) && !(kBias && i == U.m);
                    if (!whole) {
                        seen[0] = column_bits(lo, hi);
                        seen[1] = column_bits(lo - 32, hi - 32);
                    }
                    if constexpr (kBias) beta = __ldg(a.slopes + hq) * 1.44269504088896340736f;
                }
                float *pf = reinterpret_cast<float *>(sv);
                uint32_t pk[32];
                if constexpr (kCap) {
                    // keep t = tanh(alpha s / c) in sv; P = 2^(t c log2(e) - LSE2)
#pragma unroll
                    for (int c = 0; c < 64; ++c) pf[c] = tanh_approx(pf[c] * a.sc_pre);
                }
                if constexpr (kMask) {
                    // (two copies: the rare one does without packed arithmetic)
                    if (whole) {
                        // (the columns step by their distances, which are exact, and the
                        // bias joins the LSE in one FMA: both may be large, each column
                        // with an LSE of its own)
                        const float bs = i < U.m ? -beta : beta;
                        const float2 bs2 = make_float2(bs, bs), four = make_float2(-4.f, -4.f);
                        float2 even = make_float2(d0, d0 - 1.f), odd = make_float2(d0 - 2.f, d0 - 3.f);
#pragma unroll
                        for (int c = 0; c < 64; c += 4) {
                            const float4 l4 = lse_v[c / 4];
                            float2 n01 = make_float2(-l4.x, -l4.y), n23 = make_float2(-l4.z, -l4.w);
                            if constexpr (kBias) {
                                n01 = __ffma2_rn(even, bs2, n01);
                                n23 = __ffma2_rn(odd, bs2, n23);
                                even = __fadd2_rn(even, four);
                                odd = __fadd2_rn(odd, four);
                            }
                            const float2 x01 = __ffma2_rn(make_float2(pf[c], pf[c + 1]), c2, n01);
                            const float2 x23 = __ffma2_rn(make_float2(pf[c + 2], pf[c + 3]), c2, n23);
                            pf[c + 0] = ex2_approx(x01.x);
                            pf[c + 1] = ex2_approx(x01.y);
                            pf[c + 2] = ex2_approx(x23.x);
                            pf[c + 3] = ex2_approx(x23.y);
                            pk[c / 2] = pack2<kBF16>(pf[c], pf[c + 1]);
                            pk[c / 2 + 1] = pack2<kBF16>(pf[c + 2], pf[c + 3]);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const float4 l4 = lse_v[c / 4];
#pragma unroll
                            for (int e = c; e < c + 2; ++e) {
                                const float l = (e & 3) == 0 ? l4.x : (e & 3) == 1 ? l4.y : (e & 3) == 2 ? l4.z : l4.w;
                                const float x = __fmaf_rn(pf[e], sl2, kBias ? __fmaf_rn(-beta, fabsf(d0 - e), -l) : -l);
                                pf[e] = (seen[e >> 5] & (1u << (e & 31))) ? ex2_approx(x) : 0.f;
                            }
                            pk[c / 2] = pack2<kBF16>(pf[c], pf[c + 1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        const float4 l4 = kCap ? ws_load<kMask>(lse4 + c / 4) : lse_v[c / 4];
                        const float2 x01 = __ffma2_rn(make_float2(pf[c], pf[c + 1]), c2,
                                                make_float2(-l4.x, -l4.y));
                        const float2 x23 = __ffma2_rn(make_float2(pf[c + 2], pf[c + 3]), c2,
                                                make_float2(-l4.z, -l4.w));
                        const float p0 = (c + 0 >= lo && (!kWin || c + 0 < hi)) ? ex2_approx(x01.x) : 0.f;
                        const float p1 = (c + 1 >= lo && (!kWin || c + 1 < hi)) ? ex2_approx(x01.y) : 0.f;
                        const float p2 = (c + 2 >= lo && (!kWin || c + 2 < hi)) ? ex2_approx(x23.x) : 0.f;
                        const float p3 = (c + 3 >= lo && (!kWin || c + 3 < hi)) ? ex2_approx(x23.y) : 0.f;
                        if constexpr (!kCap) {
                            pf[c + 0] = p0;
                            pf[c + 1] = p1;
                            pf[c + 2] = p2;
                            pf[c + 3] = p3;
                        }
                        pk[c / 2] = pack2<kBF16>(p0, p1);
                        pk[c / 2 + 1] = pack2<kBF16>(p2, p3);
                    }
                }
                // 16-bit P^T of query columns [col0, col0+64) -> S^T columns
                // 32 + col0/2 .. +32: columns this warp has read itself
                tmem_st32(tST + 32 + half * 32, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(pbar));
                // ---- dS^T = P^T o (dP^T - D[q]) ----
                ok = mbar_wait(bar(C::KVB_DPTFULL), dpph, w, 101);
                if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
                dpph ^= 1;
                tc_fence_after();
                uint32_t dp[64];
                const uint32_t tDPT = tbase + lane_off + C::KV_COL_DPT;
                tmem_ld32(tDPT + col0, *reinterpret_cast<uint32_t(*)[32]>(&dp[0]));
                tmem_ld32(tDPT + col0 + 32, *reinterpret_cast<uint32_t(*)[32]>(&dp[32]));
                tmem_ld_wait();
                if constexpr (kMask) {
                    if (edge) {                  // dP of a row or key outside may be NaN
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!(seen[c >> 5] & (1u << (c & 31)))) dp[c] = 0u;
                    }
                }
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const float4 d4 = ws_load<kMask>(dd4 + c / 4);
                    const float2 g01 = __fadd2_rn(
                        make_float2(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1])),
                        make_float2(-d4.x, -d4.y));
                    const float2 g23 = __fadd2_rn(
                        make_float2(__uint_as_float(dp[c + 2]), __uint_as_float(dp[c + 3])),
                        make_float2(-d4.z, -d4.w));
                    float2 p01 = make_float2(pf[c], pf[c + 1]), p23 = make_float2(pf[c + 2], pf[c + 3]);
                    if constexpr (kCap) {
                        // P again from t, times dS/du = 1 - t^2
                        const float4 l4 = ws_load<kMask>(lse4 + c / 4);
                        const float2 x01 = __ffma2_rn(p01, c2, make_float2(-l4.x, -l4.y));
                        const float2 x23 = __ffma2_rn(p23, c2, make_float2(-l4.z, -l4.w));
                        const float2 t01 = __ffma2_rn(make_float2(-p01.x, -p01.y), p01, make_float2(1.f, 1.f));
                        const float2 t23 = __ffma2_rn(make_float2(-p23.x, -p23.y), p23, make_float2(1.f, 1.f));
                        p01.x = (c + 0 >= lo && (!kWin || c + 0 < hi)) ? ex2_approx(x01.x) * t01.x : 0.f;
                        p01.y = (c + 1 >= lo && (!kWin || c + 1 < hi)) ? ex2_approx(x01.y) * t01.y : 0.f;
                        p23.x = (c + 2 >= lo && (!kWin || c + 2 < hi)) ? ex2_approx(x23.x) * t23.x : 0.f;
                        p23.y = (c + 3 >= lo && (!kWin || c + 3 < hi)) ? ex2_approx(x23.y) * t23.y : 0.f;
                    }
                    const float2 ds01 = __fmul2_rn(p01, g01);
                    const float2 ds23 = __fmul2_rn(p23, g23);
                    pk[c / 2] = pack2<kBF16>(ds01.x, ds01.y);
                    pk[c / 2 + 1] = pack2<kBF16>(ds23.x, ds23.y);
                }
                tmem_st32(tDPT + 32 + half * 32, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::KVB_DSFULL));
            }
            if (!ok) break;
            if constexpr (kMask) {
                u = fetch();
                if (!ok) break;
            }
            // ---- epilogue: dV, dK * alpha -> global (this warp's half of the columns) ----
            ok = mbar_wait(bar(C::KVB_ACCFULL), accph, w, 102);
            if (__any_sync(0xffffffffu, !ok)) { ok = false; break; }
            accph ^= 1;
            tc_fence_after();
            const float undo = kScale ? __int_as_float((127 - *scale_slot) << 23) : 1.f;      // 2^-e
            constexpr int W = D / 2;
            uint32_t acc[W];
#pragma unroll
            for (int ch = 0; ch < W / 32; ++ch)
                tmem_ld32(tbase + lane_off + C::KV_COL_DV + half * W + ch * 32,
                          *reinterpret_cast<uint32_t(*)[32]>(&acc[ch * 32]));
            tmem_ld_wait();
            store_cols<D, W, kBF16>(a.dv, a, a.H / a.group, U.b, U.h, krow, half * W, acc, undo);
#pragma unroll
            for (int ch = 0; ch < W / 32; ++ch)
                tmem_ld32(tbase + lane_off + C::KV_COL_DK + half * W + ch * 32,
                          *reinterpret_cast<uint32_t(*)[32]>(&acc[ch * 32]));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::KVB_ACCEMPTY));
            store_cols<D, W, kBF16>(a.dk, a, a.H / a.group, U.b, U.h, krow, half * W, acc, kScale ? a.alpha * undo : a.alpha);
            if constexpr (!kCap) {
                if (a.N < 0 && touched_sum == 0.f) a.status[3] = 1u;    // never true: N >= 1
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tbase, C::TMEM_COLS);
    }
}

}  // namespace fa
