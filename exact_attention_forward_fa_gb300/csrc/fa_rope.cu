// fa_rope.cu -- rotary positions (fa_rope) and the serving form that rotates the
// new tokens' queries and keys and writes keys and values into their pages in
// one launch (fa_paged_rope_append).
//
// Pair c of a head, (x0, x1), at position p becomes
//     y0 = m (x0 cos t - x1 sin t),  y1 = m (x1 cos t + x0 sin t),  t = p w_c;
// the inverse (the gradient's way back) turns by -t.  Elements from `rot` on are
// copied.
//
// The angle.  p w_c in FP32 is off by p 2^-24, 0.06 rad at a million.  FP64 has few
// units here, so the angle is kept as a fraction of a turn in 64-bit integers:
// u_c = w_c / (2 pi) 2^64 (mod 2^64), formed once a thread from the bits of
// the double w_c, and p u_c mod 2^64 is the turn at p, whole turns dropped by the
// overflow.  Its upper 32 bits give the half-turns in [-1, 1) for sincospif:
// |p| 2^-53 relative to a turn, plus 2^-25 half-turns of the conversion.
//
// What bounds it: HBM, one read and one write of every element.  A warp takes
// one token at a time; a head has d / 16 tasks of two 16-byte vectors (the two
// halves of eight pairs, eight neighbouring pairs, or 16 copied elements), so a
// lane has the same eight pairs for all heads that it meets: the angles are
// formed once a token and the turns u_c once a warp.
//
// Measured (GB300): 16384 tokens of 16 + 16 heads of 128, slices of wider rows
// (268 MB in and out), 48 us, 5.6 TB/s; half of 40 heads at 6002 tokens, interleaved
// (123 MB), 26 us; chunks of 11921 tokens into pages (293 MB) 54 us; plain copies of as
// many bytes 47, 25 and 50 us; 64 single
// tokens 4.8 us, a launch and the chain offsets, length, page, store.  Runs of equal
// length took the place of whole tokens a warp (2.5 and 4.2 rounds of them: 27.4 and
// 61.6 us).  2 to 4 blocks of 8 warps an SM and 2 to 6 passes in flight lie within
// 5 % of one another; packed FP32 arithmetic changed nothing.
#include <climits>

#include "fa_paged.cuh"
#include "fa_rope.cuh"

namespace fa {

namespace {

// w / (2 pi) as a fraction of 2^64: w = +-M 2^(e - 63) with M in [2^63, 2^64), and
// 1 / (2 pi) = K 2^-66 with K = round(2^66 / (2 pi)); turns 2^64 = M K 2^-64 2^(e - 1).
__device__ __forceinline__ unsigned long long turns_of(double w) {
    const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(w));
    const int ex = static_cast<int>((bits >> 52) & 0x7ff);
    if (ex == 0) return 0ull;                               // zero (subnormals turn nothing)
    const unsigned long long M = (bits << 11) | (1ull << 63);
    const unsigned long long t = __umul64hi(M, 0xA2F9836E4E44152Aull);   // in [2^62, 2^64)
    const int s = (ex - 1023) - 1;                          // t 2^s
    unsigned long long u = s <= -64 || s >= 64 ? 0ull : s < 0 ? t >> -s : t << s;
    return (bits >> 63) ? 0ull - u : u;
}

// Eight pairs of 16-bit values: x0 and x1 packed two a word (half layout: the words
// of both vectors; interleaved: a pair a word).
template <bool kBF16>
__device__ __forceinline__ void turn8(uint4 &a, uint4 &b, bool interleaved, const float *cs, const float *sn) {
    uint32_t *w0 = reinterpret_cast<uint32_t *>(&a), *w1 = reinterpret_cast<uint32_t *>(&b);
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t &w = i < 4 ? w0[i] : w1[i - 4];
            float x0, x1;
            unpack2<kBF16>(w, x0, x1);
            w = pack2<kBF16>(__fmaf_rn(x0, cs[i], -__fmul_rn(x1, sn[i])), __fmaf_rn(x1, cs[i], __fmul_rn(x0, sn[i])));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x0, x1, y0, y1;
            unpack2<kBF16>(w0[i], x0, y0);
            unpack2<kBF16>(w1[i], x1, y1);
            w0[i] = pack2<kBF16>(__fmaf_rn(x0, cs[2 * i], -__fmul_rn(x1, sn[2 * i])),
                                 __fmaf_rn(y0, cs[2 * i + 1], -__fmul_rn(y1, sn[2 * i + 1])));
            w1[i] = pack2<kBF16>(__fmaf_rn(x1, cs[2 * i], __fmul_rn(x0, sn[2 * i])),
                                 __fmaf_rn(y1, cs[2 * i + 1], __fmul_rn(y0, sn[2 * i + 1])));
        }
    }
}

constexpr int kPasses = 2;      // heads in flight per lane: 4 loads of 16 bytes
constexpr int kBlocks = 3;      // blocks of 8 warps an SM

}  // namespace

// All tokens' passes, 32 / G heads each (G lanes a head), in a row, cut into equal
// runs for the warps: a run begins and ends within a token.
template <bool kBF16, bool kPaged>
__global__ void __launch_bounds__(256, kBlocks)
fa_rope_kernel(const RopeArgs a, const int G, const int passes, const int warps) {
    if (kPaged && blockIdx.x == gridDim.x - 1)              // the last block only checks
        return paged_check_seqs(a.cu_q, a.kv_len, a.B, a.T, a.W, a.ps_log2, a.status);
    const int warp = static_cast<int>((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
    if (warp >= warps) return;
    const int lane = threadIdx.x & 31;
    const int c = lane % G, sub = lane / G, hpp = 32 / G;   // task, head of a pass, heads a pass
    const bool turns = c * 16 < a.rot;
    // the task's two vectors within a head
    const int v0 = !turns || a.interleaved ? 2 * c : c, v1 = !turns || a.interleaved ? 2 * c + 1 : c + a.rot / 16;
    unsigned long long u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = turns ? turns_of(a.inv_freq[8 * c + i]) : 0ull;
    const int heads = a.H + a.H_kv * (kPaged ? 2 : 1);
    const uint4 *qs = reinterpret_cast<const uint4 *>(a.q), *ks = reinterpret_cast<const uint4 *>(a.k),
                *vs = reinterpret_cast<const uint4 *>(a.v);
    const long long total = static_cast<long long>(a.T) * passes;
    const long long p0 = total * warp / warps;
    int left = static_cast<int>(total * (warp + 1) / warps - p0);
    int t = static_cast<int>(p0 / passes), pass = static_cast<int>(p0 - static_cast<long long>(t) * passes);
    // paged: what the run's tokens of one sequence and of one page share (looked up
    // for each token, the chain of loads cost chunks 3 us of 56)
    int b = -1, end = INT_MIN, index = -1, page = -1;        // tokens of b end there; page number `index`
    long long len = 0;
    for (; left > 0; ++t, pass = 0) {
        const int n = min(passes - pass, left);
        left -= n;
        const int h_end = min(heads, (pass + n) * hpp);
        const uint4 *qt = qs + t * a.q_stride, *kt = ks + t * a.k_stride, *vt = vs + t * a.v_stride;
        uint4 x0[kPasses], x1[kPasses];
        auto load = [&](int h) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int hh = h + i * hpp;
                if (hh < h_end) {
                    // (values keep their order: the whole head is copied, two vectors a lane)
                    const bool is_v = kPaged && hh >= a.H + a.H_kv;
                    const uint4 *src = hh < a.H ? qt + hh * a.V : is_v ? vt + (hh - a.H - a.H_kv) * a.V : kt + (hh - a.H) * a.V;
                    x0[i] = src[is_v ? 2 * c : v0];
                    x1[i] = src[is_v ? 2 * c + 1 : v1];
                }
            }
        };
        int h = pass * hpp + sub;
        load(h);
        long long pos;
        uint4 *kd = nullptr, *vd = nullptr;                  // paged: the token's slot
        if constexpr (kPaged) {
            if (t >= end) {
                b = paged_find_seq(a.cu_q, a.B, t);
                if (b < 0) continue;                         // behind the last sequence
                end = a.cu_q[b + 1];
                len = a.kv_len[b];
                index = -1;
            }
            const long long p = len - end + t;
            pos = p + (a.offsets ? a.offsets[b] : 0);
            if (p >= 0 && p < min(len, static_cast<long long>(a.W) << a.ps_log2)) {
                if (static_cast<int>(p >> a.ps_log2) != index) {
                    index = static_cast<int>(p >> a.ps_log2);
                    page = paged_page(a.table + static_cast<long long>(b) * a.W, static_cast<int>(p), a.ps_log2,
                                      a.n_pages, a.status);
                }
                if (page >= 0) {
                    const long long at = static_cast<long long>(page) * a.page_stride +
                                         (p & ((1 << a.ps_log2) - 1)) * (static_cast<long long>(a.H_kv) * a.V);
                    kd = reinterpret_cast<uint4 *>(a.k_pages) + at;
                    vd = reinterpret_cast<uint4 *>(a.v_pages) + at;
                }
            }
        } else {
            pos = a.positions ? a.positions[t] : t % a.N;
            kd = reinterpret_cast<uint4 *>(a.k_out) + t * a.ko_stride;
        }
        uint4 *qd = reinterpret_cast<uint4 *>(a.q_out) + t * a.qo_stride;
        float cs[8], sn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned long long at = u[i] * static_cast<unsigned long long>(pos);
            float s, co;
            sincospif(static_cast<float>(static_cast<int>(at >> 32)) * 0x1p-31f, &s, &co);
            cs[i] = co * a.scale;
            sn[i] = a.inverse ? -s * a.scale : s * a.scale;
        }
        for (;;) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int hh = h + i * hpp;
                if (hh >= h_end) continue;
                const bool is_v = kPaged && hh >= a.H + a.H_kv;
                if (turns && !is_v) turn8<kBF16>(x0[i], x1[i], a.interleaved, cs, sn);
                uint4 *dst = hh < a.H ? qd + hh * a.V
                             : is_v   ? (vd ? vd + (hh - a.H - a.H_kv) * a.V : nullptr)
                                      : (kd ? kd + (hh - a.H) * a.V : nullptr);
                if (dst) {
                    dst[is_v ? 2 * c : v0] = x0[i];
                    dst[is_v ? 2 * c + 1 : v1] = x1[i];
                }
            }
            h += kPasses * hpp;
            if (h - sub >= h_end) break;
            load(h);
        }
    }
}

cudaError_t launch_rope(const RopeArgs &a, bool bf16, bool paged, int sm_count, cudaStream_t stream) {
    const int G = a.V / 2, hpp = 32 / G;
    const int heads = a.H + a.H_kv * (paged ? 2 : 1);
    const int passes = (heads + hpp - 1) / hpp;
    // as many warps as the SMs hold, a pass each at least (single tokens: spread
    // over all SMs)
    const long long total = static_cast<long long>(a.T) * passes, most = 8ll * kBlocks * sm_count;
    const int warps = static_cast<int>(total < most ? total : most);
    const unsigned grid = static_cast<unsigned>((warps + 7) / 8 + (paged ? 1 : 0));
    auto kern = paged ? (bf16 ? fa_rope_kernel<true, true> : fa_rope_kernel<false, true>)
                      : (bf16 ? fa_rope_kernel<true, false> : fa_rope_kernel<false, false>);
    kern<<<grid, 256, 0, stream>>>(a, G, passes, warps);
    return cudaGetLastError();
}

}  // namespace fa
