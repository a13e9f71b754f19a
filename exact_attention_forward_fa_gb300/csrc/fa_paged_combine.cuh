// fa_paged_combine.cuh -- joins the parts of cut units of the attention over a
// paged cache.
#pragma once

#include "fa_paged.cuh"

namespace fa {

// Joins the parts of the units that the shares' borders cut: LSE = log sum_s
// exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.  CTA (c, y) works on the cut unit
// that starts in share c; its part 0 is slot 2 c + 1, part s > 0 slot 2 (c + s).
// A part with LSE = -inf saw nothing and its O may be unwritten: it is not
// read.  Up to eight parts: a warp a row for few rows (kFew), eight lanes a row
// and four rows a warp for a chunk's (11 against 18 us for 152 cut units of 256
// rows; for few rows 4 us the first way, 5 us the second).  More (single tokens against a long cache, a
// part for every SM): the CTA takes a row, each warp every eighth part, and
// the warps' sums are added in order.
template <int D, bool kBF16, bool kFew>
__global__ void __launch_bounds__(256) fa_paged_combine_kernel(const PagedArgs a, const PagedWork wk, const int R) {
    constexpr int E = D / 32;
    __shared__ float s_acc[8][D];
    __shared__ float s_l[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 *d4 = reinterpret_cast<const int4 *>(wk.desc + 8 * c);
    const int4 d0 = d4[0], d1 = d4[1];
    const int parts = d0.x, qrow = d0.y, nl = d0.z, nh = d0.w, h = d1.x;
    if (parts == 0) return;
    const int rows = (nl + nh) * a.group;
    auto slot = [&](int s, int tile, int row) __attribute__((always_inline)) -> size_t {
        return (static_cast<size_t>(s == 0 ? 2 * c + 1 : 2 * (c + s)) * 2 + tile) * 128 + row;
    };
    auto write = [&](int tile, int row, const float (&acc)[E], float M, float L) __attribute__((always_inline)) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int tok = qrow + tile * R + row / a.group, qh = h * a.group + row % a.group;
        uint32_t pk[E / 2];
#pragma unroll
        for (int e = 0; e < E; e += 2) pk[e / 2] = pack2<kBF16>(acc[e] * inv, acc[e + 1] * inv);
        uint16_t *dst = reinterpret_cast<uint16_t *>(a.o) + (static_cast<size_t>(tok) * a.H + qh) * D + lane * E;
        if constexpr (E == 2) *reinterpret_cast<uint32_t *>(dst) = pk[0];
        else *reinterpret_cast<uint2 *>(dst) = make_uint2(pk[0], pk[1]);
        if (a.lse != nullptr && lane == 0)
            a.lse[static_cast<size_t>(qh) * a.T + tok] =
                L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
    };
    auto load = [&](size_t part, float (&v)[E]) __attribute__((always_inline)) {
        const float *src = wk.o + part * D + lane * E;
        if constexpr (E == 2) {
            const float2 t = *reinterpret_cast<const float2 *>(src);
            v[0] = t.x; v[1] = t.y;
        } else {
            const float4 t = *reinterpret_cast<const float4 *>(src);
            v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
        }
    };
    if (kFew && parts <= 8) {
        for (int rr = blockIdx.y * 8 + warp; rr < rows; rr += gridDim.y * 8) {
            float z[8], v[8][E], acc[E];
#pragma unroll
            for (int s = 0; s < 8; ++s) z[s] = s < parts ? wk.lse[slot(s, 0, rr)] : -INFINITY;
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (s < parts) load(slot(s, 0, rr), v[s]);
            float M = z[0], L = 0.f;
#pragma unroll
            for (int s = 1; s < 8; ++s) M = fmaxf(M, z[s]);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                if (z[s] == -INFINITY) continue;
                const float wt = ex2_approx(z[s] - M);
                L += wt;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, v[s][e], acc[e]);
            }
            write(0, rr, acc, M, L);
        }
        return;
    }
    if (!kFew && parts <= 8) {
        const int sub = lane & 7;                          // float4 sub, sub + 8, ... of the row
        constexpr int F = D / 32;
#pragma unroll 1
        for (int r4 = (blockIdx.y * 8 + warp) * 4; r4 < rows; r4 += gridDim.y * 32) {
            const int rr = r4 + (lane >> 3);
            if (rr >= rows) continue;
            const int tile = rr >= nl * a.group ? 1 : 0, row = tile ? rr - nl * a.group : rr;
            float z[8], M = -INFINITY, L = 0.f;
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                z[s] = s < parts ? wk.lse[slot(s, tile, row)] : -INFINITY;
                M = fmaxf(M, z[s]);
            }
            float4 acc[F];
#pragma unroll
            for (int f = 0; f < F; ++f) acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int s0 = 0; s0 < 8; s0 += 4) {
                if (s0 >= parts) continue;
                float4 v[4][F];                            // four parts in flight
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float4 *src =
                        reinterpret_cast<const float4 *>(wk.o + slot(min(s0 + s, parts - 1), tile, row) * D) + sub;
#pragma unroll
                    for (int f = 0; f < F; ++f) v[s][f] = src[8 * f];
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (z[s0 + s] == -INFINITY) continue;
                    const float wt = ex2_approx(z[s0 + s] - M);
                    L += wt;
#pragma unroll
                    for (int f = 0; f < F; ++f) {
                        acc[f].x = fmaf(wt, v[s][f].x, acc[f].x);
                        acc[f].y = fmaf(wt, v[s][f].y, acc[f].y);
                        acc[f].z = fmaf(wt, v[s][f].z, acc[f].z);
                        acc[f].w = fmaf(wt, v[s][f].w, acc[f].w);
                    }
                }
            }
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const int tok = qrow + tile * R + row / a.group, qh = h * a.group + row % a.group;
            uint2 *dst = reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(a.o) +
                                                   (static_cast<size_t>(tok) * a.H + qh) * D) + sub;
#pragma unroll
            for (int f = 0; f < F; ++f)
                dst[8 * f] = make_uint2(pack2<kBF16>(acc[f].x * inv, acc[f].y * inv),
                                        pack2<kBF16>(acc[f].z * inv, acc[f].w * inv));
            if (a.lse != nullptr && sub == 0)
                a.lse[static_cast<size_t>(qh) * a.T + tok] =
                    L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
        }
        return;
    }
    for (int rr = blockIdx.y; rr < rows; rr += gridDim.y) {
        const int tile = rr >= nl * a.group ? 1 : 0, row = tile ? rr - nl * a.group : rr;
        float M = -INFINITY;
        for (int s = lane; s < parts; s += 32) M = fmaxf(M, wk.lse[slot(s, tile, row)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float l = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        for (int s0 = warp; s0 < parts; s0 += 32) {
            float z[4], v[4][E];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int s = s0 + 8 * u;
                z[u] = s < parts ? wk.lse[slot(s, tile, row)] : -INFINITY;
                if (s < parts) load(slot(s, tile, row), v[u]);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (z[u] == -INFINITY) continue;
                const float wt = ex2_approx(z[u] - M);
                l += wt;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = fmaf(wt, v[u][e], acc[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
        if (lane == 0) s_l[warp] = l;
        __syncthreads();
        if (warp == 0) {
            float L = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                L += s_l[q];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += s_acc[q][lane * E + e];
            }
            write(tile, row, acc, M, L);
        }
        __syncthreads();
    }
}

}  // namespace fa
