// fa_rope.cuh -- rotary positions: argument records of fa_rope and
// fa_paged_rope_append.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace fa {

struct RopeArgs {
    // [T][heads][d], the strides in 16-byte vectors from token to token
    const void *q, *k, *v;            // v, k_pages, v_pages: the paged form alone
    void *q_out, *k_out;
    long long q_stride, k_stride, v_stride, qo_stride, ko_stride;
    const double *inv_freq;           // [rot / 2], radians a position
    const int *positions;             // dense: [T], or null: the row within its sequence of N
    int T, N;
    int H, H_kv, V;                   // V: 16-byte vectors of a head, d / 8
    int rot;                          // rotated elements of a head, a multiple of 16
    float scale;                      // of the rotated elements
    bool interleaved, inverse;
    // paged form (fa_paged.cuh): k and v go to their pages
    void *k_pages, *v_pages;
    const int *table, *kv_len, *cu_q, *offsets;
    uint32_t *status;
    long long page_stride;            // in vectors
    int B, W, ps_log2, n_pages;
};

// bf16 data, or fp16; paged: with k and v to their pages.
cudaError_t launch_rope(const RopeArgs &a, bool bf16, bool paged, int sm_count, cudaStream_t stream);

}  // namespace fa
