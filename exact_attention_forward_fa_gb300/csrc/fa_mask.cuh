// fa_mask.cuh -- the plan of a document / prefix / window mask: the visible keys of
// every token and the visible queries of every key as intervals, the key and query
// tiles of every work unit, and the order in which units are taken.
//
// Sequence b is packed with documents docs[k] .. docs[k + 1]; token i of document
// [s, e) with prefix p sees the keys of
//     [max(s, i - wl), min(e, max(i + 1 + wr, s + p)))         (a bound of -1: none)
// and key j is seen by the queries of [qlo, qhi): from s when it is in the prefix or
// wr < 0, else from max(s, j - wr); to e, or j + wl + 1 with a left bound.  Both ends
// grow with i and j, so the union over a tile's tokens is bounded by the first
// token's low end and the last one's high end.  Tokens outside every document
// (before docs[0] and from docs[D] on) see nothing and are not seen.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace fa {

// The plan in one device buffer.  Records are sorted by their number of tiles, the
// longest first.
struct MaskPlan {
    const int4 *live;    // [B] {first token of a document, one past the last, 0, 0}
    const int4 *pairs;   // [B][n_p][2] {pair p, lo, hi, live.x} of tile 2p, {0, lo, hi, live.y} of 2p + 1: key tiles
    const int4 *qtiles;  // [B][n_t] {query tile, lo, hi, 0}: key tiles
    const int4 *ktiles;  // [B][n_t] {key tile, lo, hi, 0}: query tiles
    const int2 *rows;    // [B][N] visible keys of a token
    const int2 *cols;    // [B][N] queries that see a key
};

// Bytes of the plan; *m gets its parts when base is given.
inline size_t mask_plan_layout(int B, int N, const void *base, MaskPlan *m) {
    const size_t n_t = (static_cast<size_t>(N) + 127) / 128, n_p = (n_t + 1) / 2, b = static_cast<size_t>(B);
    const char *p = static_cast<const char *>(base);
    size_t at = 0;
    auto part = [&](size_t bytes) { const size_t o = at; at += (bytes + 15) & ~static_cast<size_t>(15); return o; };
    const size_t live = part(16 * b), pairs = part(32 * b * n_p), qt = part(16 * b * n_t), kt = part(16 * b * n_t),
                 rows = part(8 * b * N), cols = part(8 * b * N);
    if (m) {
        m->live = reinterpret_cast<const int4 *>(p + live);
        m->pairs = reinterpret_cast<const int4 *>(p + pairs);
        m->qtiles = reinterpret_cast<const int4 *>(p + qt);
        m->ktiles = reinterpret_cast<const int4 *>(p + kt);
        m->rows = reinterpret_cast<const int2 *>(p + rows);
        m->cols = reinterpret_cast<const int2 *>(p + cols);
    }
    return at;
}

struct MaskPlanArgs {
    const int *docs;     // [B][D + 1]
    const int *prefix;   // [B][D] or nullptr
    int *positions;      // [B][N] or nullptr (written)
    MaskPlan plan;       // (written)
    uint32_t *status;
    int B, N, D, wl, wr;
};
cudaError_t launch_mask_plan(const MaskPlanArgs &a, cudaStream_t stream);

}  // namespace fa
