/*
 * fa.h -- C ABI of libfa: exact attention forward for NVIDIA GB300 (sm_103a).
 *
 * The operation ("FlashAttention-3 on Hopper", sec. 3.1 and 4.1-4.7; the
 * Blackwell schedule in "FlashAttention v1-v4", FA4 sections):
 *
 *     S = alpha * Q K^T  (+ causal mask: key j hidden from query i when
 *                          j > i, i.e. col > row + (Nk - Nq) with Nq = Nk)
 *     O = softmax_rows(S) V
 *     LSE_i = log sum_j exp(S_ij)                    (natural log)
 *
 * computed tile by tile with an online softmax, so the N x N score matrix
 * never reaches device memory.  Rows with no visible key would give O = 0,
 * LSE = -inf ("FlashAttention-3 on Hopper", sec. 4.6); with Nq = Nk every
 * row sees at least one key.
 *
 * Layouts (all contiguous, row-major):
 *     Q, K, V, O : [B][N][H][d]   (batch, sequence, head, head dim),
 *                                 element (b,n,h,c) at ((b*N + n)*H + h)*d + c
 *     LSE        : [B][H][N]      float32, element (b,h,n) at (b*H + h)*N + n
 *     FP8 scales : [B][H][ceil(N/128)] float32, one per 128-row tile of a head
 *     paged cache: pools of pages with their own strides (see "Paged
 *                  key/value cache" below)
 *
 * Conventions for every entry point:
 *   * Pointers named q, k, v, o, lse, x, x8, *_scale, *_pages, *_table,
 *     scores*, kv_len, cu_q, kept, new_len are DEVICE pointers owned by the
 *     caller; the library never frees or keeps them.
 *   * `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls are asynchronous: they validate, launch and return.
 *   * Arguments are validated on the host before anything is launched; a
 *     failed check returns an error code and launches nothing.
 *   * The library allocates no device memory per call.  It owns one small
 *     per-device status word in a static __device__ variable that kernels
 *     set when a bounded wait gives up or a device-side index is out of
 *     range; fa_check_status reads it.
 *   * Results are deterministic for fixed inputs: fixed reduction order, no
 *     atomics on outputs.
 *   * Thread safety: entry points may be called from several host threads;
 *     the per-device caches inside are guarded by a mutex.
 */
#ifndef FA_H_
#define FA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,  /* null pointer, non-positive size, bad flag, non-finite alpha */
    FA_ERR_UNSUPPORTED = 2,  /* head dim or dtype without a kernel, or not an sm_103 device */
    FA_ERR_MISALIGNED = 3,   /* a tensor pointer is not 16-byte aligned (TMA rule) */
    FA_ERR_TOO_LARGE = 4,    /* a size exceeds the TMA descriptor limits */
    FA_ERR_CUDA = 5,         /* a CUDA runtime/driver call or the launch failed */
    FA_ERR_TIMEOUT = 6,      /* a kernel's bounded wait gave up (fa_check_status) */
    FA_ERR_BAD_INDEX = 7     /* a page id, length or offset in device memory was out of
                                range; the access was skipped (fa_check_status) */
} fa_status;

typedef enum {
    FA_BF16 = 0,
    FA_FP16 = 1
} fa_dtype;

/* Scale granularity of the FP8 pre-pass (fa_quantize_fp8_granular). */
typedef enum {
    FA_SCALE_TILE = 0,    /* one scale per 128-row tile of a head (block quantization) */
    FA_SCALE_HEAD = 1,    /* one scale per (batch, head) */
    FA_SCALE_TENSOR = 2   /* one scale for the whole tensor */
} fa_scale_granularity;

/*
 * fa_fwd -- exact attention forward, BF16 or FP16 in and out.
 *   q, k, v : device, [B][N][H][d] in `dtype`, 16-byte aligned.
 *   o       : device, [B][N][H][d] in `dtype`, 16-byte aligned (written).
 *   lse     : device, float [B][H][N], 4-byte aligned, or NULL to skip.
 *   B, H, N : >= 1.  d in {64, 128, 256}; other head dims return
 *             FA_ERR_UNSUPPORTED.
 *   alpha   : the score scale (usually 1/sqrt(d)); must be finite.
 *   causal  : 0 or 1.
 * Accumulation is FP32; P is rounded to `dtype` before the P V product and
 * the softmax denominator sums those same rounded values; O is rounded to
 * `dtype` round-to-nearest-even.
 * Causal launches have one CTA per work unit and let running CTAs take over
 * those not yet started (cluster launch control), in an order that keeps
 * groups of heads together for L2 reuse of K and V; which CTA computes a
 * tile varies from launch to launch, the results do not.
 */
fa_status fa_fwd(const void *q, const void *k, const void *v, void *o,
                 float *lse, int B, int H, int N, int d, float alpha,
                 int causal, fa_dtype dtype, void *stream);

/*
 * fa_fwd_gqa -- fa_fwd with grouped key/value heads (grouped-query and
 * multi-query attention: "FlashAttention-3 on Hopper", ch. 11 and the GQA
 * remark of sec. 7.2.3): q, o are [B][N][H][d] as in fa_fwd, k, v are
 * [B][N][H_kv][d], H_kv >= 1 divides H, and query head h attends with key /
 * value head h / (H / H_kv).  H_kv = H is fa_fwd; H_kv = 1 is multi-query
 * attention.  H % H_kv != 0 or H_kv < 1 returns FA_ERR_INVALID_ARG; other
 * arguments, results and errors as fa_fwd.
 */
fa_status fa_fwd_gqa(const void *q, const void *k, const void *v, void *o,
                     float *lse, int B, int H, int H_kv, int N, int d,
                     float alpha, int causal, fa_dtype dtype, void *stream);

/*
 * fa_fwd_gqa_packed -- fa_fwd_gqa with the g = H / H_kv query heads of each
 * key/value head packed into the rows of one Q tile ("PackGQA" of the GQA
 * remark in "FlashAttention-3 on Hopper"): a tile holds 128 / g query
 * positions of all g heads, so one pass over a key/value head's K and V
 * serves the whole group and short sequences do not leave tiles half
 * empty.  Same arguments, layouts, results (up to FP32 rounding order: the
 * softmax's rescale decisions are taken per warp of rows) and errors as
 * fa_fwd_gqa; additionally d must be 64 or 128 and g must divide 128
 * (g = 1 runs fa_fwd_gqa), else FA_ERR_UNSUPPORTED.  Measured on GB300
 * (H 32 over H_kv 2 or 8, d 128): N = 64 twice the throughput of
 * fa_fwd_gqa, N = 256 about the same, N = 4096 2-5 % below it -- a choice
 * for short sequences.
 */
fa_status fa_fwd_gqa_packed(const void *q, const void *k, const void *v, void *o,
                            float *lse, int B, int H, int H_kv, int N, int d,
                            float alpha, int causal, fa_dtype dtype, void *stream);

/*
 * fa_fwd_ext -- fa_fwd_gqa with the score and mask variants of
 * "FlashAttention-3 on Hopper" sec. 4.6 (learnable sinks folded into the
 * row sum at finalize) and sec. 4.7 (local / sliding-window masks; a score
 * transformation precedes the mask), and the softcap of "03 FA3" sec. 5:
 *   window_left, window_right : key j is hidden from query i when
 *            j > i + window_right (window_right >= 0) or
 *            j < i - window_left (window_left >= 0); -1 = no bound on that
 *            side.  (-1, 0) is causal, (-1, -1) no mask; values below -1
 *            return FA_ERR_INVALID_ARG.  Every row sees at least key i.
 *   softcap : 0 for none, else c > 0: each visible score s = alpha q.k
 *            becomes c tanh(s / c) before the mask and the softmax
 *            (tanh.approx.f32: max abs error 8e-6, measured);
 *            negative or non-finite returns FA_ERR_INVALID_ARG.
 *   sinks  : device, float [H] (one logit sigma per query head, finite or
 *            -inf), 4-byte aligned, or NULL for none.  sigma joins every
 *            row's softmax denominator and carries no value:
 *            O_i = sum_j e^(S_ij) v_j / (sum_j e^(S_ij) + e^sigma),
 *            LSE_i = log(sum_j e^(S_ij) + e^sigma).
 *   d in {64, 128} (others FA_ERR_UNSUPPORTED).  Other arguments, results
 *   and errors as fa_fwd_gqa.  Key tiles entirely outside a Q tile's
 *   window are neither loaded nor computed.
 */
fa_status fa_fwd_ext(const void *q, const void *k, const void *v, void *o,
                     float *lse, int B, int H, int H_kv, int N, int d,
                     float alpha, int window_left, int window_right,
                     float softcap, const float *sinks, fa_dtype dtype,
                     void *stream);

/*
 * fa_fwd_splitkv -- fa_fwd with each work unit's key range cut into
 * n_splits parts ("FlashAttention-3 on Hopper", ch. 10: split-KV and its
 * combine kernel), for problems whose B * H * ceil(N/256) units do not
 * fill the GPU.  Every split writes its partial O (FP32, normalised over
 * its own keys) and LSE into `workspace`; a combine kernel then writes
 *   LSE = log sum_s exp(LSE_s),  O = sum_s exp(LSE_s - LSE) O_s
 * to o (dtype) and lse (if not NULL).
 *   workspace : device, fa_splitkv_workspace_floats(B, H, N, d, n_splits)
 *            floats, 16-byte aligned, caller-owned; nothing in it needs to
 *            start at zero.
 *   n_splits in [1, 16] (FA_ERR_INVALID_ARG otherwise); d in {64, 128}
 *   (others FA_ERR_UNSUPPORTED).  Other arguments and errors as fa_fwd.
 */
fa_status fa_fwd_splitkv(const void *q, const void *k, const void *v, void *o,
                         float *lse, int B, int H, int N, int d, float alpha,
                         int causal, fa_dtype dtype, int n_splits,
                         float *workspace, void *stream);

/* fa_splitkv_workspace_floats -- workspace size of fa_fwd_splitkv, in
 * floats: n_splits * (B*N*H*d + B*H*N); -1 for a non-positive argument. */
long long fa_splitkv_workspace_floats(int B, int H, int N, int d, int n_splits);

/* fa_splitkv_auto -- a split count for the current device: with
 * u = B * H * ceil(ceil(N/128)/2) work units, 1 when u already occupies 80 %
 * of the SMs, else the fewest splits S with S u >= 80 % of the SMs, keeping
 * S u within one wave, at least 4 key tiles per split and S <= 16. */
int fa_splitkv_auto(int B, int H, int N, int d);

/*
 * fa_quantize_fp8 -- FP8 pre-pass: block quantization with optional
 * incoherent processing ("FlashAttention-3 on Hopper", sec. 6.3 and 6.4).
 *   x      : device, bf16 [B][N][H][d], 16-byte aligned.
 *   x8     : device, uint8 e4m3 codes [B][N][H][d], 16-byte aligned (written).
 *   scales : device, float [B][H][ceil(N/128)] (written): one scale per
 *            128-row tile of a head, scale = amax / 448 over the (rotated)
 *            tile, 1 for an all-zero tile.
 *   hadamard_signs : device, float[d] of +-1, or NULL for no rotation.  With
 *            it, each row is replaced by y = x (1/sqrt d) H D before
 *            quantization (H: d x d Sylvester Hadamard matrix, D = diag of
 *            the signs).  Use the same signs for Q and K, none for V: the
 *            product (QM)(KM)^T equals Q K^T because M is orthogonal.
 *   d in {64, 128, 256}.
 * codes = e4m3(y * (1/scale)) with the FP32 reciprocal formed once per tile
 * (within one rounding of y / scale), round to nearest even, saturating at
 * +-448.
 */
fa_status fa_quantize_fp8(const void *x, uint8_t *x8, float *scales,
                          const float *hadamard_signs, int B, int H, int N, int d,
                          void *stream);

/*
 * fa_quantize_fp8_granular -- fa_quantize_fp8 with a coarser scale: the
 * control arm of the FA3 FP8 numerical-error ablation, which compares block
 * quantization against one scale per tensor (the FlashAttention-3 review on
 * diycv.top, "numerical error"; "FlashAttention-3 on Hopper", sec. 6.3).
 *   granularity : FA_SCALE_TILE (exactly fa_quantize_fp8), FA_SCALE_HEAD
 *            (scale = amax / 448 over each (b, h)), or FA_SCALE_TENSOR (over
 *            the whole tensor); other values give FA_ERR_INVALID_ARG.
 *   scales : written in the per-tile layout [B][H][ceil(N/128)] whatever
 *            the granularity (every tile of a group holds the group's
 *            scale), so fa_fwd_fp8 consumes them unchanged.
 * Coarser granularities run three kernels on `stream` (the per-tile pass,
 * a maximum over each group of its tile scales, and the pass again with
 * those scales).  Other arguments, results and errors as fa_quantize_fp8.
 */
fa_status fa_quantize_fp8_granular(const void *x, uint8_t *x8, float *scales,
                                   const float *hadamard_signs, int B, int H, int N,
                                   int d, int granularity, void *stream);

/*
 * fa_fwd_fp8 -- attention forward on e4m3 Q/K/V with per-tile scales
 * (as written by fa_quantize_fp8), bf16 output ("FlashAttention-3 on
 * Hopper", sec. 6.3: descales folded into the softmax scale per tile
 * pair; "03 FA3", sec. 4: the exponent of the FP8 probabilities shifted
 * into the e4m3 range: P' = 2^(s - r + c) with the reference r moved when
 * a tile's row max exceeds it by more than tau; c = 4, tau = 4.8, so
 * P' <= 2^8.8 < 448: the pages' c = 8 would leave tau = 0.8 and a rescale
 * on about half of the steps of outlier inputs).
 *   q8, k8, v8 : device, uint8 e4m3 [B][N][H][d], 16-byte aligned.
 *   q_scale, k_scale, v_scale : device, float [B][H][ceil(N/128)].
 *   o   : device, bf16 [B][N][H][d] (written).  lse : as for fa_fwd.
 *   d in {128, 256} (others return FA_ERR_UNSUPPORTED; d = 256 runs one
 *   128-row Q tile per work unit).  alpha, causal as fa_fwd.
 * P is rounded to e4m3 before the P V product with the V tile scale
 * folded in (P'_j = P_j v_j / max_j v_j); accumulation is FP32, and O is
 * normalised by the FP32 row sum of the unrounded P.  Per-tile V scales
 * are accepted, but the fold then rounds the dominant terms of P' (ratios
 * below 1 are not powers of two), which the row sum does not see; one V
 * scale per head (fa_quantize_fp8_granular with FA_SCALE_HEAD, repeated
 * over the tiles) makes every ratio 1 and is the measured better choice.
 */
fa_status fa_fwd_fp8(const uint8_t *q8, const uint8_t *k8, const uint8_t *v8,
                     const float *q_scale, const float *k_scale, const float *v_scale,
                     void *o, float *lse, int B, int H, int N, int d, float alpha,
                     int causal, void *stream);

/*
 * fa_fwd_fp8_gqa -- fa_fwd_fp8 with grouped key/value heads (as fa_fwd_gqa):
 * q8 and q_scale have H heads, k8, v8, k_scale and v_scale have H_kv heads
 * ([B][N][H_kv][d] codes, [B][H_kv][ceil(N/128)] scales), H_kv >= 1 divides
 * H, and query head h attends with key/value head h / (H / H_kv).  H_kv = H
 * is fa_fwd_fp8.  H % H_kv != 0 or H_kv < 1 returns FA_ERR_INVALID_ARG;
 * other arguments, results and errors as fa_fwd_fp8.
 */
fa_status fa_fwd_fp8_gqa(const uint8_t *q8, const uint8_t *k8, const uint8_t *v8,
                         const float *q_scale, const float *k_scale, const float *v_scale,
                         void *o, float *lse, int B, int H, int H_kv, int N, int d,
                         float alpha, int causal, void *stream);

/*
 * fa_bwd -- gradients of the attention of fa_fwd ("FlashAttention-3 on
 * Hopper", ch. 7): with S = alpha Q K^T (masked as in fa_fwd),
 * P = softmax(S) and O = P V, for the upstream gradient dO:
 *   dV = P^T dO,  dP = dO V^T,  D_i = rowsum(dO_i o O_i),
 *   dS = P o (dP - D),  dQ = alpha dS K,  dK = alpha dS^T Q.
 * P is recomputed from Q, K and the forward's LSE (sec. 7.1.3).
 *   q, k, v, o, dout : device, dtype [B][N][H][d], 16-byte aligned; o and
 *            lse are the outputs of fa_fwd on the same q, k, v, alpha and
 *            causal.
 *   lse    : device, float [B][H][N] (natural log, as fa_fwd writes it).
 *   workspace : device, float [2][B][H][ceil(N/128)*128], 16-byte aligned,
 *            caller-owned; receives D = rowsum(dO o O) and LSE*log2(e) per
 *            row (rows padded to whole 128-row tiles).
 *   dq, dk, dv : device, dtype [B][N][H][d], 16-byte aligned (written).
 *   d in {64, 128} (others return FA_ERR_UNSUPPORTED); alpha, causal,
 *   dtype and stream as fa_fwd.
 * Three kernels run in order on `stream`: the D preprocess, a key-parallel
 * kernel for dK and dV and a query-parallel kernel for dQ that recomputes S
 * and dP (sec. 7.2, first option), so no atomics are used and the results
 * are identical from run to run.  P and dS are rounded to `dtype` for the
 * GEMMs that consume them; accumulation is FP32; outputs are rounded to
 * `dtype`.  Nothing is allocated.  Errors as fa_fwd.  With causal = 1 both
 * main kernels schedule their units as fa_fwd's causal launches do (one CTA
 * per unit, head groups kept together for L2 reuse).
 */
fa_status fa_bwd(const void *q, const void *k, const void *v, const void *o,
                 const void *dout, const float *lse, float *workspace, void *dq,
                 void *dk, void *dv, int B, int H, int N, int d, float alpha,
                 int causal, fa_dtype dtype, void *stream);

/*
 * fa_bwd_ext -- fa_bwd for the forward of fa_fwd_ext with a local window,
 * an optional softcap and optional sinks ("FlashAttention-3 on Hopper",
 * sec. 7.8: a right window bounds the first query tile a key tile visits, a
 * left window the last, and the softcap enters as a score modifier; sec.
 * 4.6: sinks; "03 FA3", sec. 5: softcap).
 *   window_left, window_right : as for fa_fwd_ext (-1 = no bound; values
 *            below -1 return FA_ERR_INVALID_ARG).
 *   softcap : the forward's c (0: none).  With c > 0 both kernels recompute
 *            t = tanh(alpha s / c) (tanh.approx.f32), form P from t and the
 *            LSE, and scale dS by dS/du = 1 - t^2.  Negative, non-finite or
 *            alpha / c beyond FP32 returns FA_ERR_INVALID_ARG.
 *   lse    : from fa_fwd_ext with the same window and sinks.  The gradients
 *            of q, k and v need nothing else from the sinks: P is formed
 *            from that LSE, which already holds the sink term.
 *   sinks  : device float [H] (the forward's), or NULL.  dsinks : device
 *            float [H] or NULL; with both, dsinks[h] receives the gradient
 *            of sigma_h, -sum over batches and rows of e^(sigma_h - LSE) D
 *            (D = rowsum(dO o O)), reduced in a fixed order.  dsinks
 *            without sinks returns FA_ERR_INVALID_ARG.
 *   H_kv   : K/V heads (grouped-query attention, as for fa_fwd_ext): k, v,
 *            dk, dv are [B][N][H_kv][d], query head h uses K/V head
 *            h / (H / H_kv), and dK, dV of a K/V head sum the contributions
 *            of all its query heads (accumulated in FP32 in one kernel, no
 *            atomics).  H % H_kv != 0 or H_kv < 1 returns FA_ERR_INVALID_ARG.
 * Other arguments, results and errors as fa_bwd (d in {64, 128}).
 */
fa_status fa_bwd_ext(const void *q, const void *k, const void *v, const void *o,
                     const void *dout, const float *lse, float *workspace,
                     void *dq, void *dk, void *dv, int B, int H, int H_kv, int N, int d,
                     float alpha, int window_left, int window_right,
                     float softcap, const float *sinks, float *dsinks,
                     fa_dtype dtype, void *stream);

/*
 * fa_bwd_noalloc -- fa_bwd without a caller-provided workspace (the pages
 * have no counterpart: this is an interface convenience of this library).
 * For callers that must not allocate device memory at the point of the
 * call, e.g. a program whose device memory is reserved up front or a
 * runtime that forbids allocation inside a step.  The workspace is a
 * 16 MiB array in the library's device image (one per device that loads
 * the library, held until the process exits); nothing is allocated, and
 * nothing in it needs to start at zero.  Limit: 2 * B * H * ceil(N/128) *
 * 128 <= 4194304 floats, else FA_ERR_TOO_LARGE before anything runs; the
 * arguments fa_bwd rejects are checked first and give fa_bwd's codes.
 * Calls that overlap in time (on other streams or host threads) share the
 * array and race; serialise them.  The array's device address is looked up
 * on the first call on each device (with that device current) and cached,
 * so make that first call before any stream capture, and do not call this
 * after a cudaDeviceReset in the same process (the cached address would be
 * stale).  Other arguments, results and errors as fa_bwd.
 */
fa_status fa_bwd_noalloc(const void *q, const void *k, const void *v,
                         const void *o, const void *dout, const float *lse,
                         void *dq, void *dk, void *dv, int B, int H, int N,
                         int d, float alpha, int causal, fa_dtype dtype,
                         void *stream);

/*
 * Paged key/value cache: the entry points that answer from a cache of past
 * keys and values instead of dense tensors with Nq = Nk.
 *
 * The cache.  k_pages and v_pages are pools of pages, element (page, slot,
 * K/V head, c) at page * page_stride + (slot * H_kv + head) * d + c in
 * `dtype`: page_size slots of H_kv x d, page_stride >= page_size * H_kv * d
 * elements from page to page (one pool with K and V side by side in a page
 * has twice that), a multiple of 8.  page_size is a power of two >= 8.
 * Token p of sequence b is slot p % page_size of page
 * block_table[b * table_width + p / page_size]; kv_len[b] tokens are cached.
 * Sequences may share pages that none of them writes.
 *
 * The new tokens of a call are packed: rows cu_q[b] .. cu_q[b + 1] (cu_q has
 * B + 1 entries, ascending) of tensors with total_q rows are sequence b's
 * last cached tokens, kv_len[b] counts them, and row cu_q[b] + i has position
 * kv_len[b] - (cu_q[b + 1] - cu_q[b]) + i.  A sequence may have none.  Rows
 * at and behind cu_q[B] may hold anything and are not written (what a call
 * reads ahead there it drops).  With total_q = 0 the packed tensors may be
 * NULL.
 *
 * block_table, kv_len and cu_q are device int32, so lengths may change from
 * one replay of a captured graph to the next.  What is out of range there (a
 * page id a call needs outside [0, n_pages), kv_len outside [0, table_width *
 * page_size], cu_q outside [0, total_q] or falling) is cut off: that access is
 * skipped, the row's result is undefined, and the next fa_check_status
 * returns FA_ERR_BAD_INDEX.  Entries of block_table that no visible token
 * needs are not looked at, and slots at and behind kv_len may hold anything
 * (NaN included).
 *
 * d in {64, 128}, other head dims and page sizes give FA_ERR_UNSUPPORTED;
 * B, H_kv <= 65535.
 */

/*
 * fa_paged_append -- writes the new tokens' keys and values into their pages.
 *   k, v : device, total_q rows of [H_kv][d], kv_stride elements from row to
 *          row (>= H_kv * d, a multiple of 8: a slice of a fused projection's
 *          rows is fine), 16-byte aligned.
 * Tokens without a slot are dropped and nothing is written in their place: a
 * negative position (more new tokens than kv_len counts), or one at or behind
 * table_width * page_size (a full cache; FA_ERR_BAD_INDEX).  Any 16-bit
 * element type.
 */
fa_status fa_paged_append(const void *k, const void *v, void *k_pages, void *v_pages,
                          const int32_t *block_table, const int32_t *kv_len,
                          const int32_t *cu_q, int B, int H_kv, int d, int total_q,
                          int page_size, int n_pages, int table_width, long long kv_stride,
                          long long page_stride, void *stream);

/*
 * fa_fwd_paged -- exact attention of the new tokens over the cache (which
 * already holds them), with grouped K/V heads as in fa_fwd_gqa:
 *     S = alpha * q K^T over the visible keys, O = softmax(S) V,
 *     LSE = log sum exp(S).
 * Key j is visible to the row at position p when j < kv_len and
 *     j <= p + window_right            (window_right >= 0; -1: no bound), and
 *     j >= p - window_left  or  j < first   (window_left >= 0; -1: no bound):
 * (-1, 0) is causal, (-1, -1) no mask, and with a left bound the first
 * `first` tokens of the sequence stay visible beside the sliding window.  A
 * row that sees no key gives O = 0, LSE = -inf.  A NaN in q or in a key that a
 * row sees makes its O and LSE NaN.  An infinity or NaN in a value reaches, as
 * 0 times it, every row of the K/V head whose tile of rows sees that token.
 *   q    : device, total_q rows of [H][d], q_stride elements from row to row
 *          (>= H * d, a multiple of 8), 16-byte aligned.
 *   o    : device, [total_q][H][d], 16-byte aligned (written).
 *   lse  : device, float [H][total_q], or NULL to skip.
 *   workspace : device, fa_paged_workspace_bytes(d) bytes, 32-byte aligned,
 *          caller-owned; nothing in it needs to start at zero.  Calls that
 *          may overlap in time need one each.
 *   max_q : the most new tokens of one sequence, >= 1; it only chooses tile
 *          shapes (a larger sequence is still computed in full).
 *   alpha : the score scale, positive.
 *   H / H_kv <= 128, else FA_ERR_UNSUPPORTED.
 * Accumulation is FP32, P is rounded to `dtype` before the P V product.
 * The key ranges of all rows together are cut into equal shares for the SMs
 * and the shares' results joined in a fixed order: the same call repeats its
 * bits, but where a sequence is cut depends on the whole batch's lengths.
 */
fa_status fa_fwd_paged(const void *q, const void *k_pages, const void *v_pages,
                       const int32_t *block_table, const int32_t *kv_len,
                       const int32_t *cu_q, void *o, float *lse, void *workspace, int B,
                       int H, int H_kv, int total_q, int max_q, int d, int page_size,
                       int n_pages, int table_width, long long q_stride,
                       long long page_stride, float alpha, int window_left,
                       int window_right, int first, fa_dtype dtype, void *stream);

/* fa_paged_workspace_bytes -- workspace of fa_fwd_paged on the current
 * device, whatever the problem's other sizes; -1 for a head dim without a
 * kernel or without an sm_103 device. */
long long fa_paged_workspace_bytes(int d);

/*
 * fa_paged_scores -- the attention weight that every cached token gets from
 * the new ones, summed over the rows and over the query heads of each K/V
 * head, on top of what it had:
 *     scores[b][h][j] = (j older than the new tokens ? scores_in[b][h][j] : 0)
 *                       + sum over rows i that see j, heads of group h, of
 *                         exp(alpha q_i . k_j - LSE_i)
 * for j < kv_len[b]; the rest of scores is left as it was.
 *   lse    : device, float [H][total_q], from fa_fwd_paged with the same
 *            arguments (rows with LSE = -inf add nothing, a NaN makes the
 *            weights of the tokens that its row sees NaN, and no others).
 *   scores_in, scores : device, float [B][H_kv][score_width]; scores_in may
 *            be scores itself, or NULL for zeros.  score_width >= every
 *            kv_len (of a longer cache the first score_width tokens get their
 *            weights: FA_ERR_BAD_INDEX).
 * A sequence whose kv_len or offsets are out of range adds nothing, so that
 * weights collected in place survive it.
 * Summed in FP32 in a fixed order, without atomics.  Other arguments as
 * fa_fwd_paged.
 */
fa_status fa_paged_scores(const void *q, const float *lse, const void *k_pages,
                          const int32_t *block_table, const int32_t *kv_len,
                          const int32_t *cu_q, const float *scores_in, float *scores, int B,
                          int H, int H_kv, int total_q, int max_q, int d, int page_size,
                          int n_pages, int table_width, int score_width, long long q_stride,
                          long long page_stride, float alpha, int window_left,
                          int window_right, int first, fa_dtype dtype, void *stream);

/*
 * fa_paged_evict -- cuts every sequence of the cache to its `keep` most
 * important tokens, for each K/V head by itself: the first `first`, the last
 * `recent`, and of the others those with the largest score (equal scores: the
 * lower position; NaN ranks above +inf).  The kept tokens go, in their order,
 * to positions 0, 1, ... of the pages of dst_table (their slots then hold
 * different tokens for different heads); a sequence of at most `keep` tokens
 * keeps all.  The old pages are left as they were: other sequences may share
 * them, and the caller frees them.
 *   scores : device, float [B][H_kv][score_width] (fa_paged_scores).
 *   dst_table : device, int32 [B][dst_width], pages of the same pools that no
 *            sequence of the call reads and no two entries name twice;
 *            dst_width * page_size >= keep.
 *   kept   : device, int32 [B][H_kv][keep] (written): the kept tokens' old
 *            positions, ascending; entries at and behind new_len[b] are left.
 *   scores_out : device, float [B][H_kv][keep], their scores (as kept), or
 *            NULL.  No part of scores, else FA_ERR_INVALID_ARG.
 *   new_len : device, int32 [B] (written): min(kv_len[b], keep).  It may be
 *            kv_len itself, but overlap it in no other way
 *            (FA_ERR_INVALID_ARG).
 *   keep >= 1, first, recent >= 0, first + recent <= keep.
 * Any 16-bit element type.  kv_len beyond score_width is cut off.
 */
fa_status fa_paged_evict(void *k_pages, void *v_pages, const float *scores,
                         const int32_t *block_table, const int32_t *kv_len,
                         const int32_t *dst_table, int32_t *kept, float *scores_out,
                         int32_t *new_len, int B, int H_kv, int d, int page_size,
                         int n_pages, int table_width, int dst_width, int score_width,
                         long long page_stride, int keep, int first, int recent,
                         void *stream);

/*
 * fa_check_status -- synchronizes `stream`, then reports and clears the
 * device status word of the current device.  Returns FA_ERR_TIMEOUT if a
 * kernel launched since the last check gave up on a bounded wait (its
 * outputs are then undefined), FA_ERR_BAD_INDEX if one met an index out of
 * range in device memory, FA_ERR_CUDA if the synchronization failed, FA_OK
 * otherwise.  (The first of several events is the one reported.)
 */
fa_status fa_check_status(void *stream);

/*
 * fa_status_detail -- the status word captured by the last fa_check_status
 * that returned FA_ERR_TIMEOUT or FA_ERR_BAD_INDEX: out[0] code, out[1] role
 * that gave up (1/2 softmax group L/H, 3 producer, 4 MMA issuer, 6 FP8
 * pre-pass, 7 self-test, 8 paged cache),
 * out[2] wait site (bad index: 1 kv_len or cu_q, 2 page id, 3 kv_len beyond
 * the scores),
 * out[3] block index.  Zeros if nothing was ever reported.
 */
void fa_status_detail(uint32_t out[4]);

/*
 * fa_selftest_wait_timeout -- exercises the failure path without a fault:
 * one CTA whose two warps wait (with the pipeline kernels' bounded wait) on
 * valid mbarriers that nobody arrives on.  The first wait gives up after
 * its time limit (2 s), records role 7 and its site (1 or 2) in the status
 * word and raises the CTA's abort flag; the other then returns promptly.
 *   result : device, uint32_t[2], 4-byte aligned (written): result[w] = 1
 *            when warp w's wait returned false.
 * The next fa_check_status then returns FA_ERR_TIMEOUT and
 * fa_status_detail gives {1, 7, site, 0}; the CUDA context stays usable.
 * Returns FA_ERR_INVALID_ARG for a null result, FA_ERR_MISALIGNED,
 * FA_ERR_UNSUPPORTED / FA_ERR_CUDA as fa_fwd.
 */
fa_status fa_selftest_wait_timeout(uint32_t *result, void *stream);

/* fa_status_string -- a static, human-readable name for a status code. */
const char *fa_status_string(fa_status s);

/* fa_version -- library version as major*10000 + minor*100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
