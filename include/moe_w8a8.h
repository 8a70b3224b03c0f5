/*
 * moe_w8a8.h -- C ABI of the W8A8-quantised Mixture-of-Experts expert layer
 * for AMD Instinct MI355X (gfx950).
 *
 * The layer (one call to moe_w8a8_forward) computes, for T tokens x[T][H]:
 *   1. route    top-k experts per token from router logits (given, or
 *               projected from x by the bf16 router matrix in the same call),
 *               ties to the lower expert index, softmax weights renormalised
 *               over the chosen k
 *               ("超大规模模型推理的Day0适配实践" §四: the fused MoE operator's
 *               top-k must equal the reference, tie-break included);
 *   2. permute  group the T*k (token, slot) assignments expert by expert,
 *               (token, slot) order inside a group, an optional expert
 *               capacity dropping the overflow (same page, §二.2);
 *   3. quantise each token to INT8 per token after dividing by the
 *               SmoothQuant scales ("MiniMax-M3 W8A8 inference on K100AI",
 *               mhpq.cn/news/1068415, §3.2 and §6.4), at the token's absolute
 *               maximum or, when a clip is set, at the smaller of that and
 *               the clip thresholds (values beyond saturate at +-127: K100AI
 *               page §6.4; "一晚上完成MoE模型推理优化…" §3.2);
 *   4. GEMM1    per expert, INT8 x INT8 -> INT32 gate and up projections,
 *               dequantised per token and per output channel, h = silu(g)*u,
 *               requantised to INT8 per (token, expert) row (K100AI page
 *               §1.2 and §4.3: INT8 GEMM with integer accumulation; stay in
 *               the INT8 domain between consecutive matmuls);
 *   5. GEMM2    per expert, INT8 down projection, dequantised per row and
 *               per output channel to fp32 (for large batches held until the
 *               combine as int16 codes with one fp32 scale per 16 outputs,
 *               error at most ~2^-16 of the group's largest value);
 *   6. combine  out[t] = sum over kept slots of w[t][j] * y[row], summed in
 *               fp32 and rounded to bfloat16 (Day0 page §四: un-sort and
 *               weighted sum).
 * moe_w8a8_calibrate prepares the quantised weights (K100AI page §3.2:
 * SmoothQuant with migration strength alpha, per-output-channel weights).
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers (hipMalloc'd or equivalent) owned
 *    by the caller; nothing is allocated or freed inside the library and no
 *    library state survives a call. Layouts are row-major unless stated.
 *  - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *    Work is enqueued asynchronously; the library never synchronises. Calls on
 *    different streams with disjoint buffers may run concurrently.
 *  - Arguments are validated on the host before anything is enqueued; an
 *    invalid call enqueues nothing and returns a negative code. Faults inside
 *    kernels surface at the caller's next synchronisation.
 *  - bfloat16 values are passed as uint16_t bit patterns.
 */
#ifndef MOE_W8A8_H
#define MOE_W8A8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define MOE_W8A8_OK 0
#define MOE_W8A8_ERR_INVALID (-1)     /* NULL required pointer, bad size, k > E, ... */
#define MOE_W8A8_ERR_UNSUPPORTED (-2) /* shape outside the supported set (below)     */
#define MOE_W8A8_ERR_WORKSPACE (-3)   /* workspace NULL or smaller than required     */
#define MOE_W8A8_ERR_HIP (-4)         /* a HIP launch or copy reported an error      */
#define MOE_W8A8_ERR_SCRATCH (-5)     /* batch too large for the static scratch      */

/* Alignment of the device pointers every entry point takes (a violation is
 * MOE_W8A8_ERR_INVALID, before anything is enqueued): 16 bytes for arrays the
 * kernels move 16 bytes at a time (the tokens x, the packed weight codes
 * w_gate_up and w_down, inv_smooth when the forward reads it, the router
 * matrix, pack's src and dst, the debug accumulators acc1), 8 bytes for the
 * forward's output, the natural alignment of the element type for every other
 * array, and 256 bytes for a workspace (its regions are laid out in 256-byte
 * steps). hipMalloc and torch allocations satisfy all of them. */

/* Layer dimensions. Supported set: hidden H a multiple of 256 in [256, 65536];
 * ffn F a multiple of 128 in [128, 65536]; 1 <= num_experts E <= 1024;
 * 1 <= top_k k <= min(E, 32). */
typedef struct {
  int32_t hidden;      /* H */
  int32_t ffn;         /* F, the expert FFN width (SwiGLU gate/up/down) */
  int32_t num_experts; /* E, experts held on this device */
  int32_t top_k;       /* k, assignments per token */
} moe_w8a8_dims;

/* Code format of the expert path ("超大规模模型推理的Day0适配实践" §二.1: expert
 * layers in INT8 or FP8; §四: the activations take the weights' format).
 *   INT8: symmetric codes in [-127, 127], scale = range/127, integer
 *         accumulation.
 *   FP8:  OCP e4m3 codes (bias 7, 3 mantissa bits, subnormals, largest
 *         finite 448, NaN 0x7f/0xff), scale = range/448; a value is coded as
 *         the nearest e4m3 (ties to even, sign of zero kept) of
 *         clamp(fl32(v * fl32(448/range)), -448, 448); fp32 accumulation of
 *         the exact code products. */
#define MOE_W8A8_FORMAT_INT8 0
#define MOE_W8A8_FORMAT_FP8 1

/* Quantised layer weights (device memory, written by moe_w8a8_calibrate).
 *
 * Fragment-tiled INT8 layout. A weight matrix W[N][K] (N output channels,
 * K input channels; N % 16 == 0, K % 64 == 0) is stored as 1024-byte tiles of
 * 16 output channels x 64 input channels, tile (n/16, k/64) at byte offset
 *     ((n/16) * (K/64) + k/64) * 1024,
 * and inside a tile the element (n, k) at byte
 *     (((k % 64) / 16) * 16 + n % 16) * 16 + k % 16.
 * One tile is exactly one wavefront's 16-byte-per-lane load in the lane order
 * of the gfx950 INT8 matrix instructions, so weight panels stream from HBM as
 * contiguous 1 KB blocks.
 *   w_gate_up : E matrices of [2F][H], consecutive; rows 0..F-1 are the gate
 *               projection, rows F..2F-1 the up projection (smoothed).
 *   w_down    : E matrices of [H][F], consecutive (not smoothed).
 *   s_gate_up : fp32 [E][2F]  dequantisation scale per output channel.
 *   s_down    : fp32 [E][H]   dequantisation scale per output channel.
 *   smooth    : fp32 [H]      SmoothQuant scale s_j.
 *   inv_smooth: fp32 [H]      1/s_j rounded to fp32 (what forward multiplies by).
 *   w_router  : bf16 [E][H]   router projection, row e for expert e, or NULL.
 *               Not quantised ("MiniMax-M3 W8A8 inference on K100AI" §6.1:
 *               the layers at the routing stay in 16-bit floating point) and
 *               not written by moe_w8a8_calibrate.
 *   act_clip  : fp32 [1]      static activation clipping threshold c written by
 *               moe_w8a8_calibrate_clip, or NULL (no static clip). A value
 *               <= 0 also means no clip.
 *   act_sat_percentile  (a value, not a buffer) dynamic saturation of the
 *               activations: 0 = off, else p in (0, 100]: each token is
 *               quantised at most at the nearest-rank p-th percentile of its
 *               own |x_j / s_j| (the m-th largest, m = H - ceil(p/100*H) + 1,
 *               m <= 16 supported).
 *   format    : MOE_W8A8_FORMAT_INT8 or _FP8, set by the caller before
 *               moe_w8a8_calibrate (which codes the weights in it); forward
 *               codes the activations and runs the GEMMs in the same format.
 * Code of W'[n][k] is q with W' ~= q * scale[n] (INT8: codes lie in
 * [-127, 127]; FP8: W' ~= e4m3 value of q * scale[n]). */
typedef struct {
  int8_t *w_gate_up;
  int8_t *w_down;
  float *s_gate_up;
  float *s_down;
  float *smooth;
  float *inv_smooth;
  uint16_t *w_router;
  float *act_clip;
  float act_sat_percentile;
  int32_t format;
} moe_w8a8_weights;

/* Optional per-stage outputs of moe_w8a8_forward for checking; every pointer
 * may be NULL. A = T*k. Rows of the permuted tensors are positions in the
 * expert-grouped order; entries past the number of kept rows (the last
 * expert_offsets value) are unspecified.
 *   topk_ids int32 [T][k], topk_w fp32 [T][k]  (routing result or the given ids)
 *   expert_counts int32 [E] kept rows per expert; expert_offsets int32 [E+1]
 *   sorted_assign int32 [A] assignment t*k+j of each permuted row
 *   row_of int32 [A] permuted row of assignment t*k+j, -1 if dropped
 *   qx int8 [T][H], sx fp32 [T]   per-token codes (e4m3 bytes in FP8 format)
 *                                 and scales
 *   acc1 int32 [A][2F]            GEMM1 accumulators (gate then up; the
 *                                 bits of the fp32 sums in FP8 format)
 *   h fp32 [A][F]                 SwiGLU output before requantisation
 *   qh int8 [A][F], sh fp32 [A]   requantised hidden rows and their scales
 *   y fp32 [A][H]                 dequantised down-projection rows, as the
 *                                 combine reads them */
typedef struct {
  int32_t *topk_ids;
  float *topk_w;
  int32_t *expert_counts;
  int32_t *expert_offsets;
  int32_t *sorted_assign;
  int32_t *row_of;
  int8_t *qx;
  float *sx;
  int32_t *acc1;
  float *h;
  int8_t *qh;
  float *sh;
  float *y;
  /* Kernel family of the two grouped GEMMs: 0 = chosen from the shape
   * (streaming kernels while experts average at most 32 rows, tiled kernels
   * beyond), 1 = streaming, 2 = tiled. Any other value: MOE_W8A8_ERR_INVALID.
   * Every choice computes the same result. */
  int32_t gemm_path;
  /* NULL, or an array of 18 hipEvent_t (as void*) to time the layer's
   * kernels on its own stream: entries 2s and 2s+1 are stamped with the
   * start and the end of the execution of the launch that performs stage s
   * (s = 0 route, 1 scan, 2 scatter, 3 activation quant, 4 GEMM1, 5 requant,
   * 6 GEMM2, 7 combine, 8 router projection), by that launch's own dispatch
   * (hipExtLaunchKernel), so timing inserts nothing between the kernels.
   * Stages fused into one launch are timed by the pair of the first of them:
   * for T*k <= 2048, stages 0-3 are one launch and pairs 1-3 are left
   * untouched. NULL entries are skipped. */
  void **stage_events;
  /* fp32 [T][E]: the router logits the routing used (the projection's
   * result in router-projection mode, a copy of router_logits otherwise;
   * untouched in pre-routed mode). */
  float *router_logits;
} moe_w8a8_debug;

/* Bytes of device workspace that moe_w8a8_forward needs for T tokens, and
 * that moe_w8a8_calibrate needs (T = 0 gives at least the calibrate size).
 * The caller allocates it once and hands it to every call
 * ("MiniMax-M3 W8A8 inference on K100AI" §4.3: reuse device memory from a
 * pool instead of allocating per call); the library allocates nothing.
 * A pure function of the arguments, nondecreasing in T (a workspace sized for
 * the largest batch serves every smaller one); returns 0 for invalid or
 * unsupported dimensions, T < 0, or a batch past the row limit of
 * moe_w8a8_forward. */
size_t moe_w8a8_workspace_size(const moe_w8a8_dims *dims, int64_t T);

/* Calibrate and quantise the layer weights ("MiniMax-M3 W8A8 inference on
 * K100AI" §3.2: SmoothQuant, per-channel weights; published SmoothQuant scale).
 *   alpha      migration strength in [0, 1] (the page's default is 0.6).
 *   calib_x    bf16 [n_calib][H] calibration tokens, n_calib >= 0.
 *   w_gate, w_up fp32 [E][F][H]; w_down fp32 [E][H][F] (unquantised, row-major).
 *   out        device buffers to fill (layouts above); the struct itself is
 *              host memory.
 * Computes, per input channel j: ax_j = max |calib_x[:, j]|,
 * aw_j = max over all experts and both projections of |W_gate|, |W_up| in
 * column j, s_j = ax_j^alpha / aw_j^(1-alpha) evaluated in fp64 and rounded to
 * fp32 (s_j = 1 when ax_j or aw_j is 0), inv_s_j = 1/s_j in fp32; then the
 * gate/up rows W[n][j] * s_j (fp32) and the down rows are quantised per row:
 * a = max |row|, code = rint(v * fl32(127/a)) clamped to [-127, 127],
 * scale = a/127 (an all-zero row gets scale 0 and codes 0).
 * Workspace: at least moe_w8a8_workspace_size(dims, 0) bytes.
 * Errors: MOE_W8A8_ERR_INVALID (NULL pointer, alpha outside [0,1],
 * n_calib < 0 or n_calib * H >= 2^61), MOE_W8A8_ERR_UNSUPPORTED, MOE_W8A8_ERR_WORKSPACE,
 * MOE_W8A8_ERR_HIP. */
int moe_w8a8_calibrate(const moe_w8a8_dims *dims, float alpha,
                       const uint16_t *calib_x, int64_t n_calib,
                       const float *w_gate, const float *w_up, const float *w_down,
                       const moe_w8a8_weights *out,
                       void *workspace, size_t workspace_bytes, void *stream);

/* Static activation clipping threshold ("一晚上完成MoE模型推理优化…" §3.2:
 * the calibration clips activations beyond the 99.9th percentile of their
 * range). Writes act_clip[0] = the nearest-rank percentile `percentile` of
 * |fl32(calib_x[n][j] * inv_smooth[j])| over all n_calib * H entries: the
 * value of rank ceil(percentile/100 * N) (evaluated in fp64, clamped to
 * [1, N]) in ascending order; 0 when n_calib = 0.
 *   percentile in (0, 100]; calib_x bf16 [n_calib][H]; inv_smooth fp32 [H]
 *   (from moe_w8a8_calibrate); act_clip fp32 [1]. All device memory.
 * Errors: MOE_W8A8_ERR_INVALID (also n_calib * H >= 2^61),
 * MOE_W8A8_ERR_UNSUPPORTED, MOE_W8A8_ERR_HIP. */
int moe_w8a8_calibrate_clip(const moe_w8a8_dims *dims, float percentile,
                            const uint16_t *calib_x, int64_t n_calib,
                            const float *inv_smooth, float *act_clip, void *stream);

/* Forward pass of the layer for T tokens (steps 1-6 above).
 *   x           bf16 [T][H] input tokens.
 *   Routing input, one of three modes:
 *   router_logits fp32 [T][E] given; or
 *   topk_ids    int32 [T][k] and topk_w fp32 [T][k] (pre-routed mode): the
 *               assignments and their weights (ids outside [0, E) are treated
 *               as dropped; the weights are used as given; an expert named in
 *               several slots of a token gets one row per slot, each weighted
 *               by its own slot's weight and counted against the capacity); or
 *   neither (router-projection mode): the logits are x . w_router^T from
 *               weights->w_router, as moe_w8a8_router_logits computes them,
 *               and the routing of step 1 is taken on them.
 *   Giving router_logits together with topk_ids or topk_w, only one of
 *   topk_ids and topk_w, or neither with w_router NULL is an error.
 *   capacity_factor  > 0: each expert keeps at most
 *               C = ceil(capacity_factor * T * k / E) assignments (evaluated
 *               in fp64), the first C in (token, slot) order; dropped slots
 *               contribute nothing and the remaining weights are not
 *               renormalised. <= 0: no limit.
 *   out         bf16 [T][H] layer output (written for every token; a token
 *               whose every slot was dropped gets zeros).
 *   workspace   at least moe_w8a8_workspace_size(dims, T) bytes; contents on
 *               entry are ignored.
 *   debug       NULL, or a host struct of optional device outputs (above).
 * T == 0 is a successful no-op whatever the other pointers are (empty
 * tensors may carry NULL addresses). Errors: MOE_W8A8_ERR_INVALID (NULL required
 * pointer, T < 0, T*k >= 2^31 or T*k + 15*min(T*k, E) >= 2^31 (the permuted
 * rows with every expert group padded to 16), routing inputs as above, act_sat_percentile
 * outside {0} and (0, 100]), MOE_W8A8_ERR_UNSUPPORTED (also a saturation
 * rank m > 16), MOE_W8A8_ERR_WORKSPACE, MOE_W8A8_ERR_HIP. */
int moe_w8a8_forward(const moe_w8a8_dims *dims, const moe_w8a8_weights *weights,
                     const uint16_t *x, int64_t T,
                     const float *router_logits,
                     const int32_t *topk_ids, const float *topk_w,
                     float capacity_factor,
                     uint16_t *out,
                     void *workspace, size_t workspace_bytes,
                     const moe_w8a8_debug *debug, void *stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * forward as moe_w8a8_forward, same arguments and results, but its workspace
 * is a static device array of MOE_W8A8_SCRATCH_BYTES inside the library (one
 * per GPU, held from the first call on that GPU until the process ends)
 * instead of a caller buffer. Nothing is allocated or freed by the call.
 * Limit: moe_w8a8_workspace_size(dims, T) <= MOE_W8A8_SCRATCH_BYTES (64 MiB:
 * e.g. up to ~220 tokens of a hidden-4096, 64-expert, top-8, FFN-1536 layer);
 * a larger batch returns MOE_W8A8_ERR_SCRATCH with nothing enqueued.
 * Every call on one GPU uses that GPU's one array, so calls that overlap on a
 * GPU (concurrent streams, or host threads) race and must be serialised by
 * the caller; consecutive calls on one stream are safe (each call's kernels
 * ignore what the array held before). Errors: as moe_w8a8_forward, with
 * MOE_W8A8_ERR_SCRATCH in place of MOE_W8A8_ERR_WORKSPACE. */
#define MOE_W8A8_SCRATCH_BYTES ((size_t)64 << 20)
int moe_w8a8_forward_noalloc(const moe_w8a8_dims *dims, const moe_w8a8_weights *weights,
                             const uint16_t *x, int64_t T,
                             const float *router_logits,
                             const int32_t *topk_ids, const float *topk_w,
                             float capacity_factor,
                             uint16_t *out,
                             const moe_w8a8_debug *debug, void *stream);

/* Router projection ("超大规模模型推理的Day0适配实践" §四: the gate belongs to
 * the fused MoE operator and the top-k it feeds must be exact; "MiniMax-M3
 * W8A8 inference on K100AI" §6.1: the routing layers stay in 16-bit float):
 *   logits[t][e] = sum_j x[t][j] * w_router[e][j]
 * with x bf16 [T][H], w_router bf16 [E][H] (device), accumulated in fp32 on
 * the bf16 matrix instructions (each product exact), written to logits fp32
 * [T][E] (device). The order of the sum depends on H only, never on T: H
 * is cut into parts of 512 channels, each part into 4 runs of 128 summed
 * ((r0 + r1) + r2) + r3, and the parts are added in order; within a run the
 * matrix instructions accumulate 16 channels at a time. A token's logits are
 * therefore the same whatever batch it comes in.
 * Workspace: at least moe_w8a8_workspace_size(dims, T) bytes (the per-part
 * sums; none is needed when H <= 512).
 * T == 0 is a successful no-op. Errors: MOE_W8A8_ERR_INVALID (NULL pointer,
 * T < 0), MOE_W8A8_ERR_UNSUPPORTED, MOE_W8A8_ERR_WORKSPACE, MOE_W8A8_ERR_HIP. */
int moe_w8a8_router_logits(const moe_w8a8_dims *dims, const uint16_t *x, int64_t T,
                           const uint16_t *w_router, float *logits,
                           void *workspace, size_t workspace_bytes, void *stream);

/* Pack row-major codes into the fragment-tiled layout of moe_w8a8_weights
 * ("MiniMax-M3 W8A8 inference on K100AI" §3.2-§3.3: weights quantised by an
 * offline tool are built into the engine's own layout), so that INT8 or FP8
 * codes quantised elsewhere can be loaded:
 *   src   int8 (or e4m3 bytes) [count][N][K], row-major, device memory;
 *   dst   int8 [count][N][K] in the fragment-tiled layout (matrix c at byte
 *         c*N*K), device memory, not overlapping src.
 * Per expert: w_gate_up is count = E, N = 2F (gate rows, then up rows),
 * K = H; w_down is count = E, N = H, K = F. The scales (s_gate_up, s_down)
 * and smooth/inv_smooth are plain arrays and need no packing.
 * Nothing is allocated; the copy is enqueued on `stream`.
 * Errors: MOE_W8A8_ERR_INVALID (NULL pointer, count, N or K <= 0, a pointer
 * not 16-byte aligned, overlapping buffers, more than 2^40 bytes),
 * MOE_W8A8_ERR_UNSUPPORTED (N % 16 != 0 or K % 64 != 0), MOE_W8A8_ERR_HIP. */
int moe_w8a8_pack(int64_t count, int32_t N, int32_t K, const int8_t *src, int8_t *dst,
                  void *stream);

/* ------------------------------------------------ the block around the layer
 * Operators of the decoder block that holds the layer, in the layer's own
 * quantisation scheme ("MiniMax-M3 W8A8 inference on K100AI" §3.2: per-channel
 * weights, per-token activations; §4.3: consecutive matmuls stay in the 8-bit
 * domain, conversion only where a norm or a residual needs it):
 *   moe_w8a8_act_quant  per-token codes of bf16 rows;
 *   moe_w8a8_linear     the matrix product with a scale per token and per
 *                       output channel (QKV and output projections, LM head);
 *   moe_w8a8_ffn        the gated feed-forward block (a dense layer's FFN, or
 *                       a shared expert whose gated result is added to the
 *                       routed experts' output);
 *   moe_w8a8_add_norm   the norms before and after a block with its gate,
 *                       residual scale and residual add, and the codes the
 *                       next product takes.
 *
 * Per-token codes, for a row v of fp32 values (v_j = fl32(x_j * inv_smooth_j)):
 * a = max |v_j|, code = rint(fl32(v_j * fl32(127/a))) clamped to [-127, 127]
 * (FP8: the nearest e4m3 of fl32(v_j * fl32(448/a)) clamped to +-448), scale =
 * fl32(a/127) (a/448). a = 0 gives codes 0 and scale 0. A row that holds a NaN
 * or an infinity gets codes 0 and a NaN scale, so that everything computed
 * from it is NaN and no other row is touched. For a < 2^-64 both v_j and a are
 * multiplied by 2^64 (exactly) before the two divisions, so that 127/a cannot
 * overflow; the scale is then taken back by 2^-64.
 *
 * Code rows q are row-major int8 (or e4m3 bytes) [T][Kp] with the row pitch
 * Kp = moe_w8a8_row_pitch(K), K rounded up to a multiple of 128. The operators
 * that make codes write zeros into columns K..Kp-1; codes from elsewhere must
 * have zeros there too (the products multiply those columns by zero weights:
 * INT8 garbage is harmless, but an e4m3 NaN is not).
 *
 * Rows of other matrices may be strided: ld_* is the distance between two rows
 * in elements, at least the row's width and at most 2^26. bf16 and fp32 rows
 * need only the alignment of their element type. T is below 2^22.
 *
 * T == 0 is a successful no-op whatever the pointers to tokens, results and
 * workspace are. */

/* Code rows' pitch in bytes for K columns; 0 for K outside [1, 65536]. */
int64_t moe_w8a8_row_pitch(int32_t K);

/* A quantised weight matrix W[N][K] (device memory; the struct is host memory).
 *   w          codes in the fragment-tiled layout of moe_w8a8_weights, with N
 *              padded to a multiple of 16 rows and K to Kp columns, zero codes
 *              in the padding: moe_w8a8_linear_codes_bytes(N, K, gated) bytes.
 *   scale      fp32 [moe_w8a8_linear_scales(N, gated)], one per (padded) row.
 *   inv_smooth fp32 [K], the reciprocal SmoothQuant scales that the tokens are
 *              multiplied by before they are coded, or NULL (all 1). Not used
 *              when the call is given codes.
 *   bias       fp32 [N], or NULL. Must be NULL where gated.
 *   gated      0: plain. 1: the gate and up projections of moe_w8a8_ffn,
 *              N = 2F rows given gate 0..F-1, then up 0..F-1, and held as F
 *              rounded up to a multiple of 32 rows of each, in alternating
 *              runs of 32 gate and 32 up rows (so that a gate value and its
 *              up value come out of one tile); `scale` follows that order.
 * Supported: K in [1, 65536], N in [1, 1048576]. */
typedef struct {
  int32_t in_features;  /* K */
  int32_t out_features; /* N (gated: 2F) */
  int32_t format;       /* MOE_W8A8_FORMAT_INT8 or _FP8 */
  int32_t gated;
  int8_t *w;
  float *scale;
  float *inv_smooth;
  float *bias;
} moe_w8a8_linear_weights;

/* Sizes of the buffers above; 0 for unsupported N, K or (gated) odd N. */
size_t moe_w8a8_linear_codes_bytes(int32_t N, int32_t K, int32_t gated);
int64_t moe_w8a8_linear_scales(int32_t N, int32_t gated);

/* Fill out->w and out->scale from unquantised weights: src fp32 (src_type
 * MOE_W8A8_F32) or bf16 (MOE_W8A8_BF16) [N][K] with row pitch ld_src. Rows are
 * multiplied by smooth (fp32 [K], or NULL) in fp32, then coded per row by the
 * rule above (a row with a NaN or an infinity gets codes 0 and scale NaN). The
 * buffers filled overlap neither src nor smooth (nor, below, src_scale). */
#define MOE_W8A8_BF16 0
#define MOE_W8A8_F32 1
int moe_w8a8_linear_quantise(const moe_w8a8_linear_weights *out, const void *src,
                             int32_t src_type, int64_t ld_src, const float *smooth,
                             void *stream);

/* The same from codes quantised elsewhere: src int8 (or e4m3 bytes) [N][K]
 * with row pitch ld_src, src_scale fp32 [N]. */
int moe_w8a8_linear_pack(const moe_w8a8_linear_weights *out, const int8_t *src, int64_t ld_src,
                         const float *src_scale, void *stream);

/* Activations of a product: exactly one of x and (q, s).
 *   x  bf16 [T][K], row pitch ld_x: coded per token inside the call;
 *   q  codes [T][Kp] (16-byte aligned, pitch Kp), s fp32 [T]. */
typedef struct {
  const uint16_t *x;
  int64_t ld_x;
  const int8_t *q;
  const float *s;
} moe_w8a8_act;

/* Result of a product y[T][N]: out[t][n] = round(gate[t] * y[t][n] + add[t][n]),
 * all in fp32 before the one rounding to out_type.
 *   out   bf16 or fp32 [T][N], row pitch ld_out; columns past N and rows past
 *         T are left as they were;
 *   gate  fp32 [T], or NULL (1);
 *   add   bf16 [T][N], row pitch ld_add, or NULL (0). May be `out` itself
 *         (out_type MOE_W8A8_BF16 and ld_add == ld_out); otherwise it must not
 *         overlap it. `out` overlaps no other input, the weights' buffers
 *         included (column blocks of one buffer with one pitch do not overlap). */
typedef struct {
  void *out;
  int64_t ld_out;
  int32_t out_type;
  const float *gate;
  const uint16_t *add;
  int64_t ld_add;
} moe_w8a8_result;

/* Per-token codes of bf16 rows x[T][K] (row pitch ld_x) in `format`, after
 * multiplying by inv_smooth (fp32 [K], or NULL): q [T][Kp], s fp32 [T], which
 * overlap neither an input nor each other. One launch, no workspace. Errors:
 * MOE_W8A8_ERR_INVALID, MOE_W8A8_ERR_UNSUPPORTED (K outside [1, 65536]),
 * MOE_W8A8_ERR_HIP. */
int moe_w8a8_act_quant(int32_t K, int32_t format, const uint16_t *x, int64_t ld_x, int64_t T,
                       const float *inv_smooth, int8_t *q, float *s, void *stream);

/* y[t][n] = s[t] * scale[n] * sum_k q[t][k] * w[n][k] + bias[n], then the
 * result's gate and add: the sum times s[t] first, in fp32, so a sum that leaves
 * the range there is infinite. INT8: the sum is exact (INT32). FP8: exact products
 * accumulated in fp32, except for bf16 results of more than 32 tokens. Those may
 * come from the FP8 matrix instructions, which keep the products of each eight
 * consecutive k (from a multiple of eight) to 13 bits below the largest of them
 * (truncated) before they add them in fp32: a sum is then off by at most
 * 7 * 2^-13 times the sum of the groups' largest |q| * largest |w| (1.5e-5 of the
 * sums' rms on normal data) beside the fp32 roundings. The sum's order depends on
 * the shape (T, N, K) and, for FP8, on out_type only: not on whether tokens or
 * their codes are given. `workspace` holds at least
 * moe_w8a8_linear_workspace_size(N, K, T) bytes (NULL where that is 0).
 * Errors: MOE_W8A8_ERR_INVALID (NULL or misaligned pointer, T outside
 * [0, 2^22), bad pitch, format or types, overlap, gated weights),
 * MOE_W8A8_ERR_UNSUPPORTED, MOE_W8A8_ERR_WORKSPACE, MOE_W8A8_ERR_HIP. */
size_t moe_w8a8_linear_workspace_size(int32_t N, int32_t K, int64_t T);
int moe_w8a8_linear(const moe_w8a8_linear_weights *weights, const moe_w8a8_act *act, int64_t T,
                    const moe_w8a8_result *result, void *workspace, size_t workspace_bytes,
                    void *stream);

/* Gated feed-forward block: (g, u) = the two halves of act . gate_up^T,
 * h = g / (1 + exp(-g)) * u in fp32, h coded per token by the rule above, then
 * y = h . down^T and the result's gate and add, as moe_w8a8_linear.
 * The sums of g and u are exact (INT8) or exact products accumulated in fp32
 * (FP8) at every T; those of y are moe_w8a8_linear's.
 *   gate_up  gated weights, N = 2F, K = H (no bias);
 *   down     plain weights, K = F, any N, the same format; inv_smooth NULL.
 * Workspace: moe_w8a8_ffn_workspace_size(H, F, N, T) bytes. */
size_t moe_w8a8_ffn_workspace_size(int32_t H, int32_t F, int32_t N, int64_t T);
int moe_w8a8_ffn(const moe_w8a8_linear_weights *gate_up, const moe_w8a8_linear_weights *down,
                 const moe_w8a8_act *act, int64_t T, const moe_w8a8_result *result,
                 void *workspace, size_t workspace_bytes, void *stream);

/* Norms before and after a block, fused with its gate and residual scale. For
 * each of T rows, in fp32:
 *   b = block_scale * gate * post(y)
 *   r = residual_scale * residual + b          -> residual_out (rounded once)
 *   n = pre(r)                                 -> normed (rounded once)
 *   codes of n (times inv_smooth)              -> q, s
 * r and n are not rounded in between. post and pre are one of
 *   MOE_W8A8_NORM_NONE   the identity (weight and bias must be NULL)
 *   MOE_W8A8_NORM_RMS    v / sqrt(mean(v^2) + eps) * weight + bias
 *   MOE_W8A8_NORM_LAYER  (v - mean) / sqrt(mean((v - mean)^2) + eps) * weight + bias
 * with fp32 [H] weight (NULL: 1) and bias (NULL: 0).
 *   y            bf16 [T][H], row pitch ld_y: the block's output
 *   residual     bf16 or fp32 (residual_type) [T][H], pitch ld_residual, or
 *                NULL (0); residual_out, of the same type with pitch
 *                ld_residual_out, or NULL. It may be `residual` itself with
 *                the same pitch.
 *   gate_token   fp32 [T], or NULL (1); and
 *   gate_rows    bf16 [ceil(T / gate_group)][H], pitch ld_gate: row t takes
 *                gate row t / gate_group (gate_group >= T: one gate per
 *                channel; 1: a gate of its own; the tokens of a sequence: a
 *                gate per sequence), or NULL (1). At most one of the two.
 *   normed       bf16 [T][H], pitch ld_normed, or NULL; may be `y` itself with
 *                the same pitch.
 *   q, s         codes [T][Kp] and scales [T] in `format`, or both NULL.
 * At least one of residual_out, normed and q. Apart from what is said above,
 * outputs overlap neither inputs nor each other. Supported: H in [1, 65536].
 * One launch, no workspace. */
#define MOE_W8A8_NORM_NONE 0
#define MOE_W8A8_NORM_RMS 1
#define MOE_W8A8_NORM_LAYER 2
typedef struct {
  int32_t hidden;
  int32_t pre_norm, post_norm;
  int32_t residual_type; /* MOE_W8A8_BF16 or MOE_W8A8_F32 */
  int32_t format;        /* of q */
  float eps, residual_scale, block_scale;
  const uint16_t *y;
  int64_t ld_y;
  const void *residual;
  int64_t ld_residual;
  void *residual_out;
  int64_t ld_residual_out;
  const float *post_weight, *post_bias;
  const float *pre_weight, *pre_bias;
  const float *gate_token;
  const uint16_t *gate_rows;
  int64_t ld_gate, gate_group;
  uint16_t *normed;
  int64_t ld_normed;
  const float *inv_smooth;
  int8_t *q;
  float *s;
} moe_w8a8_add_norm_args;
int moe_w8a8_add_norm(const moe_w8a8_add_norm_args *args, int64_t T, void *stream);

/* ------------------------------------------- attention between the projections
 * What lies between a block's QKV projection and its output projection, over a
 * paged cache in the same quantisation, and what the LM head's logits answer:
 *   moe_w8a8_qk_norm_rope      norms of queries and keys for each head and the
 *                              position rotation in one pass; keys and values go
 *                              into the cache;
 *   moe_w8a8_paged_attention   attention of the batch's new tokens (one for each
 *                              sequence, or chunks) over the cache;
 *   moe_w8a8_token_logprobs    log probabilities of given tokens, entropy, top
 *                              alternatives.
 *
 * A cache of keys and values in pages (device memory; the struct is host memory).
 *   k, v         [num_pages][kv_heads][page_size][head_dim] in `format`: bf16, int8
 *                or e4m3 bytes; 16-byte aligned. Each page is contiguous; page p
 *                begins page_stride elements after page p - 1 (at least a page, a
 *                multiple of 16), so that one buffer can hold many caches.
 *   k_scale,     fp32 [num_pages][kv_heads][page_size], 16-byte aligned, pages
 *   v_scale      scale_stride values apart (a multiple of 4): an element stands for
 *                code * scale. NULL for a bf16 cache.
 * Supported: head_dim 64, 128, 256; page_size 16, 32, 64, 128, 256; kv_heads up to
 * 1024; num_pages from 1; strides up to 2^34. */
#define MOE_W8A8_CACHE_BF16 2
typedef struct {
  int32_t num_pages, page_size, kv_heads, head_dim;
  int32_t format; /* MOE_W8A8_CACHE_BF16, MOE_W8A8_FORMAT_INT8 or _FP8 */
  void *k, *v;
  int64_t page_stride;
  float *k_scale, *v_scale;
  int64_t scale_stride;
} moe_w8a8_kv_cache;

/* The sequences of a step (device memory, read when the kernels run: a captured
 * call follows what is written there later).
 *   cu_tokens   int32 [num_seqs + 1]: the new tokens of sequence b are token rows
 *               cu_tokens[b] .. cu_tokens[b + 1] - 1. Values are taken into
 *               [0, T], a sequence that ends before it begins has none. Rows behind
 *               the last sequence are neither read nor written.
 *   lengths     int32 [num_seqs]: keys of the sequence in the cache, its new tokens
 *               (the last ones) included: new token i of n is at place
 *               length - n + i. A token of negative place has no place in the
 *               cache. Lengths are taken into [0, table_width * page_size], and to
 *               2^31 - 1024 at most.
 *   page_table  int32 [num_seqs][table_width], pitch ld_table: place p of sequence b
 *               lies in page page_table[b][p / page_size]. A page outside [0,
 *               num_pages) holds nothing: its keys are not seen, and what is
 *               written there is dropped.
 *   max_tokens  the most new tokens of a sequence: a bound (tokens past it are not
 *               computed).
 *   max_length  about the longest length: it sizes the launch, a longer one is still
 *               computed right. */
typedef struct {
  int32_t num_seqs, max_tokens, max_length, table_width;
  const int32_t *cu_tokens, *lengths, *page_table;
  int64_t ld_table;
} moe_w8a8_batch;

/* Queries and keys normed for each head and rotated by their position; keys and
 * values written into the cache at their tokens' places. With D = head_dim, for each
 * head row x[D] of the queries and of the keys, in fp32:
 *   norm != 0:   x = x / sqrt(mean(x^2) + eps) * weight (q_weight or k_weight, fp32
 *                [D], or NULL: 1)
 *   rotary > 0:  for i < rotary / 2, with t = position * inv_freq[i] (in fp64):
 *                (a, b) = (a cos t - b sin t, b cos t + a sin t), where (a, b) is
 *                (x[i], x[i + rotary/2]), or, interleaved, (x[2i], x[2i + 1])
 * and one rounding: queries and a bf16 cache to bf16, an INT8 or FP8 cache to codes of
 * the D values with a scale of their own by the rule of the per-token codes above (a
 * head row that holds a NaN or an infinity gets codes 0 and a NaN scale). Values are
 * written as they are (or coded). No two tokens may have the same place.
 *   qkv        bf16 [T][(heads + 2 kv_heads) D], pitch ld_qkv: query heads, key heads,
 *              value heads
 *   q          bf16 [T][heads D], pitch ld_q; may be `qkv` itself with the same pitch
 *   inv_freq   fp64 [rotary / 2], not NULL where rotary > 0
 *   positions  int64 [T], or NULL: each token's place
 * q_weight and k_weight are NULL where norm is 0. `q` overlaps no other input and not
 * the cache, nor does the cache overlap an input. Supported: heads up to 65536 / D,
 * rotary a multiple of 16 up to D. One launch, no workspace. T below 2^22. Errors:
 * MOE_W8A8_ERR_INVALID, MOE_W8A8_ERR_UNSUPPORTED, MOE_W8A8_ERR_HIP. T == 0 is a no-op. */
typedef struct {
  int32_t heads, norm, rotary, interleaved;
  float eps;
  const uint16_t *qkv;
  int64_t ld_qkv;
  uint16_t *q;
  int64_t ld_q;
  const float *q_weight, *k_weight;
  const double *inv_freq;
  const int64_t *positions;
} moe_w8a8_qk_norm_rope_args;
int moe_w8a8_qk_norm_rope(const moe_w8a8_qk_norm_rope_args *args, const moe_w8a8_kv_cache *cache,
                          const moe_w8a8_batch *batch, int64_t T, void *stream);

/* Attention of the new tokens over the cache. Query head j of `heads` reads kv head
 * j / (heads / kv_heads). A token at place p sees the keys at places c < length with
 * c <= p (causal) and c > p - window (window > 0), in pages that exist:
 *   out = sum_c softmax_c(scale * q . k_c) v_c
 * A token that sees no key gets zeros; keys and values that it does not see have no
 * part in its result, whatever they hold. What it does see counts as it is: a score of -inf
 * has no weight, and if every one is, or one is +inf or NaN, the result is NaN. Products are
 * exact and summed in fp32, the softmax is fp32, and each probability (times its value's
 * scale) is rounded to bf16 before it multiplies the values, half a step of 2^-8: to two bf16
 * terms, 2^-17, for sequences of up to 32 query rows of a kv head (new tokens times heads /
 * kv_heads; 16 of 256-wide heads) in any batch. The result is divided by the probabilities'
 * sum at the end (values whose sum over the keys passes 2^119 may be infinite there) and
 * rounded once.
 *   q    bf16 [T][heads D], pitch ld_q;  out  bf16 [T][heads D], pitch ld_out, which
 *        overlaps neither q nor the cache nor the batch's arrays.
 * Supported: heads a multiple of kv_heads up to 65536 / D; window >= 0 (0: none); scale
 * finite. `workspace` holds at least moe_w8a8_paged_attention_workspace_size bytes
 * (256-byte aligned; 0 for arguments that are refused). T below 2^22. Errors:
 * MOE_W8A8_ERR_INVALID, MOE_W8A8_ERR_UNSUPPORTED, MOE_W8A8_ERR_WORKSPACE,
 * MOE_W8A8_ERR_HIP. T == 0 is a no-op. */
typedef struct {
  int32_t heads, causal, window;
  float scale;
  const uint16_t *q;
  int64_t ld_q;
  uint16_t *out;
  int64_t ld_out;
} moe_w8a8_attention_args;
size_t moe_w8a8_paged_attention_workspace_size(const moe_w8a8_kv_cache *cache,
                                               const moe_w8a8_batch *batch, int32_t heads,
                                               int64_t T);
int moe_w8a8_paged_attention(const moe_w8a8_attention_args *args, const moe_w8a8_kv_cache *cache,
                             const moe_w8a8_batch *batch, int64_t T, void *workspace,
                             size_t workspace_bytes, void *stream);

/* For each row x[V] of logits (bf16 or fp32, `type`), with z = log sum_j exp(x_j):
 *   logprobs[t]      x[tokens[t]] - z (NaN for a token outside [0, V))
 *   entropy[t]       z - sum_j exp(x_j - z) x_j
 *   top_tokens[t][]  the `top` tokens of largest logit, in falling order, of equal
 *                    ones the lower first; top_logprobs[t][]  their x - z
 * in fp32, relative to the row's largest logit. Logits of -inf have probability 0. A row
 * that holds a NaN or +inf, or nothing but -inf, has NaN results; its top tokens are
 * still ordered (a NaN counts as larger than every number).
 *   logits  [T][V], pitch ld;  tokens int64 [T], or NULL (then logprobs is NULL)
 *   logprobs, entropy  fp32 [T], or NULL;  top_tokens int64, top_logprobs fp32
 *           [T][top], both or neither (top 0)
 * Supported: V in [1, 2^20], top in [0, min(V, 64)]. Outputs overlap neither an input
 * nor each other. Workspace: moe_w8a8_token_logprobs_workspace_size bytes, 256-byte
 * aligned (NULL where that is 0). T below 2^22. Errors: MOE_W8A8_ERR_INVALID,
 * MOE_W8A8_ERR_UNSUPPORTED, MOE_W8A8_ERR_WORKSPACE, MOE_W8A8_ERR_HIP. T == 0 is a
 * no-op. */
typedef struct {
  int32_t vocab, type, top; /* type: MOE_W8A8_BF16 or MOE_W8A8_F32 */
  const void *logits;
  int64_t ld;
  const int64_t *tokens;
  float *logprobs, *entropy;
  int64_t *top_tokens;
  float *top_logprobs;
} moe_w8a8_logprobs_args;
size_t moe_w8a8_token_logprobs_workspace_size(int32_t vocab, int32_t top, int64_t T);
int moe_w8a8_token_logprobs(const moe_w8a8_logprobs_args *args, int64_t T, void *workspace,
                            size_t workspace_bytes, void *stream);

/* Static description of a return code (never NULL). */
const char *moe_w8a8_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W8A8_H */
