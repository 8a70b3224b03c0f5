// block_internal.h -- internal declarations of the operators of the block
// around the layer (moe_w8a8_linear, _ffn, _act_quant, _add_norm). Not part of
// the public ABI (include/moe_w8a8.h).
#pragma once

#include "moe_internal.h"
#include "moe_w8a8.h"

namespace moe {

constexpr int kMaxWidth = 65536;      // K, H, F
constexpr int kMaxOutputs = 1 << 20;  // N
// Pitch of code rows (and of the h rows): 128 columns are one cache line of
// codes and the pair of 64-k tiles that an FP8 matrix instruction takes.
inline __host__ __device__ int row_pitch(int K) { return (K + 127) / 128 * 128; }
// Rows of a packed weight matrix: N rounded up to whole 16-row tiles; gated,
// F = N/2 rounded up to 32 in runs of 32 gate rows and 32 up rows.
inline __host__ __device__ int packed_rows(int N, bool gated) {
  return gated ? (N / 2 + 31) / 32 * 64 : (N + 15) / 16 * 16;
}
// Source row of packed row p, or -1 (padding).
inline __host__ __device__ int source_row(int p, int N, bool gated) {
  if (!gated) return p < N ? p : -1;
  const int F = N / 2, f = p / 64 * 32 + p % 32;
  return f < F ? (p / 32 % 2) * F + f : -1;
}

// Where code k of row t is. Codes that only a streaming product reads lie in
// tiles of 16 rows x 64 k, as the weights do: an operand load then takes whole
// cache lines, against half a line of each of 16 rows (and the lines in flight are
// what bounds it). The row count is rounded up to whole tiles.
inline __host__ __device__ size_t code_at(bool tiles, int64_t t, int k, int Kp) {
  return tiles ? ((size_t)(t >> 4) * (size_t)(Kp >> 6) + (size_t)(k >> 6)) * 1024 +
                     (size_t)((((k >> 4) & 3) * 16 + (int)(t & 15)) * 16 + (k & 15))
               : (size_t)t * (size_t)Kp + (size_t)k;
}

// What a product does with its sums.
struct Epilogue {
  const float *row_scale;  // [T]
  const float *scale;      // per packed row
  const float *bias;       // [N] or NULL
  int N;                   // columns of out (plain), F (gated)
  void *out;               // plain: bf16 or fp32 [T][ld_out]; gated: h fp32 [T][ld_out]
  int64_t ld_out;
  int out_f32;
  const float *gate;  // [T] or NULL
  const uint16_t *add;
  int64_t ld_add;
  uint32_t *amax;  // gated: row max |h| (float bits), or NULL
};

// Which product runs. Streaming reads the weights once and every block all
// tokens; tiles read both several times, but the weights in larger panels, and
// split K over blocks. Up to 32 tokens streaming is the faster almost
// everywhere, beyond 64 never; between them it depends on how much there is to
// read (us, streaming against tiles, INT8, from bf16 tokens): 32 tokens, K 4096,
// 8192 outputs 11.9, 14.7; 40 tokens, K 4096, 8192 outputs 12.8, 15.6; 64 tokens,
// K 4096, 4096 outputs 10.7, 14.4, 8192 outputs 14.2, 15.8, 11000 outputs 21.0,
// 17.6; K 8192, 4096 outputs 17.7, 16.7; K 2048, 16384 outputs 14.1, 13.2, 32003
// outputs 25.2, 18.0. (Row-major codes cost streaming up to 2.2 more at 64 tokens;
// the choice is the same for both, so that a sum's order is.)
constexpr int kStreamRows = 64;   // most that stream
constexpr int kAlwaysStream = 32; // fewer always do
inline bool streams(int64_t T, int K, int Np) {
  if (T <= kAlwaysStream) return true;
  if (T > kStreamRows) return false;
  return K <= 4096 && Np <= 8192;
}
// Rows that a streaming product codes itself, every block over again: tokens,
// and the hidden rows of a feed-forward block (twice the values to read, and
// SwiGLU to compute).
constexpr int kFusedRows = 4;
constexpr int kFusedTokens = 16384, kFusedHidden = 8192;
inline bool fused_tokens(int64_t T, int K) {
  return T <= kFusedRows && T * row_pitch(K) <= kFusedTokens;
}
inline bool fused_hidden(int64_t T, int F) {
  return T <= kFusedRows && T * row_pitch(F) <= kFusedHidden;
}
// Partial sums of the products that split K over blocks.
constexpr size_t kPartialBytes = (size_t)32 << 20;

hipError_t launch_act_rows(const uint16_t *x, int64_t ld_x, int64_t T, int K, const float *inv,
                           bool fp8, bool tiles, int8_t *q, float *s, uint32_t *clear,
                           hipStream_t st);
hipError_t launch_clear(uint32_t *p, int64_t n, hipStream_t st);
// Gate and up values fp32 [T][ld] in packed order (a streaming product's plain
// output) -> codes [T][Fp] and scales of h = silu(g) u
hipError_t launch_hidden_rows(const float *gu, int64_t ld, int64_t T, int F, bool fp8, bool tiles,
                              int8_t *q, float *s, hipStream_t st);
// h fp32 [T][Fp] with row max |h| -> codes [T][Fp], scales
hipError_t launch_requant_rows(const float *h, const uint32_t *amax, int64_t T, int F, bool fp8,
                               int8_t *q, float *s, hipStream_t st);
hipError_t launch_add_norm(const moe_w8a8_add_norm_args &a, int64_t T, hipStream_t st);
// src_type: MOE_W8A8_BF16, MOE_W8A8_F32, or -1 for codes (with their scales)
hipError_t launch_pack_rows(const moe_w8a8_linear_weights &w, const void *src, int src_type,
                            int64_t ld, const float *smooth, const float *src_scale,
                            hipStream_t st);
// T <= kStreamRows; codes q (row scales in Epilogue), or (T <= kFusedRows) rows
// that the kernel codes itself: bf16 tokens x, or the hidden rows of gate and
// up values h in packed order.
struct StreamIn {
  const int8_t *q;  // codes, or NULL
  bool tiles;       // codes in tiles of 16 rows x 64 k (code_at), not [T][Kp]
  const uint16_t *x;
  const float *h;
  int64_t ld;        // of x or h
  const float *inv;  // of x
};
hipError_t launch_linear_stream(const StreamIn &in, int T, const int8_t *w, int K, int Np, bool fp8,
                                const Epilogue &ep, hipStream_t st);
hipError_t launch_linear_tiled(const int8_t *q, int64_t T, const int8_t *w, int K, int Np,
                               bool gated, bool fp8, const Epilogue &ep, void *partial,
                               hipStream_t st);

}  // namespace moe
