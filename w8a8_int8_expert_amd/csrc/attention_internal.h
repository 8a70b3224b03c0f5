// attention_internal.h -- internal declarations of the operators over the paged
// cache (moe_w8a8_qk_norm_rope, _paged_attention) and of _token_logprobs. Not part
// of the public ABI (include/moe_w8a8.h).
#pragma once

#include "block_internal.h"

namespace moe {

constexpr int kBf16Cache = MOE_W8A8_CACHE_BF16;

// A cache and a step's sequences as the kernels take them. Sizes in bytes are of
// keys and values alike.
struct CacheView {
  char *k, *v;
  float *k_scale, *v_scale;
  int64_t page_bytes, scale_stride;  // from one page to the next
  int num_pages, log2_page, kv_heads;
};
struct BatchView {
  const int32_t *cu, *lengths, *table;
  int64_t ld_table;
  int num_seqs, max_tokens, T;
  int most;  // places that the page table has room for
};

// Rows and keys of one sequence: first token row, new tokens, keys. Whatever the
// arrays hold, rows lie in [0, T) and keys in what the table covers.
struct Seq {
  int start, n, len;
};

#if defined(__HIP_DEVICE_COMPILE__) || defined(__HIPCC__)
__device__ __forceinline__ int clamp_int(int v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : v;
}
__device__ __forceinline__ Seq seq_of(const BatchView &bt, int b) {
  Seq s;
  s.start = clamp_int(bt.cu[b], 0, bt.T);
  const int end = clamp_int(bt.cu[b + 1], s.start, bt.T);
  s.n = end - s.start;
  s.len = clamp_int(bt.lengths[b], 0, bt.most);
  return s;
}
// Keys [lo, hi) that the token at `place` of a sequence of `len` keys sees.
__device__ __forceinline__ int seen_hi(int place, int len, bool causal) {
  return causal ? (place + 1 < len ? place + 1 : len) : len;
}
__device__ __forceinline__ int seen_lo(int place, int window) {
  // (places may be negative: nothing is taken from one)
  return window > 0 && place >= window ? place - window + 1 : 0;
}
#endif

struct RopeArgs {
  const uint16_t *qkv;
  int64_t ld_qkv;
  uint16_t *q;
  int64_t ld_q;
  const float *q_weight, *k_weight;
  const double *inv_freq;
  const int64_t *positions;
  int heads, rotary;
  bool norm, interleaved;
  float eps;
};
hipError_t launch_qk_norm_rope(const RopeArgs &a, const CacheView &c, int D, int format,
                               const BatchView &b, hipStream_t st);

struct AttnArgs {
  const uint16_t *q;
  int64_t ld_q;
  uint16_t *out;
  int64_t ld_out;
  int heads, group;  // query heads, and of them to one kv head
  bool causal;
  int window;
  float scale2;   // scale * log2(e): the softmax is taken to base 2
  int few_rows;   // sequences of at most so many query rows of a kv head go to the kernel
                  // of few rows, the others to that of tiles
};

constexpr int kMostBlocks = 1 << 20;  // a launch counts threads in 32 bits
constexpr int kFewKeys = 32;  // keys of a tile of the kernel of few rows
template <int D>
constexpr int kManyKeys = D == 256 ? 32 : 64;  // of the kernel of tiles
constexpr int kLeastFew = 4;                   // least piece: 128 keys, a tile a wavefront
template <int D>
constexpr int kLeastMany = 512 / kManyKeys<D>;  // 512 keys

// Which kernels run, their launch sizes and the workspace, from shapes alone. Of each
// kv head: a number of units that the keys are split into, about; the slots for partial
// results that these can need; and the units launched (a block strides over the rest).
struct AttnPlan {
  int few_rows;   // as in AttnArgs; 0: the kernel of few rows does not run
  int row_tiles;  // 16-row tiles of the kernel of few rows
  int row_target, row_slots, row_grid;
  bool tiles;     // whether the kernel of tiles runs
  int tile_target, tile_slots, tile_grid;
  size_t tile_at, total;  // bytes before the partial results of tiles, and of all
};
// Blocks of the kernel of few rows that its units are made for, on a compute unit: as many as
// its LDS holds tiles for (of narrow 8-bit heads half as many; 32 rows of 128-wide heads fill
// its registers). One round of long units: each wavefront has the next tile on its way all
// along, and there are fewer partial results. With 1024 units whatever the type, 1 sequence of
// 16384 keys, 8 kv heads of 128, bf16, takes 33.9 us instead of 22.1, 32 of 8192 with 8 tokens 237
// instead of 194, with INT8 223 instead of 191, 16 of 4096, 2 of 256, 58 instead of 36, 32 of
// 8192, one token, INT8, 114 instead of 110; with 256 units these last take 142.
constexpr int rows_per_unit(int D, int format, int row_tiles) {
  return D * (format == kBf16Cache ? 2 : 1) < 256 && D * row_tiles < 256 ? 2 : 1;
}
AttnPlan attention_plan(const CacheView &c, int D, int format, const BatchView &b, int heads,
                        int max_length);
hipError_t launch_attention_rows(const AttnArgs &a, const CacheView &c, int D, int format,
                                 const BatchView &b, const AttnPlan &p, float *partial,
                                 hipStream_t st);
// Partial results: of each kv head `slots` of so many rows (16 or 32, and kTileRows) of
// D values, then as many (maximum, sum).
struct Partial {
  float *o, *ml;
  int slots;
};
constexpr int kTileRows = 128;  // query rows of a block of the kernel of tiles
inline Partial partial_few(const AttnPlan &p, int kv_heads, int D, float *ws) {
  return Partial{ws, ws + (size_t)p.row_slots * kv_heads * 16 * p.row_tiles * D, p.row_slots};
}
inline Partial partial_many(const AttnPlan &p, int kv_heads, int D, float *ws) {
  float *const at = reinterpret_cast<float *>((char *)ws + p.tile_at);
  return Partial{at, at + (size_t)p.tile_slots * kv_heads * kTileRows * D, p.tile_slots};
}
hipError_t launch_attention_tiles(const AttnArgs &a, const CacheView &c, int D, int format,
                                  const BatchView &b, const AttnPlan &p, float *partial,
                                  hipStream_t st);
hipError_t launch_attention_join(const AttnArgs &a, const CacheView &c, int D, const BatchView &b,
                                 const AttnPlan &p, float *partial, hipStream_t st);

struct LogprobArgs {
  const void *x;
  int64_t ld;
  const int64_t *tokens;
  float *logprobs, *entropy;
  int64_t *top_tokens;
  float *top_logprobs;
  int V, top;
};
size_t token_logprobs_workspace(int V, int top, int64_t T);
hipError_t launch_token_logprobs(const LogprobArgs &a, bool f32, int64_t T, void *ws,
                                 hipStream_t st);

}  // namespace moe
