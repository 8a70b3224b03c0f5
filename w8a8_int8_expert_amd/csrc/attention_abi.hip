// attention_abi.hip -- host side of moe_w8a8_qk_norm_rope, _paged_attention and
// _token_logprobs: argument validation before anything touches HIP, workspace sizes
// and the launches on the caller's stream.
#include <math.h>

#include "attention_internal.h"
#include "host_checks.h"

using namespace moe;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 34;  // (16ths of a page's bytes: 32 bits)
constexpr int kMaxSeqs = 1 << 20;
constexpr int kMaxTop = 64;
constexpr int kMaxVocab = 1 << 20;

int elem(const moe_w8a8_kv_cache &c) { return c.format == kBf16Cache ? 2 : 1; }
int64_t page_elems(const moe_w8a8_kv_cache &c) {
  return (int64_t)c.page_size * c.kv_heads * c.head_dim;
}
int log2_of(int v) {
  int l = 0;
  while (v >> (l + 1)) ++l;
  return l;
}

// Shape and format (what the workspace depends on), without the pointers.
int cache_shape(const moe_w8a8_kv_cache *c) {
  if (!c || c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1 ||
      (c->format != kBf16Cache && !format_ok(c->format)))
    return MOE_W8A8_ERR_INVALID;
  if ((c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) || c->page_size < 16 ||
      c->page_size > 256 || (c->page_size & (c->page_size - 1)) || c->kv_heads > 1024)
    return MOE_W8A8_ERR_UNSUPPORTED;
  return MOE_W8A8_OK;
}
int cache_check(const moe_w8a8_kv_cache *c) {
  MOE_TRY(cache_shape(c));
  if (!c->k || !c->v || !al(c->k, 16) || !al(c->v, 16) || c->page_stride < page_elems(*c) ||
      c->page_stride > kMaxStride || c->page_stride % 16)
    return MOE_W8A8_ERR_INVALID;
  if (c->format == kBf16Cache)
    return c->k_scale || c->v_scale ? MOE_W8A8_ERR_INVALID : MOE_W8A8_OK;
  if (!c->k_scale || !c->v_scale || !al(c->k_scale, 16) || !al(c->v_scale, 16) ||
      c->scale_stride < (int64_t)c->page_size * c->kv_heads || c->scale_stride > kMaxStride ||
      c->scale_stride % 4)
    return MOE_W8A8_ERR_INVALID;
  return MOE_W8A8_OK;
}
int batch_shape(const moe_w8a8_batch *b) {
  if (!b || b->num_seqs < 0 || b->max_tokens < 0 || b->max_length < 0 || b->table_width < 0)
    return MOE_W8A8_ERR_INVALID;
  return b->num_seqs > kMaxSeqs ? MOE_W8A8_ERR_UNSUPPORTED : MOE_W8A8_OK;
}
int batch_check(const moe_w8a8_batch *b) {
  MOE_TRY(batch_shape(b));
  if (b->num_seqs == 0) return MOE_W8A8_OK;
  if (!b->cu_tokens || !b->lengths || !al(b->cu_tokens, 4) || !al(b->lengths, 4) ||
      !al(b->page_table, 4) || (b->table_width > 0 && !b->page_table) ||
      b->ld_table < b->table_width || b->ld_table > kMaxPitch)
    return MOE_W8A8_ERR_INVALID;
  return MOE_W8A8_OK;
}

// The cache's buffers, as their pages span them, and the batch's arrays.
struct Buffers {
  Mat m[7];
};
Buffers buffers(const moe_w8a8_kv_cache &c, const moe_w8a8_batch &b) {
  Buffers r{};
  auto pages = [&](const void *p, int64_t stride, int64_t each, size_t size) {
    return mat(p, c.num_pages, stride, each, size);
  };
  r.m[0] = pages(c.k, c.page_stride, page_elems(c), elem(c));
  r.m[1] = pages(c.v, c.page_stride, page_elems(c), elem(c));
  if (c.k_scale) {
    r.m[2] = pages(c.k_scale, c.scale_stride, (int64_t)c.page_size * c.kv_heads, 4);
    r.m[3] = pages(c.v_scale, c.scale_stride, (int64_t)c.page_size * c.kv_heads, 4);
  }
  r.m[4] = flat(b.cu_tokens, ((size_t)b.num_seqs + 1) * 4);
  r.m[5] = flat(b.lengths, (size_t)b.num_seqs * 4);
  r.m[6] = mat(b.table_width ? b.page_table : nullptr, b.num_seqs, b.ld_table, b.table_width, 4);
  return r;
}

CacheView view(const moe_w8a8_kv_cache &c) {
  CacheView v{};
  v.k = (char *)c.k; v.v = (char *)c.v; v.k_scale = c.k_scale; v.v_scale = c.v_scale;
  v.page_bytes = c.page_stride * elem(c); v.scale_stride = c.scale_stride;
  v.num_pages = c.num_pages; v.log2_page = log2_of(c.page_size); v.kv_heads = c.kv_heads;
  return v;
}
BatchView view(const moe_w8a8_batch &b, int page_size, int64_t T) {
  BatchView v{};
  v.cu = b.cu_tokens; v.lengths = b.lengths; v.table = b.page_table; v.ld_table = b.ld_table;
  v.num_seqs = b.num_seqs; v.T = (int)T;
  // (no sequence has more new tokens than there are rows)
  v.max_tokens = b.max_tokens < T ? b.max_tokens : (int)T;
  // (tiles are looked up to 8 tiles and a half of 32 keys past a sequence's end, in 32 bits)
  const int64_t most = (int64_t)b.table_width * page_size, top = 0x7fffffff - 1023;
  v.most = (int)(most < top ? most : top);
  return v;
}
bool heads_ok(int32_t heads, int D) { return heads <= kMaxWidth / D; }

}  // namespace

extern "C" int moe_w8a8_qk_norm_rope(const moe_w8a8_qk_norm_rope_args *a,
                                     const moe_w8a8_kv_cache *c, const moe_w8a8_batch *b, int64_t T,
                                     void *stream) {
  if (!a || T < 0 || T > kMaxRows || a->heads < 1 || a->rotary < 0 || !isfinite(a->eps) ||
      a->eps < 0.0f || (!a->norm && (a->q_weight || a->k_weight)))
    return MOE_W8A8_ERR_INVALID;
  MOE_TRY(cache_check(c));
  MOE_TRY(batch_check(b));
  const int D = c->head_dim;
  if (!heads_ok(a->heads, D) || a->rotary > D || a->rotary % 16) return MOE_W8A8_ERR_UNSUPPORTED;
  if (T == 0 || b->num_seqs == 0) return MOE_W8A8_OK;
  const int64_t in = (int64_t)(a->heads + 2 * c->kv_heads) * D, out = (int64_t)a->heads * D;
  if (!a->qkv || !a->q || !al(a->qkv, 2) || !al(a->q, 2) || !pitch_ok(a->ld_qkv, in) ||
      !pitch_ok(a->ld_q, out) || !al(a->q_weight, 4) || !al(a->k_weight, 4) ||
      (a->rotary > 0 && !a->inv_freq) || !al(a->inv_freq, 8) || !al(a->positions, 8))
    return MOE_W8A8_ERR_INVALID;
  const Mat q = mat(a->q, T, a->ld_q, out, 2), qkv = mat(a->qkv, T, a->ld_qkv, in, 2);
  const Mat ins[4] = {flat(a->q_weight, (size_t)D * 4), flat(a->k_weight, (size_t)D * 4),
                      flat(a->inv_freq, (size_t)a->rotary * 4),
                      flat(a->positions, (size_t)T * 8)};
  const bool in_place = a->q == a->qkv && a->ld_q == a->ld_qkv;
  if (!in_place && overlap(q, qkv)) return MOE_W8A8_ERR_INVALID;
  const Buffers bf = buffers(*c, *b);
  for (const Mat &m : ins)
    if (overlap(q, m)) return MOE_W8A8_ERR_INVALID;
  for (int i = 0; i < 7; ++i) {
    if (overlap(q, bf.m[i])) return MOE_W8A8_ERR_INVALID;
    if (i >= 4) continue;
    if (overlap(bf.m[i], qkv)) return MOE_W8A8_ERR_INVALID;
    for (const Mat &m : ins)
      if (overlap(bf.m[i], m)) return MOE_W8A8_ERR_INVALID;
    for (int j = i + 1; j < 7; ++j)
      if (overlap(bf.m[i], bf.m[j])) return MOE_W8A8_ERR_INVALID;
  }
  RopeArgs r{};
  r.qkv = a->qkv; r.ld_qkv = a->ld_qkv; r.q = a->q; r.ld_q = a->ld_q;
  r.q_weight = a->q_weight; r.k_weight = a->k_weight; r.inv_freq = a->inv_freq;
  r.positions = a->positions; r.heads = a->heads; r.rotary = a->rotary;
  r.norm = a->norm != 0; r.interleaved = a->interleaved != 0; r.eps = a->eps;
  MOE_CHECK(launch_qk_norm_rope(r, view(*c), D, c->format, view(*b, c->page_size, T),
                                (hipStream_t)stream));
  return MOE_W8A8_OK;
}

AttnPlan moe::attention_plan(const CacheView &c, int D, int format, const BatchView &b, int heads,
                             int max_length) {
  AttnPlan p{};
  const int group = heads / c.kv_heads;
  const int64_t rows = (int64_t)b.max_tokens * group;  // most of a sequence and kv head
  const int most_few = D == 256 ? 16 : 32;
  const int grid_cap = kMostBlocks / 2 / c.kv_heads;
  auto at_most = [](int64_t v, int64_t most) { return (int)(v < most ? v : most); };
  // Slots for pieces: about twice the target at most, and no more than the table's places can
  // be cut into, for every row block that a sequence may have (whatever the arrays hold). A
  // sequence whose places make one piece needs none.
  auto slots = [&](int64_t row_blocks, int keys, int least, int target) {
    const int64_t tiles = ((int64_t)b.most + keys - 1) / keys, pieces = (tiles + least - 1) / least;
    const int64_t of_one = at_most(row_blocks * pieces, 2 * target);
    return pieces > 1 ? at_most(b.num_seqs * of_one, 2 * target) : 0;
  };
  // All sequences have few rows; or some may, beside longer ones or alone in a step with room
  // for more (rows and bounds say nothing of what the arrays hold: a sequence of few rows is
  // taken the same way in every batch). A launch that finds none costs 4 us: 64 tokens over
  // 4096 keys, bf16, 30.4 us, 26.5 without it, 8192 from their start 565 and 561.
  const bool all_few = rows <= most_few;
  const bool some_few = group <= most_few;
  size_t total = 0;
  if (all_few || some_few) {
    p.few_rows = most_few;
    p.row_tiles = at_most(rows, most_few) <= 16 ? 1 : 2;
    p.row_target = (256 * rows_per_unit(D, format, p.row_tiles) + c.kv_heads - 1) / c.kv_heads;
    p.row_slots = slots(1, kFewKeys, kLeastFew, p.row_target);
    // (keys of 128 at least make a unit)
    const int64_t units = (int64_t)b.num_seqs * ((max_length + 127) / 128 + 1);
    p.row_grid = at_most(at_most(units, (int64_t)p.row_target + b.num_seqs), grid_cap);
    total += up256((size_t)p.row_slots * c.kv_heads * 16 * p.row_tiles * (D + 2) * sizeof(float));
  }
  p.tile_at = total;
  if (!all_few) {
    p.tiles = true;
    // blocks of rows that the batch can make
    const int64_t blocks = (int64_t)b.T * group / kTileRows + at_most(b.num_seqs, b.T);
    const int64_t of_one = (rows + kTileRows - 1) / kTileRows;  // the most of one sequence
    p.tile_target = (1024 + c.kv_heads - 1) / c.kv_heads;
    p.tile_slots = D == 256 ? slots(of_one, kManyKeys<256>, kLeastMany<256>, p.tile_target)
                            : slots(of_one, kManyKeys<128>, kLeastMany<128>, p.tile_target);
    p.tile_grid = at_most(blocks + p.tile_target, grid_cap);
    total += up256((size_t)p.tile_slots * c.kv_heads * kTileRows * (D + 2) * sizeof(float));
  }
  p.total = total;
  return p;
}

namespace {
// Checks of the shapes that the workspace depends on.
int attention_shape(const moe_w8a8_kv_cache *c, const moe_w8a8_batch *b, int32_t heads,
                    int64_t T) {
  if (T < 0 || T > kMaxRows || heads < 1) return MOE_W8A8_ERR_INVALID;
  MOE_TRY(cache_shape(c));
  MOE_TRY(batch_shape(b));
  if (!heads_ok(heads, c->head_dim) || heads % c->kv_heads) return MOE_W8A8_ERR_UNSUPPORTED;
  // query rows of a kv head are counted in 32 bits
  if (T * (heads / c->kv_heads) > 0x7fffffff - kTileRows) return MOE_W8A8_ERR_UNSUPPORTED;
  return MOE_W8A8_OK;
}
AttnPlan plan_of(const moe_w8a8_kv_cache &c, const moe_w8a8_batch &b, int32_t heads, int64_t T) {
  return attention_plan(view(c), c.head_dim, c.format, view(b, c.page_size, T), heads,
                        b.max_length);
}
}  // namespace

extern "C" size_t moe_w8a8_paged_attention_workspace_size(const moe_w8a8_kv_cache *c,
                                                          const moe_w8a8_batch *b, int32_t heads,
                                                          int64_t T) {
  if (attention_shape(c, b, heads, T) != MOE_W8A8_OK) return 0;
  if (T == 0 || b->num_seqs == 0 || b->max_tokens == 0) return 0;
  return plan_of(*c, *b, heads, T).total;
}

extern "C" int moe_w8a8_paged_attention(const moe_w8a8_attention_args *a,
                                        const moe_w8a8_kv_cache *c, const moe_w8a8_batch *b,
                                        int64_t T, void *workspace, size_t workspace_bytes,
                                        void *stream) {
  if (!a || a->window < 0 || !isfinite(a->scale)) return MOE_W8A8_ERR_INVALID;
  MOE_TRY(attention_shape(c, b, a->heads, T));
  MOE_TRY(cache_check(c));
  MOE_TRY(batch_check(b));
  if (T == 0 || b->num_seqs == 0 || b->max_tokens == 0) return MOE_W8A8_OK;
  const int D = c->head_dim;
  const int64_t width = (int64_t)a->heads * D;
  if (!a->q || !a->out || !al(a->q, 2) || !al(a->out, 2) || !pitch_ok(a->ld_q, width) ||
      !pitch_ok(a->ld_out, width))
    return MOE_W8A8_ERR_INVALID;
  const Mat out = mat(a->out, T, a->ld_out, width, 2);
  const AttnPlan p = plan_of(*c, *b, a->heads, T);
  const Mat ws = flat(workspace, p.total), q = mat(a->q, T, a->ld_q, width, 2);
  if (!al(workspace, 256) || overlap(out, q) || overlap(ws, q) || overlap(ws, out))
    return MOE_W8A8_ERR_INVALID;
  const Buffers bf = buffers(*c, *b);
  for (const Mat &m : bf.m)
    if (overlap(out, m) || overlap(ws, m)) return MOE_W8A8_ERR_INVALID;
  if (p.total > 0 && (!workspace || workspace_bytes < p.total)) return MOE_W8A8_ERR_WORKSPACE;
  AttnArgs r{};
  r.q = a->q; r.ld_q = a->ld_q; r.out = a->out; r.ld_out = a->ld_out;
  r.heads = a->heads; r.group = a->heads / c->kv_heads; r.causal = a->causal != 0;
  r.window = a->window; r.scale2 = a->scale * 1.44269504088896340736f;
  r.few_rows = p.few_rows;
  const CacheView cv = view(*c);
  const BatchView bv = view(*b, c->page_size, T);
  if (p.tiles)
    MOE_CHECK(launch_attention_tiles(r, cv, D, c->format, bv, p, (float *)workspace,
                                     (hipStream_t)stream));
  if (p.few_rows > 0)
    MOE_CHECK(launch_attention_rows(r, cv, D, c->format, bv, p, (float *)workspace,
                                    (hipStream_t)stream));
  MOE_CHECK(launch_attention_join(r, cv, D, bv, p, (float *)workspace, (hipStream_t)stream));
  return MOE_W8A8_OK;
}

extern "C" size_t moe_w8a8_token_logprobs_workspace_size(int32_t V, int32_t top, int64_t T) {
  if (V < 1 || V > kMaxVocab || top < 0 || top > kMaxTop || top > V || T < 1 || T > kMaxRows)
    return 0;
  return up256(token_logprobs_workspace(V, top, T));
}

extern "C" int moe_w8a8_token_logprobs(const moe_w8a8_logprobs_args *a, int64_t T,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  if (!a || T < 0 || T > kMaxRows || a->vocab < 1 || a->top < 0 || a->top > a->vocab ||
      !type_ok(a->type))
    return MOE_W8A8_ERR_INVALID;
  if (a->vocab > kMaxVocab || a->top > kMaxTop) return MOE_W8A8_ERR_UNSUPPORTED;
  if (T == 0) return MOE_W8A8_OK;
  const int64_t V = a->vocab;
  const size_t size = a->type == MOE_W8A8_F32 ? 4 : 2;
  if (!a->logits || !al(a->logits, size) || !pitch_ok(a->ld, V) ||
      (a->tokens == nullptr) != (a->logprobs == nullptr) ||
      (a->top > 0) != (a->top_tokens != nullptr) || (a->top > 0) != (a->top_logprobs != nullptr) ||
      (!a->logprobs && !a->entropy && a->top == 0))
    return MOE_W8A8_ERR_INVALID;
  if (!al(a->tokens, 8) || !al(a->logprobs, 4) || !al(a->entropy, 4) || !al(a->top_tokens, 8) ||
      !al(a->top_logprobs, 4))
    return MOE_W8A8_ERR_INVALID;
  const Mat ins[2] = {mat(a->logits, T, a->ld, V, size), flat(a->tokens, (size_t)T * 8)};
  const Mat outs[4] = {flat(a->logprobs, (size_t)T * 4), flat(a->entropy, (size_t)T * 4),
                       flat(a->top_tokens, (size_t)T * a->top * 8),
                       flat(a->top_logprobs, (size_t)T * a->top * 4)};
  for (int i = 0; i < 4; ++i) {
    if (overlap(outs[i], ins[0]) || overlap(outs[i], ins[1])) return MOE_W8A8_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return MOE_W8A8_ERR_INVALID;
  }
  const size_t need = moe_w8a8_token_logprobs_workspace_size(a->vocab, a->top, T);
  const Mat ws = flat(workspace, need);
  if (!al(workspace, 256) || overlap(ws, ins[0]) || overlap(ws, ins[1])) return MOE_W8A8_ERR_INVALID;
  for (const Mat &o : outs)
    if (overlap(ws, o)) return MOE_W8A8_ERR_INVALID;
  if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_W8A8_ERR_WORKSPACE;
  LogprobArgs r{};
  r.x = a->logits; r.ld = a->ld; r.tokens = a->tokens; r.logprobs = a->logprobs;
  r.entropy = a->entropy; r.top_tokens = a->top_tokens; r.top_logprobs = a->top_logprobs;
  r.V = a->vocab; r.top = a->top;
  MOE_CHECK(launch_token_logprobs(r, a->type == MOE_W8A8_F32, T, workspace,
                                  (hipStream_t)stream));
  return MOE_W8A8_OK;
}
