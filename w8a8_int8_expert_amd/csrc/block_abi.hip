// block_abi.hip -- host side of the block operators of include/moe_w8a8.h:
// argument validation before anything touches HIP, workspace carving and the
// launch sequence on the caller's stream.
#include <math.h>

#include "block_internal.h"

using namespace moe;

namespace {

constexpr int64_t kMaxRows = ((int64_t)1 << 22) - 1;  // a launch counts rows x threads in 32 bits
// Rows a distance of ld elements apart stay addressable (2^48 elements in all).
constexpr int64_t kMaxPitch = (int64_t)1 << 26;

bool al(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
bool width_ok(int64_t k) { return k >= 1 && k <= kMaxWidth; }
bool outputs_ok(int64_t n) { return n >= 1 && n <= kMaxOutputs; }
bool format_ok(int32_t f) { return f == MOE_W8A8_FORMAT_INT8 || f == MOE_W8A8_FORMAT_FP8; }
bool type_ok(int32_t t) { return t == MOE_W8A8_BF16 || t == MOE_W8A8_F32; }
bool pitch_ok(int64_t ld, int64_t width) { return ld >= width && ld <= kMaxPitch; }
// A strided matrix in memory: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Mat {
  const void *p;
  size_t rows, pitch, width;
};
Mat mat(const void *p, int64_t rows, int64_t ld, int64_t width, size_t size) {
  return Mat{rows > 0 ? p : nullptr, (size_t)rows, (size_t)ld * size, (size_t)width * size};
}
Mat flat(const void *p, size_t bytes) { return Mat{bytes ? p : nullptr, 1, bytes, bytes}; }
// Whether two matrices may share a byte. Column blocks of one buffer (the same
// pitch) are told apart by their columns; anything else by the ranges they span.
bool overlap(const Mat &a, const Mat &b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x >= y + (b.rows - 1) * b.pitch + b.width || y >= x + (a.rows - 1) * a.pitch + a.width)
    return false;
  if (a.pitch != b.pitch) return true;
  const size_t d = y >= x ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
  return d < a.width || d + b.width > a.pitch;
}

// Structural checks of weights (shape, format, pointers); sizes separately.
int weights_check(const moe_w8a8_linear_weights *w) {
  if (!w || w->in_features <= 0 || w->out_features <= 0) return MOE_W8A8_ERR_INVALID;
  if (w->gated != 0 && w->gated != 1) return MOE_W8A8_ERR_INVALID;
  if (w->gated && (w->out_features % 2 != 0 || w->bias)) return MOE_W8A8_ERR_INVALID;
  if (!format_ok(w->format) || !w->w || !w->scale) return MOE_W8A8_ERR_INVALID;
  if (!al(w->w, 16) || !al(w->scale, 4) || !al(w->inv_smooth, 4) || !al(w->bias, 4))
    return MOE_W8A8_ERR_INVALID;
  if (!width_ok(w->in_features) || !outputs_ok(w->out_features)) return MOE_W8A8_ERR_UNSUPPORTED;
  return MOE_W8A8_OK;
}
// Whether m shares a byte with packed codes or scales; with anything of the weights.
bool over_weights(const moe_w8a8_linear_weights &w, const Mat &m) {
  const size_t rows = (size_t)packed_rows(w.out_features, w.gated != 0);
  return overlap(m, flat(w.w, rows * row_pitch(w.in_features))) ||
         overlap(m, flat(w.scale, rows * 4));
}
bool over_any(const moe_w8a8_linear_weights &w, const Mat &m) {
  return over_weights(w, m) || overlap(m, flat(w.inv_smooth, (size_t)w.in_features * 4)) ||
         overlap(m, flat(w.bias, (size_t)w.out_features * 4));
}
int act_check(const moe_w8a8_act *a, int64_t K) {
  if (!a) return MOE_W8A8_ERR_INVALID;
  const bool x = a->x != nullptr, q = a->q != nullptr || a->s != nullptr;
  if (x == q || (q && (!a->q || !a->s))) return MOE_W8A8_ERR_INVALID;
  if (x && (!al(a->x, 2) || !pitch_ok(a->ld_x, K))) return MOE_W8A8_ERR_INVALID;
  if (q && (!al(a->q, 16) || !al(a->s, 4))) return MOE_W8A8_ERR_INVALID;
  return MOE_W8A8_OK;
}
Mat act_mat(const moe_w8a8_act *a, int64_t T, int K) {
  return a->x ? mat(a->x, T, a->ld_x, K, 2) : mat(a->q, T, row_pitch(K), row_pitch(K), 1);
}
int result_check(const moe_w8a8_result *r, const moe_w8a8_act *act, int64_t T,
                 const moe_w8a8_linear_weights &in, const moe_w8a8_linear_weights &last) {
  const int K = in.in_features;
  const int64_t N = last.out_features;
  if (!r || !r->out || !type_ok(r->out_type)) return MOE_W8A8_ERR_INVALID;
  const size_t size = r->out_type == MOE_W8A8_F32 ? 4 : 2;
  if (!al(r->out, size) || !pitch_ok(r->ld_out, N) || !al(r->gate, 4)) return MOE_W8A8_ERR_INVALID;
  const Mat out = mat(r->out, T, r->ld_out, N, size);
  if (r->add) {
    if (!al(r->add, 2) || !pitch_ok(r->ld_add, N)) return MOE_W8A8_ERR_INVALID;
    const bool same = r->add == r->out && r->out_type == MOE_W8A8_BF16 && r->ld_add == r->ld_out;
    if (!same && overlap(out, mat(r->add, T, r->ld_add, N, 2))) return MOE_W8A8_ERR_INVALID;
  }
  if (overlap(out, act_mat(act, T, K)) || overlap(out, flat(act->s, (size_t)T * 4)) ||
      overlap(out, flat(r->gate, (size_t)T * 4)) || over_any(in, out) ||
      (&last != &in && over_any(last, out)))
    return MOE_W8A8_ERR_INVALID;
  return MOE_W8A8_OK;
}
Epilogue epilogue(const moe_w8a8_linear_weights &w, const moe_w8a8_result &r) {
  Epilogue e{};
  e.scale = w.scale; e.bias = w.bias; e.N = w.out_features;
  e.out = r.out; e.ld_out = r.ld_out; e.out_f32 = r.out_type == MOE_W8A8_F32;
  e.gate = r.gate; e.add = r.add; e.ld_add = r.ld_add;
  return e;
}

// Room for codes of T rows, row-major or in tiles.
size_t codes_bytes(int64_t T, int K) { return (size_t)((T + 15) / 16 * 16) * row_pitch(K); }

struct LinearLayout {
  size_t q, s, partial, total;
};
LinearLayout linear_layout(int K, int64_t T) {
  LinearLayout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
  if (T == 0 || fused_tokens(T, K)) return L;
  L.q = take(codes_bytes(T, K));
  L.s = take((size_t)T * 4);
  L.partial = take(T > kAlwaysStream ? kPartialBytes : 0);
  L.total = o;
  return L;
}
// h holds gate and up values (of a streaming product: fp32 [T][packed rows]) or
// hidden values (fp32 [T][Fp]).
struct FfnLayout {
  size_t q, s, h, amax, qh, sh, partial, total;
};
FfnLayout ffn_layout(int H, int F, int64_t T) {
  FfnLayout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += up256(bytes); return at; };
  if (T == 0) return L;
  // (the larger of the two for few rows: a workspace never shrinks as T grows)
  const int64_t few = T < kStreamRows ? T : kStreamRows;
  const size_t gu = (size_t)few * packed_rows(2 * F, true) * 4;
  const size_t hid = (size_t)T * row_pitch(F) * 4;
  L.h = take(gu > hid ? gu : hid);
  if (!fused_tokens(T, H)) {
    L.q = take(codes_bytes(T, H));
    L.s = take((size_t)T * 4);
  }
  if (!fused_hidden(T, F)) {
    L.amax = take((size_t)T * 4);
    L.qh = take(codes_bytes(T, F));
    L.sh = take((size_t)T * 4);
  }
  L.partial = take(T > kAlwaysStream ? kPartialBytes : 0);
  L.total = o;
  return L;
}

hipError_t product(const StreamIn &in, const int8_t *q, int64_t T,
                   const moe_w8a8_linear_weights &w, const Epilogue &ep, void *partial,
                   hipStream_t st) {
  const bool gated = w.gated != 0, fp8 = w.format == MOE_W8A8_FORMAT_FP8;
  const int K = w.in_features, Np = packed_rows(w.out_features, gated);
  if (streams(T, K, Np))
    return launch_linear_stream(in, (int)T, w.w, K, Np, fp8, ep, st);
  return launch_linear_tiled(q, T, w.w, K, Np, gated, fp8, ep, partial, st);
}

}  // namespace

#define MOE_CHECK(expr)                                \
  do {                                                 \
    if ((expr) != hipSuccess) return MOE_W8A8_ERR_HIP; \
  } while (0)
#define MOE_TRY(expr)              \
  do {                             \
    const int rc_ = (expr);        \
    if (rc_ != MOE_W8A8_OK) return rc_; \
  } while (0)

extern "C" int64_t moe_w8a8_row_pitch(int32_t K) { return width_ok(K) ? row_pitch(K) : 0; }

extern "C" size_t moe_w8a8_linear_codes_bytes(int32_t N, int32_t K, int32_t gated) {
  if (!width_ok(K) || !outputs_ok(N) || (gated && N % 2)) return 0;
  return (size_t)packed_rows(N, gated != 0) * row_pitch(K);
}
extern "C" int64_t moe_w8a8_linear_scales(int32_t N, int32_t gated) {
  if (!outputs_ok(N) || (gated && N % 2)) return 0;
  return packed_rows(N, gated != 0);
}

extern "C" int moe_w8a8_linear_quantise(const moe_w8a8_linear_weights *out, const void *src,
                                        int32_t src_type, int64_t ld_src, const float *smooth,
                                        void *stream) {
  MOE_TRY(weights_check(out));
  if (!src || !type_ok(src_type) || !al(src, src_type == MOE_W8A8_F32 ? 4 : 2) ||
      !al(smooth, 4) || !pitch_ok(ld_src, out->in_features))
    return MOE_W8A8_ERR_INVALID;
  if (over_weights(*out, mat(src, out->out_features, ld_src, out->in_features,
                             src_type == MOE_W8A8_F32 ? 4 : 2)) ||
      over_weights(*out, flat(smooth, (size_t)out->in_features * 4)))
    return MOE_W8A8_ERR_INVALID;
  MOE_CHECK(launch_pack_rows(*out, src, src_type, ld_src, smooth, nullptr, (hipStream_t)stream));
  return MOE_W8A8_OK;
}

extern "C" int moe_w8a8_linear_pack(const moe_w8a8_linear_weights *out, const int8_t *src,
                                    int64_t ld_src, const float *src_scale, void *stream) {
  MOE_TRY(weights_check(out));
  if (!src || !src_scale || !al(src_scale, 4) || !pitch_ok(ld_src, out->in_features))
    return MOE_W8A8_ERR_INVALID;
  if (over_weights(*out, mat(src, out->out_features, ld_src, out->in_features, 1)) ||
      over_weights(*out, flat(src_scale, (size_t)out->out_features * 4)))
    return MOE_W8A8_ERR_INVALID;
  MOE_CHECK(launch_pack_rows(*out, src, -1, ld_src, nullptr, src_scale, (hipStream_t)stream));
  return MOE_W8A8_OK;
}

extern "C" int moe_w8a8_act_quant(int32_t K, int32_t format, const uint16_t *x, int64_t ld_x,
                                  int64_t T, const float *inv_smooth, int8_t *q, float *s,
                                  void *stream) {
  if (K <= 0 || !format_ok(format) || T < 0 || T > kMaxRows) return MOE_W8A8_ERR_INVALID;
  if (!width_ok(K)) return MOE_W8A8_ERR_UNSUPPORTED;
  if (T == 0) return MOE_W8A8_OK;
  if (!x || !q || !s || !al(x, 2) || !al(inv_smooth, 4) || !al(q, 16) || !al(s, 4) ||
      !pitch_ok(ld_x, K))
    return MOE_W8A8_ERR_INVALID;
  const Mat xm = mat(x, T, ld_x, K, 2), qm = flat(q, (size_t)T * row_pitch(K)),
            sm = flat(s, (size_t)T * 4);
  const Mat im = flat(inv_smooth, (size_t)K * 4);
  if (overlap(xm, qm) || overlap(xm, sm) || overlap(qm, sm) || overlap(im, qm) || overlap(im, sm))
    return MOE_W8A8_ERR_INVALID;
  MOE_CHECK(launch_act_rows(x, ld_x, T, K, inv_smooth, format == MOE_W8A8_FORMAT_FP8, false, q, s,
                            nullptr, (hipStream_t)stream));
  return MOE_W8A8_OK;
}

extern "C" size_t moe_w8a8_linear_workspace_size(int32_t N, int32_t K, int64_t T) {
  if (!width_ok(K) || !outputs_ok(N) || T < 0 || T > kMaxRows) return 0;
  return linear_layout(K, T).total;
}

extern "C" int moe_w8a8_linear(const moe_w8a8_linear_weights *w, const moe_w8a8_act *act,
                               int64_t T, const moe_w8a8_result *res, void *workspace,
                               size_t workspace_bytes, void *stream) {
  if (T < 0 || T > kMaxRows) return MOE_W8A8_ERR_INVALID;
  MOE_TRY(weights_check(w));
  if (w->gated) return MOE_W8A8_ERR_INVALID;
  if (T == 0) return MOE_W8A8_OK;
  const int K = w->in_features;
  MOE_TRY(act_check(act, K));
  MOE_TRY(result_check(res, act, T, *w, *w));
  const LinearLayout L = linear_layout(K, T);
  if (!al(workspace, 256)) return MOE_W8A8_ERR_INVALID;
  if (L.total > 0 && (!workspace || workspace_bytes < L.total)) return MOE_W8A8_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  char *ws = (char *)workspace;
  Epilogue ep = epilogue(*w, *res);
  StreamIn in{};
  if (act->x && fused_tokens(T, K)) {
    in.x = act->x; in.ld = act->ld_x; in.inv = w->inv_smooth;
  } else if (act->x) {
    int8_t *q = (int8_t *)(ws + L.q);
    float *s = (float *)(ws + L.s);
    in.q = q; ep.row_scale = s;
    in.tiles = streams(T, K, packed_rows(w->out_features, false));
    MOE_CHECK(launch_act_rows(act->x, act->ld_x, T, K, w->inv_smooth,
                              w->format == MOE_W8A8_FORMAT_FP8, in.tiles, q, s, nullptr, st));
  } else {
    in.q = act->q; ep.row_scale = act->s;
  }
  MOE_CHECK(product(in, in.q, T, *w, ep, ws + L.partial, st));
  return MOE_W8A8_OK;
}

extern "C" size_t moe_w8a8_ffn_workspace_size(int32_t H, int32_t F, int32_t N, int64_t T) {
  if (!width_ok(H) || !width_ok(F) || !outputs_ok(N) || T < 0 || T > kMaxRows) return 0;
  return ffn_layout(H, F, T).total;
}

extern "C" int moe_w8a8_ffn(const moe_w8a8_linear_weights *gu, const moe_w8a8_linear_weights *dn,
                            const moe_w8a8_act *act, int64_t T, const moe_w8a8_result *res,
                            void *workspace, size_t workspace_bytes, void *stream) {
  if (T < 0 || T > kMaxRows) return MOE_W8A8_ERR_INVALID;
  MOE_TRY(weights_check(gu));
  MOE_TRY(weights_check(dn));
  if (!gu->gated || dn->gated || gu->out_features / 2 != dn->in_features ||
      gu->format != dn->format || dn->inv_smooth)
    return MOE_W8A8_ERR_INVALID;
  if (T == 0) return MOE_W8A8_OK;
  const int H = gu->in_features, F = dn->in_features;
  MOE_TRY(act_check(act, H));
  MOE_TRY(result_check(res, act, T, *gu, *dn));
  const FfnLayout L = ffn_layout(H, F, T);
  if (!al(workspace, 256)) return MOE_W8A8_ERR_INVALID;
  if (!workspace || workspace_bytes < L.total) return MOE_W8A8_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  const bool fp8 = gu->format == MOE_W8A8_FORMAT_FP8;
  char *ws = (char *)workspace;
  float *h = (float *)(ws + L.h);
  uint32_t *amax = (uint32_t *)(ws + L.amax);
  // Few tokens stream; of more, the first product applies SwiGLU and takes row maxima.
  const bool few = streams(T, H, packed_rows(2 * F, true));

  Epilogue ep{};
  ep.scale = gu->scale; ep.out = h; ep.out_f32 = 1;
  const int Np = packed_rows(2 * F, true);
  ep.N = few ? Np : F;
  ep.ld_out = few ? Np : row_pitch(F);
  ep.amax = amax;
  StreamIn in{};
  if (act->x && fused_tokens(T, H)) {
    in.x = act->x; in.ld = act->ld_x; in.inv = gu->inv_smooth;
  } else if (act->x) {
    int8_t *q = (int8_t *)(ws + L.q);
    float *s = (float *)(ws + L.s);
    in.tiles = few;
    MOE_CHECK(launch_act_rows(act->x, act->ld_x, T, H, gu->inv_smooth, fp8, few, q, s,
                              few ? nullptr : amax, st));
    in.q = q; ep.row_scale = s;
  } else {
    in.q = act->q; ep.row_scale = act->s;
    if (!few) MOE_CHECK(launch_clear(amax, T, st));
  }
  MOE_CHECK(product(in, in.q, T, *gu, ep, ws + L.partial, st));

  Epilogue ed = epilogue(*dn, *res);
  StreamIn hin{};
  if (fused_hidden(T, F)) {
    hin.h = h; hin.ld = Np;
  } else {
    int8_t *qh = (int8_t *)(ws + L.qh);
    float *sh = (float *)(ws + L.sh);
    if (few) {
      hin.tiles = streams(T, F, packed_rows(dn->out_features, false));
      MOE_CHECK(launch_hidden_rows(h, Np, T, F, fp8, hin.tiles, qh, sh, st));
    } else {
      MOE_CHECK(launch_requant_rows(h, amax, T, F, fp8, qh, sh, st));
    }
    hin.q = qh; ed.row_scale = sh;
  }
  MOE_CHECK(product(hin, hin.q, T, *dn, ed, ws + L.partial, st));
  return MOE_W8A8_OK;
}

extern "C" int moe_w8a8_add_norm(const moe_w8a8_add_norm_args *a, int64_t T, void *stream) {
  if (!a || T < 0 || T > kMaxRows || a->hidden <= 0) return MOE_W8A8_ERR_INVALID;
  auto kind_ok = [](int32_t k, const float *w, const float *b) {
    if (k == MOE_W8A8_NORM_NONE) return !w && !b;
    return k == MOE_W8A8_NORM_RMS || k == MOE_W8A8_NORM_LAYER;
  };
  if (!kind_ok(a->pre_norm, a->pre_weight, a->pre_bias) ||
      !kind_ok(a->post_norm, a->post_weight, a->post_bias) || !type_ok(a->residual_type) ||
      !format_ok(a->format) || !isfinite(a->eps) || a->eps < 0.0f ||
      !isfinite(a->residual_scale) || !isfinite(a->block_scale))
    return MOE_W8A8_ERR_INVALID;
  const int64_t H = a->hidden;
  if (!width_ok(H)) return MOE_W8A8_ERR_UNSUPPORTED;
  if (T == 0) return MOE_W8A8_OK;
  const size_t rsize = a->residual_type == MOE_W8A8_F32 ? 4 : 2;
  if (!a->y || !al(a->y, 2) || !pitch_ok(a->ld_y, H)) return MOE_W8A8_ERR_INVALID;
  if ((a->q == nullptr) != (a->s == nullptr) || (!a->residual_out && !a->normed && !a->q))
    return MOE_W8A8_ERR_INVALID;
  if (a->gate_token && a->gate_rows) return MOE_W8A8_ERR_INVALID;
  if ((a->residual && !(al(a->residual, rsize) && pitch_ok(a->ld_residual, H))) ||
      (a->residual_out && !(al(a->residual_out, rsize) && pitch_ok(a->ld_residual_out, H))) ||
      (a->normed && !(al(a->normed, 2) && pitch_ok(a->ld_normed, H))) ||
      (a->gate_rows && !(al(a->gate_rows, 2) && pitch_ok(a->ld_gate, H) && a->gate_group > 0)) ||
      !al(a->post_weight, 4) || !al(a->post_bias, 4) || !al(a->pre_weight, 4) ||
      !al(a->pre_bias, 4) || !al(a->gate_token, 4) || !al(a->inv_smooth, 4) || !al(a->q, 16) ||
      !al(a->s, 4))
    return MOE_W8A8_ERR_INVALID;
  // Outputs overlap nothing but what the header allows.
  const int64_t groups = a->gate_rows ? (T - 1) / a->gate_group + 1 : 0;
  const size_t vec = (size_t)H * 4, col = (size_t)T * 4;
  const Mat outs[4] = {mat(a->residual_out, T, a->ld_residual_out, H, rsize),
                       mat(a->normed, T, a->ld_normed, H, 2),
                       flat(a->q, (size_t)T * row_pitch((int)H)), flat(a->s, col)};
  const Mat ins[9] = {mat(a->y, T, a->ld_y, H, 2), mat(a->residual, T, a->ld_residual, H, rsize),
                      mat(a->gate_rows, groups, a->ld_gate, H, 2), flat(a->gate_token, col),
                      flat(a->post_weight, vec), flat(a->post_bias, vec),
                      flat(a->pre_weight, vec), flat(a->pre_bias, vec),
                      flat(a->inv_smooth, vec)};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 9; ++i) {
      const bool in_place =
          (o == 0 && i == 1 && a->residual_out == a->residual &&
           a->ld_residual_out == a->ld_residual) ||
          (o == 1 && i == 0 && a->normed == a->y && a->ld_normed == a->ld_y);
      if (!in_place && overlap(outs[o], ins[i]))
        return MOE_W8A8_ERR_INVALID;
    }
    for (int p = 0; p < o; ++p)
      if (overlap(outs[o], outs[p])) return MOE_W8A8_ERR_INVALID;
  }
  MOE_CHECK(launch_add_norm(*a, T, (hipStream_t)stream));
  return MOE_W8A8_OK;
}
