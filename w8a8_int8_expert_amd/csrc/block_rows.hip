// block_rows.hip -- the row operators of the decoder block: per-token codes,
// the norms around a block, requantisation of the feed-forward's hidden rows,
// and the layout of weights.
//
// "MiniMax-M3 W8A8 inference on K100AI" (mhpq.cn/news/1068415) §3.2 (per-token
// activations, per-channel weights, SmoothQuant) and §4.3 (stay in 8 bits
// between matmuls; convert where a norm or residual needs it).
#include "row_device.h"

namespace moe {
namespace {

// A row is held by TPR threads, NC chunks of eight consecutive elements each:
// thread i has chunks i, i + TPR, ... Every element is read once and stays in
// registers between the reductions, so a row costs its own bytes and nothing
// else. TPR = 64: four rows per 256-thread block, reductions inside one
// wavefront; otherwise a block per row, reductions through LDS.
template <int TPR>
struct RowGroup {
  static constexpr int kWaves = TPR / 64;
  static constexpr int kRows = TPR == 64 ? 4 : 1;
  static constexpr int kThreads = TPR * kRows;
  // `slot`: a cell row of its own for each reduction of a kernel, so that one
  // barrier per reduction is enough.
  static __device__ __forceinline__ float sum(float v, float *slot) {
    v = wave_sum_f32(v);
    if constexpr (kWaves > 1) {
      if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
      __syncthreads();
      v = slot[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += slot[w];
    }
    return v;
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t m, float *slot) {
    m = wave_max_bits(m);
    if constexpr (kWaves > 1) {
      uint32_t *s = reinterpret_cast<uint32_t *>(slot);
      if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = m;
      __syncthreads();
      m = s[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) m = umax(m, s[w]);
    }
    return m;
  }
};

// Codes of row t, whose scaled values v are in registers; columns past the
// width hold zeros and give zero codes, up to the pitch Kp.
template <int TPR, int NC>
__device__ __forceinline__ void emit_codes(const float (&v)[NC][8], int lane, int64_t t, int Kp,
                                           uint32_t amax, bool fp8, bool tiles, int8_t *q,
                                           float *s) {
  const RowCode rc = row_code(amax, fp8);
  if (lane == 0) s[t] = rc.scale;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * 8;
    if (c < Kp)
      *reinterpret_cast<v2i *>(q + code_at(tiles, t, c, Kp)) =
          v2i{(int)row_codes4(v[i], rc, fp8), (int)row_codes4(v[i] + 4, rc, fp8)};
  }
}

template <int TPR, int NC, bool kOdd>
__global__ __launch_bounds__(RowGroup<TPR>::kThreads) void act_rows_kernel(
    const uint16_t *__restrict__ x, int64_t ld, int64_t T, int K, const float *__restrict__ inv,
    bool fp8, bool tiles, int8_t *__restrict__ q, float *__restrict__ s,
    uint32_t *__restrict__ clear) {
  typedef RowGroup<TPR> G;
  __shared__ float cells[G::kWaves];
  const int lane = threadIdx.x % TPR;
  const int64_t t = (int64_t)blockIdx.x * G::kRows + threadIdx.x / TPR;
  if (t >= T) return;  // whole wavefronts; a block of one row never has t >= T
  v4i raw[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) raw[i] = fetch8<kOdd>(x + t * ld, (lane + i * TPR) * 8, K);
  float v[NC][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * 8;
    unpack8<kOdd>(raw[i], c, K, v[i]);
    if (inv) {
      float f[8];
      load8<kOdd>(inv, c, K, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(v[i][j]));
  }
  m = G::max_bits(m, cells);
  if (clear && lane == 0) clear[t] = 0u;
  emit_codes<TPR, NC>(v, lane, t, row_pitch(K), m, fp8, tiles, q, s);
}

// Codes of the hidden rows of a streaming gate/up product.
template <int TPR, int NC>
__global__ __launch_bounds__(RowGroup<TPR>::kThreads) void hidden_rows_kernel(
    const float *__restrict__ gu, int64_t ld, int64_t T, int F, bool fp8, bool tiles,
    int8_t *__restrict__ q, float *__restrict__ s) {
  typedef RowGroup<TPR> G;
  __shared__ float cells[G::kWaves];
  const int lane = threadIdx.x % TPR;
  const int64_t t = (int64_t)blockIdx.x * G::kRows + threadIdx.x / TPR;
  if (t >= T) return;  // as in act_rows_kernel
  float v[NC][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * 8;
    hidden8(gu + t * ld, c, F - c, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(v[i][j]));
  }
  m = G::max_bits(m, cells);
  emit_codes<TPR, NC>(v, lane, t, row_pitch(F), m, fp8, tiles, q, s);
}

__global__ __launch_bounds__(256) void clear_kernel(uint32_t *__restrict__ p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0u;
}

// ----------------------------------------------------------------- add_norm
// v = norm(v) for the row in v (elements past H are zero, and stay zero but for a
// bias). Four cell rows; a second use of one lies behind the barrier of another.
template <int TPR, int NC, bool kOdd>
__device__ __forceinline__ void norm_row(float (&v)[NC][8], int kind, const float *w,
                                         const float *b, int H, float eps, int lane,
                                         float *cells) {
  typedef RowGroup<TPR> G;
  if (kind == MOE_W8A8_NORM_NONE) return;
  const float width = (float)H;
  const bool layer = kind == MOE_W8A8_NORM_LAYER;
  // (the mean as a sum of quotients: it stays in range where the sum would not)
  auto mean_of = [&](float *slot) {
    const float inv = 1.0f / width;
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) a = __builtin_fmaf(v[i][j], inv, a);
    return G::sum(a, slot);
  };
  auto centre = [&](float mean) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[i][j] = (lane + i * TPR) * 8 + j < H ? v[i][j] - mean : 0.0f;
  };
  auto squares = [&](float *slot) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) a = __builtin_fmaf(v[i][j], v[i][j], a);
    return G::sum(a, slot) / width;
  };
  // Rows at the ends of the fp32 range are scaled by a power of two, exactly but for
  // what is too small to matter, and eps with the square of it (an eps stays one:
  // zeros keep their norm). Down by 2^80: 65536 squares of 2^49 (a difference from
  // the mean at most) stay below 2^114.
  auto scale = [&](float f) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= f;
    if (eps > 0.0f) eps = __builtin_fmaxf(eps * f * f, 0x1p-126f);
  };
  float mean = layer ? mean_of(cells) : 0.0f;
  const bool far = __builtin_fabsf(mean) > 0x1p100f;  // a difference may pass the range
  if (far) {
    scale(0x1p-80f);
    mean = mean_of(cells + G::kWaves);
  }
  if (layer) centre(mean);
  float ms = squares(cells + 2 * G::kWaves);
  // Squares that leave the range: down as above, or, where they (and eps) lie below
  // 2^-90, up by 2^100. The mean is off by its rounding, which is no small part of a
  // row that spreads over less than 2^-10 of it, or lies that low: the mean of what
  // is left is taken off again.
  const bool large = !far && ms + eps > 0x1p127f, small = !far && ms + eps < 0x1p-90f;
  const bool again = layer && !large && (small || ms < mean * mean * 0x1p-20f);
  if (large || small || again) {
    if (large || small) scale(large ? 0x1p-80f : 0x1p100f);
    if (again) centre(mean_of(cells + 3 * G::kWaves));
    ms = squares(cells + G::kWaves);
  }
  const float rstd = 1.0f / __builtin_sqrtf(ms + eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
    if (w) {
      float f[8];
      load8<kOdd>(w, c, H, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
    }
    if (b) {
      float f[8];
      load8<kOdd>(b, c, H, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += f[j];
    }
  }
}

template <int TPR, int NC, bool kOdd>
__global__ __launch_bounds__(RowGroup<TPR>::kThreads) void add_norm_kernel(
    const moe_w8a8_add_norm_args a, int64_t T) {
  typedef RowGroup<TPR> G;
  __shared__ float cells[9][G::kWaves];
  const int lane = threadIdx.x % TPR;
  const int64_t t = (int64_t)blockIdx.x * G::kRows + threadIdx.x / TPR;
  if (t >= T) return;  // as in act_rows_kernel
  const int H = a.hidden;
  float v[NC][8], r[NC][8];
  v4i raw[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) raw[i] = fetch8<kOdd>(a.y + t * a.ld_y, (lane + i * TPR) * 8, H);
  // The residual is read before the reductions of the post norm, which would
  // otherwise hold its loads back.
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (lane + i * TPR) * 8;
      if (a.residual_type == MOE_W8A8_F32)
        load8<kOdd>(static_cast<const float *>(a.residual) + t * a.ld_residual, c, H, r[i]);
      else
        load8<kOdd>(static_cast<const uint16_t *>(a.residual) + t * a.ld_residual, c, H, r[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) unpack8<kOdd>(raw[i], (lane + i * TPR) * 8, H, v[i]);
  norm_row<TPR, NC, kOdd>(v, a.post_norm, a.post_weight, a.post_bias, H, a.eps, lane, cells[0]);
  const float bs = a.block_scale * (a.gate_token ? a.gate_token[t] : 1.0f);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * 8;
    if (a.gate_rows) {
      float g[8];
      load8<kOdd>(a.gate_rows + t / a.gate_group * a.ld_gate, c, H, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] *= bs;
      if (a.residual) v[i][j] = __builtin_fmaf(a.residual_scale, r[i][j], v[i][j]);
    }
    if (a.residual_out) {
      if (a.residual_type == MOE_W8A8_F32)
        store8<kOdd>(static_cast<float *>(a.residual_out) + t * a.ld_residual_out, c, H, v[i]);
      else
        store8<kOdd>(static_cast<uint16_t *>(a.residual_out) + t * a.ld_residual_out, c, H, v[i]);
    }
  }
  if (!a.normed && !a.q) return;  // uniform over the grid
  norm_row<TPR, NC, kOdd>(v, a.pre_norm, a.pre_weight, a.pre_bias, H, a.eps, lane, cells[4]);
  if (a.normed) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      store8<kOdd>(a.normed + t * a.ld_normed, (lane + i * TPR) * 8, H, v[i]);
  }
  if (!a.q) return;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (lane + i * TPR) * 8, rem = H - c;
    if (a.inv_smooth) {
      float f[8];
      load8<kOdd>(a.inv_smooth, c, H, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
    }
    // A bias or a NaN row leaves values past the width; they are no values.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= rem) v[i][j] = 0.0f;
      m = umax(m, abs_bits(v[i][j]));
    }
  }
  m = G::max_bits(m, cells[8]);
  emit_codes<TPR, NC>(v, lane, t, row_pitch(H), m, a.format == MOE_W8A8_FORMAT_FP8, false, a.q,
                      a.s);
}

// ------------------------------------------------------------------- requant
// Thread = 16 consecutive columns of one row (one 16-byte store). h has the
// pitch of the codes; columns F..Fp-1 are not read and get zero codes.
__global__ __launch_bounds__(256) void requant_rows_kernel(const float *__restrict__ h,
                                                           const uint32_t *__restrict__ amax,
                                                           int64_t chunks, int F, bool fp8,
                                                           int8_t *__restrict__ q,
                                                           float *__restrict__ s) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const int Fp = row_pitch(F), per = Fp / 16;
  const int64_t t = i / per;
  const int c = (int)(i - t * per) * 16;
  const RowCode rc = row_code(amax[t], fp8);
  if (c == 0) s[t] = rc.scale;
  v4i o;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float v[4];
    if (c + 4 * k + 3 < F) {
      const v4f f = *reinterpret_cast<const v4f *>(h + t * Fp + c + 4 * k);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = f[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = c + 4 * k + j < F ? h[t * Fp + c + 4 * k + j] : 0.0f;
    }
    o[k] = (int)row_codes4(v, rc, fp8);
  }
  *reinterpret_cast<v4i *>(q + t * Fp + c) = o;
}

// ------------------------------------------------------------------- weights
// One wavefront per packed row (off the hot path: the source is read twice).
// Lane l makes the 16-byte chunks l, l + 64, ... of the row, zeros past K and
// in padding rows. kSrc: MOE_W8A8_F32, MOE_W8A8_BF16, or -1 (codes).
template <int kSrc>
__global__ __launch_bounds__(256) void pack_rows_kernel(const void *__restrict__ src, int64_t ld,
                                                        const float *__restrict__ smooth,
                                                        const float *__restrict__ src_scale, int N,
                                                        int K, int Np, bool gated, bool fp8,
                                                        int8_t *__restrict__ w,
                                                        float *__restrict__ scale) {
  const int lane = threadIdx.x & 63;
  const int p = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6);
  if (p >= Np) return;
  const int n = source_row(p, N, gated);
  const int Kp = row_pitch(K);
  auto value = [&](int k) -> float {
    float v;
    if constexpr (kSrc == MOE_W8A8_F32) v = static_cast<const float *>(src)[(int64_t)n * ld + k];
    else v = bf16_to_f32(static_cast<const uint16_t *>(src)[(int64_t)n * ld + k]);
    return smooth ? v * smooth[k] : v;
  };
  RowCode rc{1.0f, 0.0f, 0.0f, true};
  if constexpr (kSrc >= 0) {
    uint32_t m = 0;
    if (n >= 0)
      for (int k = lane; k < K; k += 64) m = umax(m, abs_bits(value(k)));
    rc = row_code(wave_max_bits(m), fp8);
  } else if (n >= 0) {
    rc.scale = src_scale[n];
  }
  if (lane == 0) scale[p] = n >= 0 ? rc.scale : 0.0f;
  for (int c = lane; c < Kp / 16; c += 64) {
    v4i o = {0, 0, 0, 0};
    if (n >= 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = c * 16 + 4 * i;
        if constexpr (kSrc >= 0) {
          float v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = k + j < K ? value(k + j) : 0.0f;
          o[i] = (int)row_codes4(v, rc, fp8);
        } else {
          uint32_t u = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (k + j < K)
              u |= (uint32_t)static_cast<const uint8_t *>(src)[(int64_t)n * ld + k + j] << (8 * j);
          o[i] = (int)u;
        }
      }
    }
    int8_t *d = w + frag_tile(p >> 4, c >> 2, Kp) + (((c & 3) << 4) + (p & 15)) * 16;
    *reinterpret_cast<v4i *>(d) = o;
  }
}

}  // namespace

// Threads per row and chunks per thread: a kernel<TPR, NC> holds rows of up to
// TPR * NC * 8 elements.
template <int TPR, int NC>
struct RowShape {
  static constexpr int kTpr = TPR, kNc = NC;
};
template <int TPR, typename K, typename... A>
static hipError_t launch_rows(K kernel, int64_t T, hipStream_t st, A... args) {
  typedef RowGroup<TPR> G;
  return launch_kernel(kernel, dim3((unsigned)((T + G::kRows - 1) / G::kRows)), dim3(G::kThreads),
                       st, Timing{}, args...);
}
// A thread per chunk up to 8192 columns: the shortest chain for a row alone (one
// row of 4096: 3.4 us, against 4.2 with two chunks a thread and 9.3 with one
// wavefront), and the most loads in flight for many (add_norm of 16384 rows of
// 4096, bf16: 95 us = 5.6 TB/s, against 100 and 127). Two or four rows per
// block, sharing the weights' loads, were no faster (98, 106).
template <typename F>
static hipError_t by_width(int width, F f) {
  if (width <= 512) return f(RowShape<64, 1>{});
  if (width <= 2048) return f(RowShape<256, 1>{});
  if (width <= 4096) return f(RowShape<512, 1>{});
  if (width <= 8192) return f(RowShape<1024, 1>{});
  if (width <= 32768) return f(RowShape<1024, 4>{});
  return f(RowShape<1024, 8>{});
}

hipError_t launch_act_rows(const uint16_t *x, int64_t ld, int64_t T, int K, const float *inv,
                           bool fp8, bool tiles, int8_t *q, float *s, uint32_t *clear,
                           hipStream_t st) {
  auto run = [&](auto shape) {
    constexpr int TPR = decltype(shape)::kTpr, NC = decltype(shape)::kNc;
    return launch_rows<TPR>(
        K % 8 ? act_rows_kernel<TPR, NC, true> : act_rows_kernel<TPR, NC, false>, T, st, x, ld, T,
        K, inv, fp8, tiles, q, s, clear);
  };
  // Many rows and one reduction: two chunks a thread, half the wavefronts that meet
  // (us, without and with smoothing scales: 16384 x 4096 34.6, 41.3 against 45.6,
  // 47.6; 8192 x 8192 33.8, 41.7 against 43.1, 48.6; 2100 x 4096 7.0, 8.5 against
  // 8.0, 8.6).
  if (T > 2048 && K > 2048 && K <= 4096) return run(RowShape<256, 2>{});
  if (T > 2048 && K > 4096 && K <= 8192) return run(RowShape<512, 2>{});
  return by_width(K, run);
}

hipError_t launch_hidden_rows(const float *gu, int64_t ld, int64_t T, int F, bool fp8, bool tiles,
                              int8_t *q, float *s, hipStream_t st) {
  return by_width(F, [&](auto shape) {
    constexpr int TPR = decltype(shape)::kTpr, NC = decltype(shape)::kNc;
    return launch_rows<TPR>(hidden_rows_kernel<TPR, NC>, T, st, gu, ld, T, F, fp8, tiles, q, s);
  });
}

hipError_t launch_add_norm(const moe_w8a8_add_norm_args &a, int64_t T, hipStream_t st) {
  return by_width(a.hidden, [&](auto shape) {
    constexpr int TPR = decltype(shape)::kTpr, NC = decltype(shape)::kNc;
    return launch_rows<TPR>(
        a.hidden % 8 ? add_norm_kernel<TPR, NC, true> : add_norm_kernel<TPR, NC, false>, T, st, a,
        T);
  });
}

hipError_t launch_clear(uint32_t *p, int64_t n, hipStream_t st) {
  return launch_kernel(clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), st, Timing{}, p,
                       n);
}

hipError_t launch_requant_rows(const float *h, const uint32_t *amax, int64_t T, int F, bool fp8,
                               int8_t *q, float *s, hipStream_t st) {
  const int64_t chunks = T * (row_pitch(F) / 16);
  return launch_kernel(requant_rows_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), st,
                       Timing{}, h, amax, chunks, F, fp8, q, s);
}

hipError_t launch_pack_rows(const moe_w8a8_linear_weights &w, const void *src, int src_type,
                            int64_t ld, const float *smooth, const float *src_scale,
                            hipStream_t st) {
  const int N = w.out_features, K = w.in_features;
  const bool gated = w.gated != 0, fp8 = w.format == MOE_W8A8_FORMAT_FP8;
  const int Np = packed_rows(N, gated);
  const dim3 grid((unsigned)((Np + 3) / 4));
  if (src_type == MOE_W8A8_F32)
    return launch_kernel(pack_rows_kernel<MOE_W8A8_F32>, grid, dim3(256), st, Timing{}, src, ld,
                         smooth, src_scale, N, K, Np, gated, fp8, w.w, w.scale);
  if (src_type == MOE_W8A8_BF16)
    return launch_kernel(pack_rows_kernel<MOE_W8A8_BF16>, grid, dim3(256), st, Timing{}, src, ld,
                         smooth, src_scale, N, K, Np, gated, fp8, w.w, w.scale);
  return launch_kernel(pack_rows_kernel<-1>, grid, dim3(256), st, Timing{}, src, ld, smooth,
                       src_scale, N, K, Np, gated, fp8, w.w, w.scale);
}

}  // namespace moe
