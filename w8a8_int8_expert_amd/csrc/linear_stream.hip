// linear_stream.hip -- W8A8 products of few tokens (T <= 64), bound by reading
// the weights once.
//
// "MiniMax-M3 W8A8 inference on K100AI" (mhpq.cn/news/1068415) §1.1, §1.3:
// decode is bound by reading weights, and W8A8 halves those bytes.
//
// A block of W wavefronts owns NPW panels of 16 output channels and splits K
// among its wavefronts in pairs of 64-k tiles (2 KB of a panel, contiguous),
// interleaved so that the block reads adjacent tiles at any moment. Weights go
// straight to registers as the A operand (nothing is read twice, so LDS would
// only add a copy); the tokens are the B operand, 16 per row tile. The W
// partial sums meet in LDS, and the wavefronts share the epilogue. INT8 sums
// are exact; FP8 sums are added in wavefront order.
//
// Up to four tokens the kernel codes the rows itself (kSrc 1: bf16 tokens, 2:
// fp32 hidden rows): every block does it over again, which costs less than a
// launch of its own, and the weights' first loads are in flight meanwhile.
#include "epilogue_device.h"

namespace moe {
namespace {

enum { kCodes, kTokens, kHidden };

struct StreamArgs {
  StreamIn in;
  int T, Kp, K;
  const int8_t *w;
  int Np;
  Epilogue ep;
};

template <bool kF8> struct Acc16v { typedef v4i T; };
template <> struct Acc16v<true> { typedef v4f T; };

template <int RT, int NPW, int W, int U, bool kF8, bool kGated, int kSrc>
__global__ __launch_bounds__(64 * W) void linear_stream_kernel(const StreamArgs a) {
  typedef typename Acc16v<kF8>::T Acc;
  static_assert(!kGated || NPW % 2 == 0, "gate and up panels come in pairs");
  static_assert(kSrc == kCodes || RT == 1, "rows coded by the block");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int pairs = a.Kp >> 7;

  // Panel of slot i. Gated: slots 0..NPW/2-1 are gate panels, the rest the
  // matching up panels (runs of two panels alternate in the packed order).
  auto panel = [&](int i) {
    if (kGated) {
      const int unit = blockIdx.x * (NPW / 2) + i % (NPW / 2);
      return unit / 2 * 4 + (i < NPW / 2 ? 0 : 2) + unit % 2;
    }
    return (int)blockIdx.x * NPW + i;
  };
  const int8_t *wp[NPW];
#pragma unroll
  for (int i = 0; i < NPW; ++i) {
    int p = panel(i);
    p = p < (a.Np >> 4) ? p : (a.Np >> 4) - 1;  // read, never stored
    wp[i] = a.w + frag_tile(p, 0, a.Kp) + lane * 16;
  }
  v4i af[U][NPW][2];
  auto load_w = [&](int b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = wave + (b * U + u) * W;
      if (p < pairs) {
#pragma unroll
        for (int i = 0; i < NPW; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            af[u][i][h] = __builtin_nontemporal_load(
                reinterpret_cast<const v4i *>(wp[i] + ((size_t)(2 * p + h) << 10)));
      }
    }
  };
  load_w(0);

  extern __shared__ __attribute__((aligned(16))) int8_t codes[];  // kSrc != kCodes: [T][Kp + 16]
  __shared__ float rscale[kFusedRows];
  __shared__ uint32_t rmax[kFusedRows][W];
  if constexpr (kSrc != kCodes) {
    // Rows of up to 64 W * 8 * kKeep elements stay in registers between their
    // maximum and their codes; wider ones are read again.
    constexpr int kKeep = 2, kStep = 64 * W * 8;
    float v[kFusedRows][kKeep][8];
    auto read = [&](int t, int c, float *o) {
      const int rem = a.K - c;
      if constexpr (kSrc == kTokens) {
        load8(a.in.x + t * a.in.ld + c, rem, o);
        if (a.in.inv && rem > 0) {
          float f[8];
          load8(a.in.inv + c, rem, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] *= f[j];
        }
      } else {
        load8(a.in.h + t * a.in.ld + c, rem, o);
      }
    };
#pragma unroll
    for (int t = 0; t < kFusedRows; ++t) {
      if (t >= a.T) break;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        read(t, threadIdx.x * 8 + i * kStep, v[t][i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(v[t][i][j]));
      }
      for (int c = threadIdx.x * 8 + kKeep * kStep; c < a.K; c += kStep) {
        float o[8];
        read(t, c, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(o[j]));
      }
      m = wave_max_bits(m);
      if (lane == 0) rmax[t][wave] = m;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kFusedRows; ++t) {
      if (t >= a.T) break;
      uint32_t m = rmax[t][0];
#pragma unroll
      for (int i = 1; i < W; ++i) m = umax(m, rmax[t][i]);
      const RowCode rc = row_code(m, kF8);
      if (threadIdx.x == 0) rscale[t] = rc.scale;
      int8_t *row = codes + t * (a.Kp + 16);
      auto put = [&](int c, const float *o) {
        if (c < a.Kp)
          *reinterpret_cast<v2i *>(row + c) =
              v2i{(int)row_codes4(o, rc, kF8), (int)row_codes4(o + 4, rc, kF8)};
      };
#pragma unroll
      for (int i = 0; i < kKeep; ++i) put(threadIdx.x * 8 + i * kStep, v[t][i]);
      for (int c = threadIdx.x * 8 + kKeep * kStep; c < a.Kp; c += kStep) {
        float o[8];
        read(t, c, o);
        put(c, o);
      }
    }
    __syncthreads();
  }

  // Token operand: lane l holds token l%16 of a row tile, 16 codes at k group
  // l/16. Rows past T repeat the last one (their sums are not stored).
  const int8_t *bp[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    int r = rt * 16 + (lane & 15);
    r = r < a.T ? r : a.T - 1;
    if constexpr (kSrc == kCodes) bp[rt] = a.in.q + (size_t)r * a.Kp + (lane >> 4) * 16;
    else bp[rt] = codes + r * (a.Kp + 16) + (lane >> 4) * 16;
  }
  Acc acc[NPW][RT];
#pragma unroll
  for (int i = 0; i < NPW; ++i)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[i][rt] = Acc{0, 0, 0, 0};
  for (int b = 0; wave + b * U * W < pairs; ++b) {
    if (b > 0) load_w(b);
    v4i bf[U][RT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = wave + (b * U + u) * W;
      if (p < pairs) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            bf[u][rt][h] = *reinterpret_cast<const v4i *>(bp[rt] + (size_t)p * 128 + h * 64);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (wave + (b * U + u) * W >= pairs) break;
#pragma unroll
      for (int i = 0; i < NPW; ++i)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          if constexpr (kF8) {
            acc[i][rt] = mfma16f8(af[u][i][0], af[u][i][1], bf[u][rt][0], bf[u][rt][1], acc[i][rt]);
          } else {
            acc[i][rt] = mfma16(af[u][i][0], bf[u][rt][0], acc[i][rt]);
            acc[i][rt] = mfma16(af[u][i][1], bf[u][rt][1], acc[i][rt]);
          }
        }
    }
  }

  __shared__ Acc red[W][NPW * RT][64];
#pragma unroll
  for (int i = 0; i < NPW; ++i)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) red[wave][i * RT + rt][lane] = acc[i][rt];
  __syncthreads();
  auto total = [&](int c) {
    Acc s = red[0][c][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) s += red[w][c][lane];
    return s;
  };
  const Epilogue &ep = a.ep;
  constexpr int kUnits = kGated ? NPW / 2 : NPW;
  const int ch0 = (lane >> 4) * 4;
  for (int c = wave; c < kUnits * RT; c += W) {
    const int i = c / RT, rt = c % RT;
    const int r = rt * 16 + (lane & 15);
    const int p = panel(i);
    const bool valid = r < a.T && p < (a.Np >> 4);
    const float rs = !valid ? 0.0f : kSrc == kCodes ? ep.row_scale[r] : rscale[r];
    if constexpr (kGated) {
      const Acc g = total(i * RT + rt), u = total((i + kUnits) * RT + rt);
      const int f0 = (p >> 2) * 32 + (p & 1) * 16 + ch0;
      uint32_t m = 0;
      if (valid) {
        const v4f sg = *reinterpret_cast<const v4f_a4 *>(ep.scale + p * 16 + ch0);
        const v4f su = *reinterpret_cast<const v4f_a4 *>(ep.scale + (p + 2) * 16 + ch0);
        v4f h;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = swiglu((float)g[j] * rs * sg[j], (float)u[j] * rs * su[j]);
          m = umax(m, f0 + j < ep.N ? abs_bits(h[j]) : 0u);
        }
        // h rows have the pitch of code rows: the padding columns are there
        *reinterpret_cast<v4f *>(static_cast<float *>(ep.out) + (int64_t)r * ep.ld_out + f0) = h;
      }
      if (ep.amax) {
        m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = umax(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (valid && lane < 16) atomicMax(ep.amax + r, m);
      }
    } else {
      const Acc s = total(c);
      if (valid) {
        const v4f sc = *reinterpret_cast<const v4f_a4 *>(ep.scale + p * 16 + ch0);
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)s[j] * rs * sc[j];
        finish_columns<4>(ep, r, p * 16 + ch0, v);
      }
    }
  }
}

template <int RT, int NPW, int W, int U, bool kGated, int kSrc>
hipError_t run(const StreamArgs &a, bool fp8, hipStream_t st) {
  const int per = kGated ? NPW / 2 : NPW;
  const int units = kGated ? a.Np / 32 : a.Np / 16;
  const dim3 grid((unsigned)((units + per - 1) / per));
  const size_t lds = kSrc == kCodes ? 0 : (size_t)a.T * (a.Kp + 16);
  (void)hipGetLastError();
  if (fp8)
    hipLaunchKernelGGL((linear_stream_kernel<RT, NPW, W, U, true, kGated, kSrc>), grid,
                       dim3(64 * W), lds, st, a);
  else
    hipLaunchKernelGGL((linear_stream_kernel<RT, NPW, W, U, false, kGated, kSrc>), grid,
                       dim3(64 * W), lds, st, a);
  return hipGetLastError();
}

template <bool kGated>
hipError_t pick(const StreamArgs &a, bool fp8, hipStream_t st) {
  constexpr int P = kGated ? 2 : 1;
  if (a.in.x) return run<1, P, 8, 4, kGated, kTokens>(a, fp8, st);
  if (a.in.h) return run<1, P, 8, 4, kGated, kHidden>(a, fp8, st);
  if (a.T <= 16) return run<1, P, 8, 4, kGated, kCodes>(a, fp8, st);
  if (a.T <= 32) return run<2, 2, 8, 2, kGated, kCodes>(a, fp8, st);
  return run<4, 2, 8, 2, kGated, kCodes>(a, fp8, st);
}

}  // namespace

hipError_t launch_linear_stream(const StreamIn &in, int T, const int8_t *w, int K, int Np,
                                bool gated, bool fp8, const Epilogue &ep, hipStream_t st) {
  StreamArgs a{};
  a.in = in; a.T = T; a.K = K; a.Kp = row_pitch(K); a.w = w; a.Np = Np; a.ep = ep;
  return gated ? pick<true>(a, fp8, st) : pick<false>(a, fp8, st);
}

}  // namespace moe
