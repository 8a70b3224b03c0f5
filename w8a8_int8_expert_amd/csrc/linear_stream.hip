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
// only add a copy), through a ring of U pairs: a pair's registers are loaded
// again as soon as its products are issued, so U - 1 pairs per panel stay in
// flight. The tokens are the B operand, 16 per row tile. The W partial sums
// meet in LDS, and the wavefronts share the epilogue. INT8 sums are exact; FP8
// sums are added in wavefront order.
//
// Up to four tokens the kernel codes the rows itself (kTokens: bf16 tokens, kHidden:
// the feed-forward's hidden rows, from its gate and up values): every block
// does it over again, which costs less than a launch of its own, and the
// weights' first loads are in flight meanwhile.
//
// The gate and up projections run here as one plain product into fp32 rows;
// whoever codes the hidden rows applies SwiGLU. (Pairing gate and up panels in
// a block would halve the blocks of a launch that has too few of them.)
#include "epilogue_device.h"

namespace moe {
namespace {

// Row-major codes, codes in tiles, bf16 tokens, the hidden rows' gate and up values.
enum { kCodes, kTiles, kTokens, kHidden };

struct StreamArgs {
  StreamIn in;
  int T, Kp, K;
  const int8_t *w;
  int Np;
  Epilogue ep;
};

template <bool kF8> struct Acc16v { typedef v4i T; };
template <> struct Acc16v<true> { typedef v4f T; };

template <int RT, int NPW, int W, int U, bool kF8, int kSrc>
__global__ __launch_bounds__(64 * W) void linear_stream_kernel(const StreamArgs a) {
  typedef typename Acc16v<kF8>::T Acc;
  constexpr bool kFused = kSrc == kTokens || kSrc == kHidden;
  static_assert(!kFused || RT == 1, "rows coded by the block");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int pairs = a.Kp >> 7;

  const int8_t *wp[NPW];
#pragma unroll
  for (int i = 0; i < NPW; ++i) {
    int p = (int)blockIdx.x * NPW + i;
    p = p < (a.Np >> 4) ? p : (a.Np >> 4) - 1;  // read, never stored
    wp[i] = a.w + frag_tile(p, 0, a.Kp) + lane * 16;
  }
  // This wavefront's pairs wave, wave + W, ...: n of them, pair s in ring slot
  // s % U.
  const int n = wave < pairs ? (pairs - wave + W - 1) / W : 0;
  v4i af[U][NPW][2], bf[U][RT][2];
  auto load_w = [&](int u, int s) {
    const size_t at = (size_t)(wave + s * W) << 11;
#pragma unroll
    for (int i = 0; i < NPW; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        af[u][i][h] =
            __builtin_nontemporal_load(reinterpret_cast<const v4i *>(wp[i] + at + h * 1024));
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < n) load_w(u, u);

  extern __shared__ __attribute__((aligned(16))) int8_t codes[];  // kFused: [T][Kp + 16]
  __shared__ float rscale[kFusedRows];
  __shared__ uint32_t rmax[kFusedRows][W];
  if constexpr (kFused) {
    // Rows of up to 64 W * 8 * kKeep elements stay in registers between their
    // maximum and their codes; wider ones are read again.
    constexpr int kKeep = 2, kStep = 64 * W * 8;
    float v[kFusedRows][kKeep][8];
    auto read = [&](int t, int c, float *o) {
      const int rem = a.K - c;
      if constexpr (kSrc == kTokens) {
        if (rem <= 0) {  // most threads of a narrow row: no element loads to skip
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = 0.0f;
          return;
        }
        load8(a.in.x + t * a.in.ld, c, a.K, o);
        if (a.in.inv) {
          float f[8];
          load8(a.in.inv, c, a.K, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] *= f[j];
        }
      } else {
        hidden8(a.in.h + t * a.in.ld, c, rem, o);
      }
    };
#pragma unroll
    for (int t = 0; t < kFusedRows; ++t) {
      if (t >= a.T) break;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        if (i * kStep >= a.Kp) break;  // uniform
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
      for (int i = 0; i < kKeep; ++i)
        if (i * kStep < a.Kp) put(threadIdx.x * 8 + i * kStep, v[t][i]);
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
    else if constexpr (kSrc == kTiles)
      bp[rt] = a.in.q + frag_tile(r >> 4, 0, a.Kp) + ((lane & 48) + (r & 15)) * 16;
    else bp[rt] = codes + r * (a.Kp + 16) + (lane >> 4) * 16;
  }
  auto load_x = [&](int u, int s) {
    constexpr int kHalf = kSrc == kTiles ? 1024 : 64;  // 64 k further
    const size_t at = (size_t)(wave + s * W) * (2 * kHalf);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        bf[u][rt][h] = *reinterpret_cast<const v4i *>(bp[rt] + at + h * kHalf);
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < n) load_x(u, u);
  Acc acc[NPW][RT];
#pragma unroll
  for (int i = 0; i < NPW; ++i)
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[i][rt] = Acc{0, 0, 0, 0};
  // FP8 codes are multiplied as bf16, into which they convert exactly: the FP8
  // instruction drops what lies 13 bits below the largest of eight products
  // (sums 3e-5 off, against 1e-7), and the matrix cores wait for memory here.
  auto multiply = [&](int u) {
    if constexpr (kF8) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v8bf b[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            b[rt] = codes_bf16(bf[u][rt][h][2 * e], bf[u][rt][h][2 * e + 1]);
#pragma unroll
          for (int i = 0; i < NPW; ++i) {
            const v8bf w = codes_bf16(af[u][i][h][2 * e], af[u][i][h][2 * e + 1]);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
              acc[i][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, b[rt], acc[i][rt], 0, 0, 0);
          }
        }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NPW; ++i)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            acc[i][rt] = mfma16(af[u][i][h], bf[u][rt][h], acc[i][rt]);
    }
  };
  int s = 0;
  for (; s + 2 * U <= n; s += U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      multiply(u);
      load_w(u, s + U + u);
      load_x(u, s + U + u);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (s + u < n) {
      multiply(u);
      if (s + U + u < n) {
        load_w(u, s + U + u);
        load_x(u, s + U + u);
      }
    }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (s + U + u < n) multiply(u);

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
  const int ch0 = (lane >> 4) * 4;
  for (int c = wave; c < NPW * RT; c += W) {
    const int r = c % RT * 16 + (lane & 15);
    const int p = (int)blockIdx.x * NPW + c / RT;
    const Acc sum = total(c);
    if (r < a.T && p < (a.Np >> 4)) {
      const float rs = kFused ? rscale[r] : ep.row_scale[r];
      const v4f sc = *reinterpret_cast<const v4f_a4 *>(ep.scale + p * 16 + ch0);
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = (float)sum[j] * rs * sc[j];
      finish_columns<4>(ep, r, p * 16 + ch0, v);
    }
  }
}

template <int RT, int NPW, int W, int U, int kSrc>
hipError_t run(const StreamArgs &a, bool fp8, hipStream_t st) {
  const dim3 grid((unsigned)((a.Np / 16 + NPW - 1) / NPW));
  const bool fused = kSrc == kTokens || kSrc == kHidden;
  const size_t lds = fused ? (size_t)a.T * (a.Kp + 16) : 0;
  (void)hipGetLastError();
  if (fp8)
    hipLaunchKernelGGL((linear_stream_kernel<RT, NPW, W, U, true, kSrc>), grid,
                       dim3(64 * W), lds, st, a);
  else
    hipLaunchKernelGGL((linear_stream_kernel<RT, NPW, W, U, false, kSrc>), grid,
                       dim3(64 * W), lds, st, a);
  return hipGetLastError();
}

// Panels a block owns: one while a launch has at most a block per compute unit
// then, more where that leaves enough blocks, so that the tokens are read a
// half or a quarter as often. Measured on MI355X (INT8, K 4096, the codes' launch
// of 2.5 included; us with 1, 2 and 4 panels a block):
//   4096 outputs:  16 tokens 8.0, 9.0, 11.3    64 tokens 10.8, 12.1, 15.8
//   8192 outputs:  16 tokens 11.7, 10.7, 12.6  64 tokens 17.0, 14.1, 17.2
//   11000 outputs: 16 tokens 14.7, 14.0, 13.5  32 tokens 18.3, 16.4, 15.4
//   16384 outputs: 16 tokens 18.2, 15.9, 16.3  32 tokens 22.8, 17.9, 17.7
//   32003 outputs: 32 tokens 38.7, 30.0, 27.6
// Between 512 and 1024 panels, blocks of two would be more than one a unit and
// fewer than two: with K from 4096 on, blocks of four take 3 to 9 % less time (32
// tokens, K 8192, 12800 outputs: 28.9, 25.9), below it 2 % more.
template <int RT, int kSrc>
hipError_t pick(const StreamArgs &a, bool fp8, hipStream_t st) {
  const int panels = a.Np / 16;
  // A call that is given the codes of such few tokens takes the same number of
  // wavefronts as one that codes them: it cuts K the same way, and FP8 sums are
  // the same to the last bit.
  bool fused = kSrc == kTokens || kSrc == kHidden;
  if constexpr (kSrc == kCodes && RT == 1) fused = fused_tokens(a.T, a.K);
  if (panels <= 256) {
    // Rows coded by the block: more wavefronts share that work (one token,
    // 4096 outputs, K 4096: 5.6 with 16 wavefronts, 6.1 with 8).
    if constexpr (kSrc != kTiles && RT == 1)
      if (fused && a.Kp >= 4096) return run<RT, 1, 16, 2, kSrc>(a, fp8, st);
    return run<RT, 1, 8, 2, kSrc>(a, fp8, st);
  }
  const bool four = !fused && a.Kp >= 4096 ? panels > 512 : (fused || RT > 1) && panels >= 1024;
  if constexpr (RT < 4)  // (33 tokens and more stream to 512 panels at most)
    if (four) return run<RT, 4, 4, 2, kSrc>(a, fp8, st);
  return run<RT, 2, 8, 2, kSrc>(a, fp8, st);
}

}  // namespace

hipError_t launch_linear_stream(const StreamIn &in, int T, const int8_t *w, int K, int Np, bool fp8,
                                const Epilogue &ep, hipStream_t st) {
  StreamArgs a{};
  a.in = in; a.T = T; a.K = K; a.Kp = row_pitch(K); a.w = w; a.Np = Np; a.ep = ep;
  if (in.x) return pick<1, kTokens>(a, fp8, st);
  if (in.h) return pick<1, kHidden>(a, fp8, st);
  if (in.tiles) {
    if (T <= 16) return pick<1, kTiles>(a, fp8, st);
    if (T <= 32) return pick<2, kTiles>(a, fp8, st);
    return pick<4, kTiles>(a, fp8, st);
  }
  if (T <= 16) return pick<1, kCodes>(a, fp8, st);
  if (T <= 32) return pick<2, kCodes>(a, fp8, st);
  return pick<4, kCodes>(a, fp8, st);
}

}  // namespace moe
