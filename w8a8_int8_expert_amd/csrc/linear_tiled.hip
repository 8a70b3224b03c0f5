// linear_tiled.hip -- W8A8 products of many tokens, bound by the matrix cores
// and by feeding them.
//
// "MiniMax-M3 W8A8 inference on K100AI" (mhpq.cn/news/1068415) §1.2, §4.3.
//
// A block computes BM tokens x BN packed weight rows, K in stages of 128. Both
// operands reach LDS by direct global -> LDS loads: tokens row-major (whole
// 128-byte lines, XOR-swizzled so that an operand read is free of bank
// conflicts), weights as fragment tiles, through rings of S stages. WM x WN
// wavefronts own MI x NJ accumulators of 32 x 32. INT8 multiplies on the
// 32x32x32 instruction (the 16x16x64 form reaches half its rate), FP8 on
// 32x32x64 or, converted, on bf16 32x32x16.
//
// What bounds the small shapes is the operand feed: a compute unit gets about
// 50 bytes per ns into LDS, whatever the depth of its rings or the number of its
// wavefronts (rings of 2 to 6 stages, one to three blocks a unit). A larger tile
// needs fewer bytes per product, a smaller one uses more compute units.
//
// Tiles are numbered (N group, M tile, N tile in group), and each XCD takes a
// contiguous eighth of that order, so that the blocks that run together on one
// L2 share token and weight panels.
//
// Few tiles: blockIdx.y cuts K into `split` parts; each writes its raw sums
// and a second launch adds them in order and finishes the columns.
#include <type_traits>

#include "epilogue_device.h"

namespace moe {
namespace {

// How codes are multiplied: INT8; FP8 by the FP8 instructions; FP8 as bf16, into
// which e4m3 converts exactly. The FP8 instructions keep the products of eight
// consecutive k to 13 bits below the largest, truncated, before they add them in
// fp32: sums are 1.5e-5 off (rms, of the sums' rms). The bf16 instructions add
// whole products (1e-7 off), at half the rate: codes of 256 tokens, K 4096, 6144
// outputs 23.6 us against 14.4; 1024 tokens 47.5, 26.2; 16384 tokens, 8192 outputs
// 801, 459. A result that is rounded to bf16 at once (1.7e-3) takes the FP8
// instructions: one value in 83 then rounds the other way, 2.3e-4 in all. A result
// that stays fp32 is multiplied as bf16, and so are the gate and up rows of a
// feed-forward block, whose hidden codes would move by whole e4m3 steps.
enum { kInt8, kFp8, kFp8Exact };

struct TiledLinear {
  const int8_t *q;
  int64_t T;
  const int8_t *w;
  int Kp, Np, mt, nt, gn, split;
  int32_t *partial;  // [split][T][Np] sums (fp32 bits for FP8)
  Epilogue ep;
};

// Tile of place L: groups of gn N tiles (the last may be smaller), M-major
// inside a group.
__device__ __forceinline__ void tile_of(const TiledLinear &a, int64_t L, int *m, int *n) {
  const int64_t per = (int64_t)a.mt * a.gn;
  const int grp = (int)(L / per);
  const int r = (int)(L - grp * per);
  const int g = a.nt - grp * a.gn < a.gn ? a.nt - grp * a.gn : a.gn;
  *m = r / g;
  *n = grp * a.gn + (r - *m * g);
}

// At most n stages of L loads each stay in flight (n <= M).
template <int M, int L>
__device__ __forceinline__ void wait_stages(int n) {
  if constexpr (M > 0) {
    if (n < M) {
      wait_stages<M - 1, L>(n);
      return;
    }
  }
  wait_barrier<M * L>();
}

template <int WM, int WN, int MI, int NJ, int S, int kMul, bool kGated, bool kSplit>
__global__ __launch_bounds__(64 * WM * WN, 1) void linear_tiled_kernel(const TiledLinear a) {
  typedef typename Acc32<kMul != kInt8>::T Acc;
  constexpr int W = WM * WN, BM = WM * MI * 32, BN = WN * NJ * 32;
  constexpr int kA = BM * 128, kB = BN * 128;  // one stage of each ring
  constexpr int kALoads = BM / 8 / W, kBLoads = BN / 8 / W;
  static_assert(kALoads * W * 8 == BM && kBLoads * W * 8 == BN, "load split");
  constexpr int kRing = S * (kA + kB);
  // Epilogue: 16 rows x the wavefront's columns per pass, pitch padded by 8
  // words so that the two 32-lane halves (rows r and r + 4) use other banks.
  constexpr int kPitch = NJ * 32 + 8, kSlice = 16 * kPitch * 4;
  static_assert(W * kSlice <= kRing, "epilogue staging");
  constexpr int kCols = (BN + 63) / 64 * 64;  // whole wavefronts fetch scales
  static_assert(BM % 64 == 0, "scales");
  __shared__ __attribute__((aligned(1024))) int8_t lds[kRing];
  __shared__ __attribute__((aligned(16))) float row_scale[BM], row_gate[BM], col_scale[kCols],
      col_bias[kCols];

  const int64_t tiles = (int64_t)a.mt * a.nt, chunk = (tiles + 7) >> 3;
  const int64_t L = (int64_t)(blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= chunk || L >= tiles) return;
  int mtile, ntile;
  tile_of(a, L, &mtile, &ntile);
  const int64_t m0 = (int64_t)mtile * BM;
  const int n0 = ntile * BN;
  const int rows = a.T - m0 < BM ? (int)(a.T - m0) : BM;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / WN, wn = wave % WN;
  // This block's stages of K: [d0, d0 + D).
  int d0 = 0, D = a.Kp >> 7;
  if (kSplit) {
    d0 = (int)((int64_t)(a.Kp >> 7) * blockIdx.y / a.split);
    D = (int)((int64_t)(a.Kp >> 7) * (blockIdx.y + 1) / a.split) - d0;
  }

  // Instruction i of a token stage fills rows 8i .. 8i+7: lane l brings chunk
  // (l%8) ^ (row/2 % 8) of row 8i + l/8 to slot l%8.
  const int8_t *asrc[kALoads];
#pragma unroll
  for (int t = 0; t < kALoads; ++t) {
    const int i = kALoads * wave + t;
    int r = 8 * i + (lane >> 3);
    r = r < rows ? r : rows - 1;  // rows past T: computed, never stored
    asrc[t] = a.q + (m0 + r) * a.Kp + (size_t)d0 * 128 +
              (((lane & 7) ^ ((4 * (i & 1) + (lane >> 4)) & 7)) << 4);
  }
  // Instruction j of a weight stage brings 1 KB tile (j/2, j%2) of the stage.
  const int8_t *bsrc[kBLoads];
#pragma unroll
  for (int t = 0; t < kBLoads; ++t) {
    const int j = kBLoads * wave + t;
    int p = (n0 >> 4) + (j >> 1);
    p = p < (a.Np >> 4) ? p : (a.Np >> 4) - 1;  // columns past Np: never stored
    bsrc[t] = a.w + frag_tile(p, 2 * d0 + (j & 1), a.Kp) + lane * 16;
  }
  // The wavefront's loads of a stage are numbered: kALoads of tokens, then
  // kBLoads of weights.
  constexpr int kLoads = kALoads + kBLoads, kEarly = kLoads / 2;
  auto load = [&](int d, int slot, int t) {
    const bool tokens = t < kALoads;
    const int u = tokens ? t : t - kALoads;
    const int8_t *src = tokens ? asrc[u] + (size_t)d * 128 : bsrc[u] + (size_t)d * 2048;
    int8_t *dst = tokens ? lds + slot * kA + (kALoads * wave + u) * 1024
                         : lds + S * kA + slot * kB + (kBLoads * wave + u) * 1024;
    dma16(src, __builtin_amdgcn_readfirstlane(lds_addr(dst)));
  };

  // What the epilogue needs of each row and column goes to LDS ahead of the
  // operands: the K loop hides its latency, and it holds no registers. Rows and
  // columns that do not exist repeat the last one.
  const Epilogue &ep = a.ep;
  const int nw = n0 + wn * NJ * 32;  // first packed row of this wavefront
  const bool biased = !kGated && ep.bias, gated = !kGated && ep.gate;
  if (!kSplit) {
    auto fetch = [&](const float *src, int64_t at, int64_t last, float *dst) {
      const int64_t i = at + lane;
      dma4(src + (i < last ? i : last), __builtin_amdgcn_readfirstlane(lds_addr(dst)));
    };
    for (int i = wave; i < (BM + kCols) / 64; i += W) {
      const int r = i * 64, c = r - BM;
      if (r < BM) {
        fetch(ep.row_scale, m0 + r, a.T - 1, row_scale + r);
        if (gated) fetch(ep.gate, m0 + r, a.T - 1, row_gate + r);
      } else {
        fetch(ep.scale, n0 + c, a.Np - 1, col_scale + c);
        if (biased) fetch(ep.bias, n0 + c, ep.N - 1, col_bias + c);
      }
    }
  }

  Acc acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int c = 0; c < NJ; ++c)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][c][v] = 0;

  // 16-row weight tile p of the stage starts at 2048 p, its k half at + 1024.
  const int boff = wn * NJ * 4096 + (((lane >> 5) * 16) + (lane & 15)) * 16 +
                   ((lane & 31) >> 4) * 2048;
  const int aoff = (wm * MI * 32 + (lane & 31)) * 128;
  int axor[4];  // chunk 2 k + lane/32 of the lane's row, k the 32-k quarter
#pragma unroll
  for (int k = 0; k < 4; ++k) axor[k] = ((2 * k + (lane >> 5)) ^ ((lane >> 1) & 7)) << 4;

  // A stage is kSteps steps of matrix work: 64 k each for the FP8 instructions,
  // 32 for the others. The operands of a step are read while the step before it
  // multiplies, and the first ones of a stage while the last step of the stage
  // before does, so that neither the reads nor the barrier between two stages
  // leave the matrix cores idle. Reads and loads go between the matrix
  // instructions one by one: a wavefront that issues its loads in a row waits for
  // the load queue with the matrix cores idle. So do the conversions of kFp8Exact,
  // whose step is two halves of eight codes a lane.
  constexpr int kSteps = kMul == kFp8 ? 2 : 4, kH = kMul == kFp8 ? 2 : 1;
  constexpr int kHalves = kMul == kFp8Exact ? 2 : 1;
  constexpr int kReads = (MI + NJ) * kH, kM = MI * NJ * kHalves;
  v4i af[2][MI][kH], bf[2][NJ][kH];
  auto read = [&](int buf, int s, const int8_t *as, const int8_t *bs, int j) {
    const int h = j % kH, i = j / kH, k = s * kH + h;
    if (i < MI)
      af[buf][i][h] = *reinterpret_cast<const v4i *>(as + aoff + i * 4096 + axor[k]);
    else
      bf[buf][i - MI][h] = *reinterpret_cast<const v4i *>(
          bs + boff + (i - MI) * 4096 + (k >> 1) * 1024 + (k & 1) * 512);
  };
  // One step: the products of buffer s % 2, the reads of step `ns` into the
  // other from a stage at as, bs (ns < 0: none), loads [t0, t1) of stage d.
  auto step = [&](int s, int ns, const int8_t *as, const int8_t *bs, int t0, int t1, int d,
                  int to) {
    constexpr int kPer = (kReads + kM - 1) / kM;
    const int buf = s & 1;
    v8bf ax[kHalves][MI], bx[2];  // kFp8Exact: as bf16, the weights a product ahead
    auto half = [](const v4i &v, int e) { return codes_bf16(v[2 * e], v[2 * e + 1]); };
    if constexpr (kMul == kFp8Exact) {
#pragma unroll
      for (int i = 0; i < MI; ++i) ax[0][i] = half(af[buf][i][0], 0);
      bx[0] = half(bf[buf][0][0], 0);
    }
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const int n = m / MI, e = n / NJ, c = n % NJ, i = m % MI;
      if constexpr (kMul == kFp8Exact) {
        acc[i][c] =
            __builtin_amdgcn_mfma_f32_32x32x16_bf16(ax[e][i], bx[n & 1], acc[i][c], 0, 0, 0);
        if (i == 0 && n + 1 < 2 * NJ)
          bx[(n + 1) & 1] = half(bf[buf][(n + 1) % NJ][0], (n + 1) / NJ);
        if (n == NJ - 1) ax[kHalves - 1][i] = half(af[buf][i][0], 1);
      } else if constexpr (kMul == kFp8) {
        acc[i][c] =
            mfma32f8(af[buf][i][0], af[buf][i][1], bf[buf][c][0], bf[buf][c][1], acc[i][c]);
      } else {
        acc[i][c] = mfma32(af[buf][i][0], bf[buf][c][0], acc[i][c]);
      }
      if (ns >= 0) {
#pragma unroll
        for (int j = m * kPer; j < (m + 1) * kPer; ++j)
          if (j < kReads) read(buf ^ 1, ns, as, bs, j);
      }
#pragma unroll
      for (int j = t0; j < t1; ++j)
        if ((j - t0) % kM == m) load(d, to, j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Stages 0 .. S-1 come first (the last of them, where all S exist, by its
  // early loads only). Once every wavefront has read the last of stage d, stage
  // d + S goes to its slot: the early loads during the last step of stage d,
  // the others during the first of stage d + 1. Loads return in order, so what
  // may still be in flight when stage d + 1 begins is what was issued after it:
  // stages d + 2 .. d + S - 1.
  const int8_t *const rings = lds;
#pragma unroll
  for (int d = 0; d < S; ++d)
    if (d < D) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        if (d < S - 1 || j < kEarly) load(d, d, j);
    }
  if (D >= S) wait_barrier<(S - 2) * kLoads + kEarly>();
  else wait_stages<S - 2, kLoads>(D - 1);
  const bool skip = wm * MI * 32 >= rows;  // no row of this wavefront exists
  int slot = 0;                            // of stage d
  auto after = [&](int s) { return s + 1 == S ? 0 : s + 1; };
  auto before = [&](int s) { return s == 0 ? S - 1 : s - 1; };
  auto stage = [&](auto late, auto early, auto last, int d) {
    const int8_t *as = rings + slot * kA, *bs = rings + S * kA + slot * kB;
#pragma unroll
    for (int s = 0; s + 1 < kSteps; ++s)
      step(s, s + 1, as, bs, late && s == 0 ? kEarly : 0, late && s == 0 ? kLoads : 0, d + S - 1,
           before(slot));
    if constexpr (last) {
      step(kSteps - 1, -1, as, bs, 0, 0, 0, 0);
    } else {
      wait_stages<S - 2, kLoads>(D - 2 - d);
      const int next = after(slot);
      step(kSteps - 1, 0, rings + next * kA, rings + S * kA + next * kB, 0, early ? kEarly : 0,
           d + S, slot);
      slot = next;
    }
  };
  int d = 0;
  if (skip) {
    for (; d + 1 < D; ++d) {
      if (d + S - 1 < D) {
        for (int j = kEarly; j < kLoads; ++j) load(d + S - 1, before(slot), j);
      }
      wait_stages<S - 2, kLoads>(D - 2 - d);
      if (d + S < D) {
        for (int j = 0; j < kEarly; ++j) load(d + S, slot, j);
      }
      slot = after(slot);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kReads; ++j) read(0, 0, rings, rings + S * kA, j);
    constexpr std::true_type yes;
    constexpr std::false_type no;
    for (; d + S < D; ++d) stage(yes, yes, no, d);
    for (; d + S <= D && d + 1 < D; ++d) stage(yes, no, no, d);
    for (; d + 1 < D; ++d) stage(no, no, no, d);
    stage(no, no, yes, d);
  }
  wait_barrier<0>();  // every wavefront is done with the rings

  // Epilogue through the wavefront's own slice of the rings, 16 rows a pass.
  // Lane holds column lane%32 of each 32 x 32 accumulator and rows 8*(v/4) +
  // 4*(lane/32) + v%4.
  if (skip) return;
  float *slice = reinterpret_cast<float *>(lds + wave * kSlice);
  const int rl = 4 * (lane >> 5);
  float sc[NJ], bs[NJ];
  if (!kSplit) {
#pragma unroll
    for (int c = 0; c < NJ; ++c) {
      sc[c] = col_scale[wn * NJ * 32 + 32 * c + (lane & 31)];
      bs[c] = biased ? col_bias[wn * NJ * 32 + 32 * c + (lane & 31)] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int vh = 0; vh < 2; ++vh) {
      const int mr = (wm * MI + i) * 32 + 16 * vh;  // first row of the pass
      if (mr >= rows) return;
      v4f rsc[2], rgt[2];
      if (!kSplit) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          rsc[g] = *reinterpret_cast<const v4f *>(row_scale + mr + 8 * g + rl);
          rgt[g] = gated ? *reinterpret_cast<const v4f *>(row_gate + mr + 8 * g + rl)
                         : v4f{1.0f, 1.0f, 1.0f, 1.0f};
        }
      }
#pragma unroll
      for (int vv = 0; vv < 8; ++vv) {
        const int v = 8 * vh + vv, r = 8 * (vv >> 2) + rl + (vv & 3);
        float *row = slice + r * kPitch + (lane & 31);
        if constexpr (kSplit) {
#pragma unroll
          for (int c = 0; c < NJ; ++c) {
            const auto e = acc[i][c][v];
            row[32 * c] = __builtin_bit_cast(float, e);
          }
        } else if constexpr (kGated) {
          const float x = rsc[vv >> 2][vv & 3];
          uint32_t m = 0;
#pragma unroll
          for (int c = 0; c < NJ; c += 2) {
            const float h = swiglu((float)acc[i][c][v] * x * sc[c],
                                   (float)acc[i][c + 1][v] * x * sc[c + 1]);
            row[16 * c] = h;
            m = umax(m, nw / 2 + 16 * c + (lane & 31) < ep.N ? abs_bits(h) : 0u);
          }
          m = half_wave_max(m);
          if ((lane & 31) == 31) slice[r * kPitch + NJ * 32] = __uint_as_float(m);
        } else {
          const float x = rsc[vv >> 2][vv & 3];
          if (!biased && !gated) {
#pragma unroll
            for (int c = 0; c < NJ; ++c) row[32 * c] = (float)acc[i][c][v] * x * sc[c];
          } else {
            const float g = rgt[vv >> 2][vv & 3];
#pragma unroll
            for (int c = 0; c < NJ; ++c)
              row[32 * c] = ((float)acc[i][c][v] * x * sc[c] + bs[c]) * g;
          }
        }
      }
      const int left = rows - mr;  // rows of the pass that exist
      if constexpr (kSplit) {
        int32_t *part = a.partial + (size_t)blockIdx.y * a.T * a.Np;
#pragma unroll
        for (int j = 0; j < NJ * 2; ++j) {
          const int r = (j * 64 + lane) / (NJ * 8), c4 = (j * 64 + lane) % (NJ * 8) * 4;
          const v4f x = *reinterpret_cast<const v4f *>(slice + r * kPitch + c4);
          if (r < left && nw + c4 < a.Np)
            *reinterpret_cast<v4f *>(part + (m0 + mr + r) * a.Np + nw + c4) = x;
        }
      } else if constexpr (kGated) {
        if (lane < 16 && lane < left)
          atomicMax(ep.amax + m0 + mr + lane, __float_as_uint(slice[lane * kPitch + NJ * 32]));
        // h columns nw/2 .. + 16 NJ; h rows have the pitch of code rows, so
        // whole 32-column runs exist
        float *h = static_cast<float *>(ep.out);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int r = (j * 64 + lane) / (NJ * 4), c4 = (j * 64 + lane) % (NJ * 4) * 4;
          const v4f x = *reinterpret_cast<const v4f *>(slice + r * kPitch + c4);
          if (r < left && nw + 2 * c4 < a.Np)
            *reinterpret_cast<v4f *>(h + (m0 + mr + r) * ep.ld_out + nw / 2 + c4) = x;
        }
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int r = (j * 64 + lane) / (NJ * 4), c8 = (j * 64 + lane) % (NJ * 4) * 8;
          float v[8];
          const v4f x = *reinterpret_cast<const v4f *>(slice + r * kPitch + c8);
          const v4f y = *reinterpret_cast<const v4f *>(slice + r * kPitch + c8 + 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = x[k];
            v[4 + k] = y[k];
          }
          if (r < left) store_columns<8>(ep, m0 + mr + r, nw + c8, v);
        }
      }
    }
  }
}

// Adds the parts of K in order and finishes the columns: 8 columns a thread.
template <bool kF8, bool kGated>
__global__ __launch_bounds__(256) void linear_join_kernel(const TiledLinear a) {
  const int per = kGated ? a.Np / 16 : a.Np / 8;  // 8-column runs of a row
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / per;
  if (t >= a.T) return;
  const int c8 = (int)(i - t * per) * 8;
  // packed column of output column c8
  const int p0 = kGated ? c8 / 32 * 64 + c8 % 32 : c8;
  const Epilogue &ep = a.ep;
  const float rs = ep.row_scale[t];
  auto sums = [&](int p, float *o) {
    typename Acc32<kF8>::T s;  // the first 8 of 16
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0;
    for (int k = 0; k < a.split; ++k) {
      const int32_t *src = a.partial + ((size_t)k * a.T + t) * a.Np + p;
      const v4i x = *reinterpret_cast<const v4i *>(src);
      const v4i y = *reinterpret_cast<const v4i *>(src + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kF8) {
          s[j] += __int_as_float(x[j]);
          s[4 + j] += __int_as_float(y[j]);
        } else {
          s[j] += x[j];
          s[4 + j] += y[j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (float)s[j] * rs * ep.scale[p + j];
  };
  float v[8];
  sums(p0, v);
  if constexpr (kGated) {
    float u[8];
    sums(p0 + 32, u);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = swiglu(v[j], u[j]);
      m = umax(m, c8 + j < ep.N ? abs_bits(v[j]) : 0u);
    }
    float *h = static_cast<float *>(ep.out) + t * ep.ld_out + c8;
    *reinterpret_cast<v4f *>(h) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f *>(h + 4) = v4f{v[4], v[5], v[6], v[7]};
    // One atomic for the lanes of a row: whole wavefronts of a wide row, runs of
    // four lanes (a row has a multiple of four) where a wavefront holds several.
    m = umax(m, (uint32_t)__shfl_xor((int)m, 1, 64));
    m = umax(m, (uint32_t)__shfl_xor((int)m, 2, 64));
    if (per % 64 == 0) {
      m = wave_max_bits(m);
      if ((threadIdx.x & 63) == 0) atomicMax(ep.amax + t, m);
    } else if ((threadIdx.x & 3) == 0) {
      atomicMax(ep.amax + t, m);
    }
  } else {
    finish_columns<8>(ep, t, c8, v);
  }
}

template <int WM, int WN, int MI, int NJ, int S, int kMul, bool kGated, bool kSplit>
hipError_t run_as(TiledLinear a, hipStream_t st) {
  constexpr int BM = WM * MI * 32, BN = WN * NJ * 32;
  a.mt = (int)((a.T + BM - 1) / BM);
  a.nt = (a.Np + BN - 1) / BN;
  const int64_t tiles = (int64_t)a.mt * a.nt;
  // N tiles per group: an XCD's share of a single round is then mt x gn (few
  // M tiles) or 8 x 4 tiles.
  const int64_t share = ((tiles < 256 ? tiles : 256) + 7) / 8;
  a.gn = (int)(a.mt >= 8 ? 4 : (share + a.mt - 1) / a.mt);
  if (a.gn > a.nt) a.gn = a.nt;
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)a.split);
  return launch_kernel(linear_tiled_kernel<WM, WN, MI, NJ, S, kMul, kGated, kSplit>, grid,
                       dim3(64 * WM * WN), st, Timing{}, a);
}
template <int WM, int WN, int MI, int NJ, int S, bool kGated, bool kSplit = false>
hipError_t run(const TiledLinear &a, int mul, hipStream_t st) {
  if (mul == kInt8) return run_as<WM, WN, MI, NJ, S, kInt8, kGated, kSplit>(a, st);
  if constexpr (!kGated)
    if (mul == kFp8) return run_as<WM, WN, MI, NJ, S, kFp8, kGated, kSplit>(a, st);
  return run_as<WM, WN, MI, NJ, S, kFp8Exact, kGated, kSplit>(a, st);
}

template <bool kGated>
hipError_t join(const TiledLinear &a, int mul, hipStream_t st) {
  const int64_t n = a.T * (kGated ? a.Np / 16 : a.Np / 8);
  const dim3 grid((unsigned)((n + 255) / 256));
  if (mul != kInt8)
    return launch_kernel(linear_join_kernel<true, kGated>, grid, dim3(256), st, Timing{}, a);
  return launch_kernel(linear_join_kernel<false, kGated>, grid, dim3(256), st, Timing{}, a);
}

// Tile shape and split of K by estimated time: what a stage of 128 k takes with
// every compute unit at work (`full`), and in a last round of fewer tiles (from
// `a` for one to a + b). Fitted to 36 shapes of 70 to 8192 tokens, K 512 to 8192,
// 2048 to 32003 outputs, of which it misses the fastest tile by 0.2 % on average
// (at most 4 %). Measured on MI355X, INT8 / FP8 codes, us at K 4096:
//   tokens, outputs  256x256  256x192  128x256  128x192  128x128  64x128
//     256,  6144      45 / 44  38 / 39  30 / 30  23 / 20  19 / 17  16 / 15
//     512,  6144      45 / 45  38 / 39  31 / 31  25 / 22  20 / 19  24 / 23
//    1024,  6144      48 / 45  40 / 40  34 / 33  32 / 28  39 / 36  39 / 36
//    1000,  8192      51 / 48  44 / 43  39 / 38  51 / 45  45 / 40  48 / 45
//    1400,  6144      49 / 43  43 / 41  65 / 62  51 / 45  58 / 53  57 / 52
//    3000,  4096      55 / 52  83 / 81  67 / 64  75 / 67  63 / 58  72 / 65
// (64x128 fits twice on a unit.) Products of one round of 64x128 on the FP8
// instructions take eight wavefronts and five stages (us, against four and three;
// tokens, K, outputs): 256, 512, 6144 6.1, 6.7; 200, 1024, 8192 7.8, 8.3; 1000, 1024,
// 1500 7.2, 8.2; 300, 2048, 5000 9.4, 10.6; 100, 2048, 16384 10.3, 11.1; 256, 4096,
// 6144 14.1, 15.0; 512, 8192, 4096 24.0, 24.7. INT8: 16.8, 16.3 (256, 4096, 6144).
// FP8 codes multiplied as bf16 follow the same estimate: of 33 shapes of 40 to 16384
// tokens the tile it names is at most 5 % behind the fastest.
//
// A launch that leaves compute units idle splits K where that saves more than
// the second launch (1.5 us) and the partial sums (2.6 us a million) cost: 100,
// 8192, 1024 takes 22 us in 16 tiles, 12 with K in four; 64, 8192, 4096: 12.8
// with K in four, 16.0 in two, 14.4 in eight.
//
// The gated product has no tiles of 192 columns: a wavefront holds whole pairs
// of gate and up runs, and there is no split of 192 columns into such.
template <bool kGated>
hipError_t pick(TiledLinear a, int mul, hipStream_t st) {
  auto tiles = [&](int bm, int bn) {
    return ((a.T + bm - 1) / bm) * (int64_t)((a.Np + bn - 1) / bn);
  };
  auto rounds = [](int64_t n, double full, double lone, double more) {
    const int64_t rest = n % 256;
    return (double)(n / 256) * full + (rest ? lone + more * (double)rest / 256 : 0.0);
  };
  auto one = [](int64_t n) { return 0.28 + 0.12 * (n < 192 ? (double)n / 192 : 1.0); };
  const int D = a.Kp >> 7;
  const int64_t t = tiles(64, 128), rest = t % 512;  // two tiles a compute unit
  const double small =
      (double)(t / 512) * 0.75 +
      (rest > 256 ? 0.57 + 0.18 * (double)(rest - 256) / 256 : rest ? one(rest) : 0.0);
  const double c0 = rounds(tiles(256, 256), 2.0, 1.25, 0.6);
  const double c1 = kGated ? 1e30 : rounds(tiles(256, 192), 1.6, 1.0, 0.4);
  const double c2 = rounds(tiles(128, 256), 1.15, 0.75, 0.35);
  const double c3 = kGated ? 1e30 : rounds(tiles(128, 192), 0.9, 0.52, 0.34);
  const double c4 = rounds(tiles(128, 128), 0.66, 0.36, 0.26);
  auto least = [&](double c) {
    return c <= c0 && c <= c1 && c <= c2 && c <= c3 && c <= c4 && c <= small;
  };
  a.split = 1;
  if (least(c0)) return run<4, 2, 2, 4, 2, kGated>(a, mul, st);
  if (least(c2)) return run<2, 4, 2, 2, 2, kGated>(a, mul, st);
  if constexpr (kGated) {
    if (least(c4)) return run<4, 2, 1, 2, 4, kGated>(a, mul, st);
  } else {
    if (least(c1)) return run<4, 2, 2, 3, 2, kGated>(a, mul, st);
    if (least(c3)) return run<4, 2, 1, 3, 3, kGated>(a, mul, st);
    if (least(c4)) return run<2, 4, 2, 1, 3, kGated>(a, mul, st);
  }
  double best = D * small;
  for (int s = 2; s <= 8 && t * s <= 256 && D >= 2 * s; ++s) {
    const double sums = (double)s * (double)a.T * a.Np;
    const double us = (double)D / s * one(t * s) + 1.5 + sums * 2.6e-6;
    if (us < best && sums * 4.0 <= (double)kPartialBytes) {
      best = us;
      a.split = s;
    }
  }
  if (a.split > 1) {
    const hipError_t e = run<2, 2, 1, 2, 3, kGated, true>(a, mul, st);
    return e == hipSuccess ? join<kGated>(a, mul, st) : e;
  }
  if constexpr (!kGated) {
    if (mul == kFp8 && t <= 256) return run_as<2, 4, 1, 1, 5, kFp8, false, false>(a, st);
  }
  return run<2, 2, 1, 2, 3, kGated>(a, mul, st);
}

}  // namespace

hipError_t launch_linear_tiled(const int8_t *q, int64_t T, const int8_t *w, int K, int Np,
                               bool gated, bool fp8, const Epilogue &ep, void *partial,
                               hipStream_t st) {
  TiledLinear a{};
  a.q = q; a.T = T; a.w = w; a.Kp = row_pitch(K); a.Np = Np; a.ep = ep;
  a.partial = static_cast<int32_t *>(partial);
  // What ends as fp32 gets fp32 sums; so do the hidden rows, whose codes would move.
  const int mul = !fp8 ? kInt8 : gated || ep.out_f32 ? kFp8Exact : kFp8;
  return gated ? pick<true>(a, mul, st) : pick<false>(a, mul, st);
}

}  // namespace moe
