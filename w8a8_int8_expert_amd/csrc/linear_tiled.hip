// linear_tiled.hip -- W8A8 products of many tokens, bound by the matrix cores
// and by feeding them.
//
// "MiniMax-M3 W8A8 inference on K100AI" (mhpq.cn/news/1068415) §1.2, §4.3.
//
// A block computes BM tokens x BN packed weight rows. Tokens are read row-major
// through a ring of two 128-k stages (whole 128-byte lines, XOR-swizzled in
// LDS so that an operand read is free of bank conflicts), weights through a
// ring of four 64-k stages of fragment tiles, both by direct global -> LDS
// loads issued up to three steps ahead. WM x WN wavefronts own MI x NJ
// accumulators of 32 x 32 each. INT8 multiplies on the 32x32x32 instruction
// (the 16x16x64 form reaches half its rate), FP8 on 32x32x64.
//
// Tiles are numbered (N group, M tile, N tile in group), and each XCD takes a
// contiguous eighth of that order, so that the blocks that run together on one
// L2 share token and weight panels.
//
// Few tiles: blockIdx.y cuts K into `split` parts; each writes its raw sums
// and a second launch adds them in order and finishes the columns.
#include "epilogue_device.h"

namespace moe {
namespace {

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

template <int WM, int WN, int MI, int NJ, bool kF8, bool kGated, bool kSplit>
__global__ __launch_bounds__(64 * WM * WN, 1) void linear_tiled_kernel(const TiledLinear a) {
  typedef typename Acc32<kF8>::T Acc;
  constexpr int W = WM * WN, BM = WM * MI * 32, BN = WN * NJ * 32;
  constexpr int kA2 = BM * 128, kB = BN * 64;         // one stage of each ring
  constexpr int kALoads = BM / 8 / W, kBLoads = BN / 16 / W;
  static_assert(kALoads * W * 8 == BM && kBLoads * W * 16 == BN, "load split");
  constexpr int kRing = 2 * kA2 + 4 * kB;
  // Epilogue: 16 rows x the wavefront's columns per pass, pitch padded by 8
  // words so that the two 32-lane halves (rows r and r + 4) use other banks.
  constexpr int kPitch = NJ * 32 + 8, kSlice = 16 * kPitch * 4;
  constexpr int kScaleAt = W * kSlice;
  constexpr int kLds = kRing > kScaleAt + BM * 4 ? kRing : kScaleAt + BM * 4;
  __shared__ __attribute__((aligned(1024))) int8_t lds[kLds];

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
  // This block's 128-k stages [d0, d1).
  const int D = a.Kp >> 7;
  int d0 = 0, d1 = D;
  if (kSplit) {
    d0 = (int)((int64_t)D * blockIdx.y / a.split);
    d1 = (int)((int64_t)D * (blockIdx.y + 1) / a.split);
  }
  const int KT = 2 * (d1 - d0);

  const int8_t *asrc[kALoads];
#pragma unroll
  for (int t = 0; t < kALoads; ++t) {
    const int i = kALoads * wave + t;
    int r = 8 * i + (lane >> 3);
    r = r < rows ? r : rows - 1;  // rows past T: computed, never stored
    asrc[t] = a.q + (m0 + r) * a.Kp + (size_t)d0 * 128 +
              (((lane & 7) ^ ((4 * (i & 1) + (lane >> 4)) & 7)) << 4);
  }
  const int8_t *bsrc[kBLoads];
#pragma unroll
  for (int t = 0; t < kBLoads; ++t) {
    int p = (n0 >> 4) + kBLoads * wave + t;
    p = p < (a.Np >> 4) ? p : (a.Np >> 4) - 1;  // columns past Np: never stored
    bsrc[t] = a.w + frag_tile(p, 2 * d0, a.Kp) + lane * 16;
  }
  auto issue_a = [&](int d) {
    int8_t *st = lds + (d & 1) * kA2;
#pragma unroll
    for (int t = 0; t < kALoads; ++t)
      dma16(asrc[t] + (size_t)d * 128,
            __builtin_amdgcn_readfirstlane(lds_addr(st + (kALoads * wave + t) * 1024)));
  };
  auto issue_b = [&](int kt) {
    int8_t *st = lds + 2 * kA2 + (kt & 3) * kB;
#pragma unroll
    for (int t = 0; t < kBLoads; ++t)
      dma16(bsrc[t] + ((size_t)kt << 10),
            __builtin_amdgcn_readfirstlane(lds_addr(st + (kBLoads * wave + t) * 1024)));
  };

  Acc acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int c = 0; c < NJ; ++c)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][c][v] = 0;

  const int frag = (((lane >> 5) * 16) + (lane & 15)) * 16 + ((lane & 31) >> 4) * 1024;
  const int boff = wn * NJ * 2048 + frag;
  int arow[MI], axor[2][2];
#pragma unroll
  for (int i = 0; i < MI; ++i) arow[i] = ((wm * MI + i) * 32 + (lane & 31)) * 128;
#pragma unroll
  for (int par = 0; par < 2; ++par)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      axor[par][h] = ((4 * par + 2 * h + (lane >> 5)) ^ ((lane >> 1) & 7)) << 4;
  const bool skip = wm * MI * 32 >= rows;  // no row of this wavefront exists

  auto step = [&](const int8_t *as, int par, const int8_t *bst) {
    v4i af[MI][2];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        af[i][h] = *reinterpret_cast<const v4i *>(as + arow[i] + axor[par][h]);
    v4i b0 = *reinterpret_cast<const v4i *>(bst + boff);
    v4i b1 = *reinterpret_cast<const v4i *>(bst + boff + 512);
#pragma unroll
    for (int c = 0; c < NJ; ++c) {
      v4i n0v = b0, n1v = b1;
      if (c + 1 < NJ) {
        n0v = *reinterpret_cast<const v4i *>(bst + boff + (c + 1) * 2048);
        n1v = *reinterpret_cast<const v4i *>(bst + boff + (c + 1) * 2048 + 512);
      }
      if constexpr (kF8) {
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][c] = mfma32f8(af[i][0], af[i][1], b0, b1, acc[i][c]);
      } else {
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][c] = mfma32(af[i][0], b0, acc[i][c]);
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][c] = mfma32(af[i][1], b1, acc[i][c]);
      }
      b0 = n0v;
      b1 = n1v;
    }
    // The A operands and two column fragments first, then each fragment's
    // instructions followed by the reads of the fragment two ahead.
    constexpr int kM = kF8 ? MI : 2 * MI;
    if constexpr (NJ >= 2) {
      __builtin_amdgcn_sched_group_barrier(0x100, 2 * MI + 4, 0);
#pragma unroll
      for (int c = 0; c < NJ - 2; ++c) {
        __builtin_amdgcn_sched_group_barrier(0x008, kM, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 2 * kM, 0);
    }
  };

  // Issue order: B(0), A(0), B(1), B(2); then at step kt, after the wait,
  // A(kt/2 + 1) on even kt and B(kt + 3). At step kt, B(kt) and A(kt/2) must
  // have landed: what may still be in flight is B(kt+1), B(kt+2) and, on odd
  // kt, A((kt+1)/2). KT is even; the last three steps drain all.
  issue_b(0);
  issue_a(0);
  issue_b(1);
  if (KT > 2) issue_b(2);
  for (int kt = 0; kt < KT; ++kt) {
    if (kt + 3 < KT) {
      if (kt & 1) wait_barrier<2 * kBLoads + kALoads>();
      else wait_barrier<2 * kBLoads>();
    } else {
      wait_barrier<0>();
    }
    if (!(kt & 1) && kt + 2 < KT) issue_a((kt >> 1) + 1);
    if (kt + 3 < KT) issue_b(kt + 3);
    if (!skip) step(lds + ((kt >> 1) & 1) * kA2, kt & 1, lds + 2 * kA2 + (kt & 3) * kB);
  }
  wait_barrier<0>();  // every wavefront is done with the rings

  // Epilogue through the wavefront's own slice of the rings, 16 rows a pass.
  // Lane holds column lane%32 of each 32 x 32 accumulator and rows 8*(v/4) +
  // 4*(lane/32) + v%4.
  const Epilogue &ep = a.ep;
  float *rs = reinterpret_cast<float *>(lds + kScaleAt);
  if (!kSplit) {
    for (int i = threadIdx.x; i < BM; i += 64 * W) rs[i] = i < rows ? ep.row_scale[m0 + i] : 0.0f;
    __syncthreads();
  }
  if (skip) return;
  float *slice = reinterpret_cast<float *>(lds + wave * kSlice);
  const int nw = n0 + wn * NJ * 32;  // first packed row of this wavefront
  const int rl = 4 * (lane >> 5);
  float sc[NJ];
#pragma unroll
  for (int c = 0; c < NJ; ++c) {
    const int n = nw + 32 * c + (lane & 31);
    sc[c] = !kSplit && n < a.Np ? ep.scale[n] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int vh = 0; vh < 2; ++vh) {
      const int mr = (wm * MI + i) * 32 + 16 * vh;  // first row of the pass
      if (mr >= rows) return;
      v4f rsc[2];
      if (!kSplit) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
          rsc[g] = *reinterpret_cast<const v4f *>(rs + mr + 8 * g + rl);
      }
#pragma unroll
      for (int vv = 0; vv < 8; ++vv) {
        const int v = 8 * vh + vv, r = 8 * (vv >> 2) + rl + (vv & 3);
        if constexpr (kSplit) {
#pragma unroll
          for (int c = 0; c < NJ; ++c) {
            const auto e = acc[i][c][v];
            slice[r * kPitch + 32 * c + (lane & 31)] = __builtin_bit_cast(float, e);
          }
        } else if constexpr (kGated) {
          const float x = rsc[vv >> 2][vv & 3];
          uint32_t m = 0;
#pragma unroll
          for (int c = 0; c < NJ; c += 2) {
            const float h = swiglu((float)acc[i][c][v] * x * sc[c],
                                   (float)acc[i][c + 1][v] * x * sc[c + 1]);
            slice[r * kPitch + 16 * c + (lane & 31)] = h;
            m = umax(m, nw / 2 + 16 * c + (lane & 31) < ep.N ? abs_bits(h) : 0u);
          }
          m = half_wave_max(m);
          if ((lane & 31) == 31) slice[r * kPitch + NJ * 32] = __uint_as_float(m);
        } else {
          const float x = rsc[vv >> 2][vv & 3];
#pragma unroll
          for (int c = 0; c < NJ; ++c)
            slice[r * kPitch + 32 * c + (lane & 31)] = (float)acc[i][c][v] * x * sc[c];
        }
      }
      const int left = rows - mr;  // rows of the pass that exist
      if constexpr (kSplit) {
        int32_t *part = a.partial + (size_t)blockIdx.y * a.T * a.Np;
        for (int j = lane; j < 16 * NJ * 8; j += 64) {
          const int r = j / (NJ * 8), c4 = j % (NJ * 8) * 4;
          if (r < left && nw + c4 < a.Np)
            *reinterpret_cast<v4f *>(part + (m0 + mr + r) * a.Np + nw + c4) =
                *reinterpret_cast<const v4f *>(slice + r * kPitch + c4);
        }
      } else if constexpr (kGated) {
        if (lane < 16 && lane < left)
          atomicMax(ep.amax + m0 + mr + lane, __float_as_uint(slice[lane * kPitch + NJ * 32]));
        // h columns nw/2 .. + 16 NJ; h rows have the pitch of code rows, so
        // whole 32-column runs exist
        float *h = static_cast<float *>(ep.out);
        for (int j = lane; j < 16 * NJ * 4; j += 64) {
          const int r = j / (NJ * 4), c4 = j % (NJ * 4) * 4;
          if (r < left && nw + 2 * c4 < a.Np)
            *reinterpret_cast<v4f *>(h + (m0 + mr + r) * ep.ld_out + nw / 2 + c4) =
                *reinterpret_cast<const v4f *>(slice + r * kPitch + c4);
        }
      } else {
        for (int j = lane; j < 16 * NJ * 4; j += 64) {
          const int r = j / (NJ * 4), c8 = j % (NJ * 4) * 8;
          float v[8];
          const v4f x = *reinterpret_cast<const v4f *>(slice + r * kPitch + c8);
          const v4f y = *reinterpret_cast<const v4f *>(slice + r * kPitch + c8 + 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = x[k];
            v[4 + k] = y[k];
          }
          if (r < left) finish_columns<8>(ep, m0 + mr + r, nw + c8, v);
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
    atomicMax(ep.amax + t, m);
  } else {
    finish_columns<8>(ep, t, c8, v);
  }
}

template <int WM, int WN, int MI, int NJ, bool kGated>
hipError_t run(TiledLinear a, bool fp8, hipStream_t st) {
  constexpr int BM = WM * MI * 32, BN = WN * NJ * 32;
  a.mt = (int)((a.T + BM - 1) / BM);
  a.nt = (a.Np + BN - 1) / BN;
  a.gn = a.nt < 4 ? a.nt : 4;
  const int64_t tiles = (int64_t)a.mt * a.nt;
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)a.split);
  const dim3 block(64 * WM * WN);
  const Timing tm{};
  if (a.split > 1) {
    const hipError_t e =
        fp8 ? launch_kernel(linear_tiled_kernel<WM, WN, MI, NJ, true, kGated, true>, grid, block,
                            st, tm, a)
            : launch_kernel(linear_tiled_kernel<WM, WN, MI, NJ, false, kGated, true>, grid, block,
                            st, tm, a);
    if (e != hipSuccess) return e;
    const int64_t n = a.T * (kGated ? a.Np / 16 : a.Np / 8);
    const dim3 jgrid((unsigned)((n + 255) / 256));
    if (fp8)
      return launch_kernel(linear_join_kernel<true, kGated>, jgrid, dim3(256), st, tm, a);
    return launch_kernel(linear_join_kernel<false, kGated>, jgrid, dim3(256), st, tm, a);
  }
  if (fp8)
    return launch_kernel(linear_tiled_kernel<WM, WN, MI, NJ, true, kGated, false>, grid, block, st,
                         tm, a);
  return launch_kernel(linear_tiled_kernel<WM, WN, MI, NJ, false, kGated, false>, grid, block, st,
                       tm, a);
}

template <bool kGated>
hipError_t pick(TiledLinear a, bool fp8, hipStream_t st) {
  const int64_t t256 = ((a.T + 255) / 256) * ((a.Np + 255) / 256);
  a.split = 1;
  if (t256 >= 192) return run<4, 2, 2, 4, kGated>(a, fp8, st);  // 256 x 256
  const int64_t t128 = ((a.T + 127) / 128) * ((a.Np + 127) / 128);
  if (t128 >= 128) return run<2, 2, 2, 2, kGated>(a, fp8, st);  // 128 x 128
  // 64 x 128, K split until the chip is covered
  const int64_t t64 = ((a.T + 63) / 64) * ((a.Np + 127) / 128);
  const int D = a.Kp / 128;
  while (a.split < 8 && t64 * a.split < 256 && D / (a.split + 1) >= 4 &&
         (size_t)(a.split + 1) * a.T * a.Np * 4 <= kPartialBytes)
    ++a.split;
  return run<2, 2, 1, 2, kGated>(a, fp8, st);
}

}  // namespace

hipError_t launch_linear_tiled(const int8_t *q, int64_t T, const int8_t *w, int K, int Np,
                               bool gated, bool fp8, const Epilogue &ep, void *partial,
                               hipStream_t st) {
  TiledLinear a{};
  a.q = q; a.T = T; a.w = w; a.Kp = row_pitch(K); a.Np = Np; a.ep = ep;
  a.partial = static_cast<int32_t *>(partial);
  return gated ? pick<true>(a, fp8, st) : pick<false>(a, fp8, st);
}

}  // namespace moe
