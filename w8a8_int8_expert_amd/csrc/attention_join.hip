// attention_join.hip -- joins the pieces that attention's keys were cut into: of each
// row, results o with their maxima m and sums l,
//   out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,  M = max m_p,
// taken along as a running maximum so that nothing waits for all the m_p first.
//
// One launch for both kernels' partial results. A slot's number finds its row block
// again; the pieces of a block share its rows. A row's elements are taken by D / 4
// lanes. Few rows have many pieces: all the block's groups of lanes take them in turn, so
// that their loads are in flight at once. Of many rows each group takes its own, and two
// blocks share a slot's: 75 MB in 24 us (37 with pieces shared out as of few rows), a few
// rows of up to 64 pieces in 4 to 6.
#include "attention_device.h"
#include "attention_work.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <bool kFew, int D, int kKeys, int kRows>
__device__ __forceinline__ void join_unit(const AttnArgs &a, const BatchView &bt, const Unit &un,
                                          const Partial &part, int h, int share, char *lds) {
  constexpr int kLanes = D / 4, kGroups = kThreads / kLanes;
  constexpr int kWays = kFew ? kGroups : 1, kTake = kGroups / kWays;  // rows at once
  struct Got {
    v4f o;
    float m, l;
  };
  Got *const got = reinterpret_cast<Got *>(lds);
  const int tid = threadIdx.x, lane = tid % kLanes, group = tid / kLanes;
  const int way = group % kWays, sub = group / kWays;
  const int r0 = un.block * kRows;
  const int rows = un.w.rows - r0 < kRows ? un.w.rows - r0 : kRows;
  const int64_t at0 = ((int64_t)h * part.slots + un.slot - un.piece) * kRows;
  // this piece's share of the rows
  constexpr int kShares = kFew ? 1 : 2;
  const int each = (rows + kShares * un.pieces - 1) / (kShares * un.pieces);
  const int from = (kShares * un.piece + share) * each, to = from + each < rows ? from + each : rows;
  for (int r = from; r < to; r += kTake) {
    const bool there = r + sub < to;
    const int row = there ? r + sub : to - 1;
    float m = kNoMax, l = 0.0f;
    v4f v = {0, 0, 0, 0};
#pragma unroll 4
    for (int p = way; p < un.pieces; p += kWays) {
      const int64_t at = at0 + (int64_t)p * kRows + row;
      const float pm = part.ml[2 * at], pl = part.ml[2 * at + 1];
      const v4f o = *reinterpret_cast<const v4f *>(part.o + at * D + 4 * lane);
      const float mm = fmaxf(m, pm), f = __builtin_amdgcn_exp2f(m - mm),
                  g = __builtin_amdgcn_exp2f(pm - mm);
      m = mm;
      l = l * f + pl * g;
      v = v * f + o * g;
    }
    if (kWays > 1) {
      __syncthreads();
      got[tid] = Got{v, m, l};
      __syncthreads();
    }
    if (way == 0 && there) {
#pragma unroll
      for (int w = 1; w < kWays; ++w) {
        const Got x = got[tid + w * kLanes];
        const float mm = fmaxf(m, x.m), f = __builtin_amdgcn_exp2f(m - mm),
                    g = __builtin_amdgcn_exp2f(x.m - mm);
        m = mm;
        l = l * f + x.l * g;
        v = v * f + x.o * g;
      }
      v *= inverse_sum(l, m);
      const int rr = r0 + row;
      uint16_t *dst = a.out + (int64_t)(un.w.s.start + rr / a.group) * a.ld_out +
                      (h * a.group + rr % a.group) * D + 4 * lane;
      *reinterpret_cast<v2i_e2 *>(dst) = v2i{(int)bf16x2(v[0], v[1]), (int)bf16x2(v[2], v[3])};
    }
  }
}

template <int D>
__global__ __launch_bounds__(kThreads) void join_kernel(AttnArgs a, int kv_heads, BatchView bt,
                                                        AttnPlan p, Partial few, Partial many) {
  __shared__ __attribute__((aligned(16))) char lds[kThreads * 32];
  const int h = blockIdx.x % kv_heads, x = blockIdx.x / kv_heads;
  if (x < p.row_target) {
    const Schedule<true, kFewKeys> s(a, bt, p.row_target, kLeastFew, kLeastFew);
    for (int u = x;; u += p.row_target) {
      const Unit un = s.template find<true>(a, bt, u);
      if (un.b < 0) break;
      if (p.row_tiles == 1) join_unit<true, D, kFewKeys, 16>(a, bt, un, few, h, 0, lds);
      else join_unit<true, D, kFewKeys, 32>(a, bt, un, few, h, 0, lds);
    }
  } else {
    const Schedule<false, kManyKeys<D>> s(a, bt, p.tile_target, kLeastMany<D>, 1);
    const int y = x - p.row_target;
    for (int u = y >> 1;; u += p.tile_target) {
      const Unit un = s.template find<true>(a, bt, u);
      if (un.b < 0) break;
      join_unit<false, D, kManyKeys<D>, kTileRows>(a, bt, un, many, h, y & 1, lds);
    }
  }
}

}  // namespace

hipError_t launch_attention_join(const AttnArgs &a, const CacheView &c, int D, const BatchView &b,
                                 const AttnPlan &p, float *partial, hipStream_t st) {
  const Partial few = partial_few(p, c.kv_heads, D, partial),
                many = partial_many(p, c.kv_heads, D, partial);
  const dim3 grid((p.row_target + 2 * p.tile_target) * c.kv_heads), block(kThreads);
  if (D == 64) return launch_kernel(join_kernel<64>, grid, block, st, {}, a, c.kv_heads, b, p, few, many);
  if (D == 128) return launch_kernel(join_kernel<128>, grid, block, st, {}, a, c.kv_heads, b, p, few, many);
  return launch_kernel(join_kernel<256>, grid, block, st, {}, a, c.kv_heads, b, p, few, many);
}

}  // namespace moe
