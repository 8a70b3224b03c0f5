// rope.hip -- norms of queries and keys for each head, the position rotation, and
// the write of keys and values into the paged cache, in one pass over the rows of
// the QKV projection. Bound by memory: a row is read once, queries and the cache's
// elements are written once (16384 tokens of 32 heads over 8 of 128, bf16: 403 MB in 84 us,
// 4.8 TB/s; INT8 and FP8 codes: 370 MB in 88 to 90). A few tokens take 5 to 6 us: the loads of
// ends, frequencies, page and rows are issued one after the other, though only the page
// depends on another one (the ends), and a token's heads are taken by one block in rounds.
//
// One block takes one token. Its sequence is found by the wavefronts' lanes, which
// compare the row with 64 sequence ends at once; the token's angles (shared by all
// heads) are taken once into LDS, in fp64 up to the turn's fraction: in fp32 the
// angle of place 10^6 is off by 0.03. D / 8 lanes then take a head, each two runs of
// four elements: the two halves of four rotated pairs where these lie rotary / 2
// apart, else eight neighbours, so that no element crosses lanes.
#include "attention_internal.h"
#include "row_device.h"

namespace moe {
namespace {

typedef v2i v2i_e2 __attribute__((aligned(2)));

template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <int kLanes>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = umax(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
}

// x / sqrt(mean x^2 + eps) over a head's lanes, times the weights.
template <int kLanes>
__device__ __forceinline__ void head_norm(float *x, const float *w, int o0, int o1, float eps) {
  constexpr float kInvD = 1.0f / (8 * kLanes);
  auto squares = [&]() {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += x[j] * x[j];
    return lanes_sum<kLanes>(s);
  };
  float ss = squares();
  // Squares that leave the fp32 range: the head is brought to about 1 by a power of two
  // first. At most 2^63: the square of the smallest number, 2^-133, is 2^-140 then, and that
  // over 256 elements still a number. Squares below 1e-28 are nothing beside an eps of 1e-20
  // or more (less than 2^-24 of it), and a smaller eps stays finite when it is lifted.
  if (!(ss < 1e38f) || (ss < 1e-28f && eps < 1e-20f)) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(x[j]));
    m = lanes_max<kLanes>(m);
    const int e = 127 - (int)(m >> 23);
    const float lift = m < 0x7f800000u ? ldexpf(1.0f, e > 63 ? 63 : e) : 1.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= lift;
    eps *= lift * lift;
    ss = squares();
  }
  const float r = 1.0f / sqrtf(ss * kInvD + eps);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] *= r;
  if (w) {
    const v4f a = *reinterpret_cast<const v4f_a4 *>(w + o0),
              b = *reinterpret_cast<const v4f_a4 *>(w + o1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] *= a[j];
      x[4 + j] *= b[j];
    }
  }
}

template <int D, int kFormat>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, CacheView c, BatchView bt) {
  constexpr int kLanes = D / 8, kHeads = 256 / kLanes;
  __shared__ float trig[2][D / 2];
  const int t = blockIdx.x, lane = threadIdx.x & 63;
  // the sequence whose rows hold this one
  int b = -1;
  Seq sq{};
  for (int b0 = 0; b0 < bt.num_seqs; b0 += 64) {
    const int i = b0 + lane;
    Seq s{};
    if (i < bt.num_seqs) s = seq_of(bt, i);
    const uint64_t hit = __ballot(i < bt.num_seqs && t >= s.start && t < s.start + s.n);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      b = b0 + l;
      sq.start = __builtin_amdgcn_readlane(s.start, l);
      sq.n = __builtin_amdgcn_readlane(s.n, l);
      sq.len = __builtin_amdgcn_readlane(s.len, l);
      break;
    }
  }
  if (b < 0) return;  // a row behind the last sequence
  const int place = sq.len - sq.n + (t - sq.start);
  const int R = a.rotary;
  if ((int)threadIdx.x < R / 2) {
    const double pos = a.positions ? (double)a.positions[t] : (double)place;
    // turns = pos * f / (2 pi), both products with their fp64 rounding errors, so that
    // what is left of a turn after many is as exact as of one
    const double f = a.inv_freq[threadIdx.x], k0 = 0x1.45f306dc9c883p-3, k1 = -0x1.6b01ec5417056p-57;
    const double x = pos * f, dx = fma(pos, f, -x);
    const double y = x * k0, dy = fma(x, k0, -y) + (x * k1 + dx * k0);
    const double turns = (y - rint(y)) + dy;
    float s, co;
    sincospif(2.0f * (float)turns, &s, &co);
    trig[0][threadIdx.x] = co;
    trig[1][threadIdx.x] = s;
  }
  __syncthreads();
  // where the token's keys and values go; -1: nowhere
  int64_t page = -1;
  if (place >= 0) {
    const int p = bt.table[(int64_t)b * bt.ld_table + (place >> c.log2_page)];
    if ((uint32_t)p < (uint32_t)c.num_pages) page = p;
  }
  const int at = place & ((1 << c.log2_page) - 1);
  const int l = threadIdx.x % kLanes;
  const bool turn = 8 * l < R, split = turn && !a.interleaved;
  const int o0 = split ? 4 * l : 8 * l, o1 = split ? R / 2 + 4 * l : 8 * l + 4;
  v4f co = {1, 1, 1, 1}, si = {0, 0, 0, 0};
  if (turn) {
    co = *reinterpret_cast<const v4f *>(&trig[0][4 * l]);
    si = *reinterpret_cast<const v4f *>(&trig[1][4 * l]);
  }
  const int Hq = a.heads, Hk = c.kv_heads, all = Hq + 2 * Hk;
  const uint16_t *row = a.qkv + (int64_t)t * a.ld_qkv;
  for (int h = threadIdx.x / kLanes; h < all; h += kHeads) {
    const uint16_t *src = row + h * D;
    const v2i r0 = *reinterpret_cast<const v2i_e2 *>(src + o0),
              r1 = *reinterpret_cast<const v2i_e2 *>(src + o1);
    float x[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      x[2 * j] = __uint_as_float((uint32_t)r0[j] << 16);
      x[2 * j + 1] = __uint_as_float((uint32_t)r0[j] & 0xffff0000u);
      x[4 + 2 * j] = __uint_as_float((uint32_t)r1[j] << 16);
      x[5 + 2 * j] = __uint_as_float((uint32_t)r1[j] & 0xffff0000u);
    }
    const bool value = h >= Hq + Hk;
    if (!value) {
      if (a.norm) head_norm<kLanes>(x, h < Hq ? a.q_weight : a.k_weight, o0, o1, a.eps);
      if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // (selects, not an index that varies: x stays in registers)
          const float p = a.interleaved ? x[2 * j] : x[j];
          const float q = a.interleaved ? x[2 * j + 1] : x[4 + j];
          const float y = p * co[j] - q * si[j], z = q * co[j] + p * si[j];
          if (a.interleaved) {
            x[2 * j] = y;
            x[2 * j + 1] = z;
          } else {
            x[j] = y;
            x[4 + j] = z;
          }
        }
      }
    }
    if (h < Hq) {
      uint16_t *dst = a.q + (int64_t)t * a.ld_q + h * D;
      *reinterpret_cast<v2i_e2 *>(dst + o0) = v2i{(int)bf16x2(x[0], x[1]), (int)bf16x2(x[2], x[3])};
      *reinterpret_cast<v2i_e2 *>(dst + o1) = v2i{(int)bf16x2(x[4], x[5]), (int)bf16x2(x[6], x[7])};
      continue;
    }
    const int kh = value ? h - Hq - Hk : h - Hq;
    const int64_t slot = (int64_t)kh << c.log2_page | at;
    char *base = (value ? c.v : c.k) + page * c.page_bytes;
    if constexpr (kFormat == kBf16Cache) {
      if (page >= 0) {
        uint16_t *dst = reinterpret_cast<uint16_t *>(base) + slot * D;
        // values as they are, bit for bit
        *reinterpret_cast<v2i *>(dst + o0) =
            value ? r0 : v2i{(int)bf16x2(x[0], x[1]), (int)bf16x2(x[2], x[3])};
        *reinterpret_cast<v2i *>(dst + o1) =
            value ? r1 : v2i{(int)bf16x2(x[4], x[5]), (int)bf16x2(x[6], x[7])};
      }
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = umax(m, abs_bits(x[j]));
      const RowCode rc = row_code(lanes_max<kLanes>(m), kFormat == MOE_W8A8_FORMAT_FP8);
      if (page >= 0) {
        char *dst = base + slot * D;
        *reinterpret_cast<uint32_t *>(dst + o0) =
            row_codes4(x, rc, kFormat == MOE_W8A8_FORMAT_FP8);
        *reinterpret_cast<uint32_t *>(dst + o1) =
            row_codes4(x + 4, rc, kFormat == MOE_W8A8_FORMAT_FP8);
        if (l == 0) (value ? c.v_scale : c.k_scale)[page * c.scale_stride + slot] = rc.scale;
      }
    }
  }
}

template <int D>
hipError_t launch(const RopeArgs &a, const CacheView &c, int format, const BatchView &b,
                  hipStream_t st) {
  const dim3 grid((unsigned)b.T), block(256);
  if (format == kBf16Cache)
    return launch_kernel(rope_kernel<D, kBf16Cache>, grid, block, st, {}, a, c, b);
  if (format == MOE_W8A8_FORMAT_FP8)
    return launch_kernel(rope_kernel<D, MOE_W8A8_FORMAT_FP8>, grid, block, st, {}, a, c, b);
  return launch_kernel(rope_kernel<D, MOE_W8A8_FORMAT_INT8>, grid, block, st, {}, a, c, b);
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs &a, const CacheView &c, int D, int format,
                               const BatchView &b, hipStream_t st) {
  if (D == 64) return launch<64>(a, c, format, b, st);
  if (D == 128) return launch<128>(a, c, format, b, st);
  return launch<256>(a, c, format, b, st);
}

}  // namespace moe
