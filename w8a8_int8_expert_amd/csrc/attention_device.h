// attention_device.h -- device building blocks of attention over the paged cache:
// where the elements of a staged tile lie, the fragments of the matrix instructions,
// and the conversion of codes. Included by the HIP sources only.
#pragma once

#include "attention_internal.h"
#include "row_device.h"

namespace moe {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef v2i v2i_e2 __attribute__((aligned(2)));

// Running maximum before the first key: finite, so that no difference of two is NaN, and not
// above any score.
constexpr float kNoMax = -3.402823466e38f;
// The maximum that a piece leaves for a row that sees keys in it, but of whose scores every
// one is -inf: just above kNoMax. A sum of 0 with it, of all pieces, is a softmax of NaN; a row
// that sees no key gets zeros.
constexpr float kSeenMax = -0x1.fffffcp127f;
__device__ __forceinline__ float inverse_sum(float l, float m) {
  return l != 0.0f ? 1.0f / l : m > kNoMax ? NAN : 0.0f;
}
// The maximum m of a row with sum l that sees the places [from, to) of a piece, in pages that
// exist or not. (A sum is seldom 0: nothing is kept for this while the keys are taken.)
__device__ __forceinline__ float seen_max(float m, float l, const CacheView &c,
                                          const int32_t *table, int from, int to) {
  if (l != 0.0f || from >= to) return m;
  for (int i = from >> c.log2_page; i << c.log2_page < to; ++i)
    if ((uint32_t)table[i] < (uint32_t)c.num_pages) return kSeenMax;
  return m;
}

__device__ __forceinline__ v4f mfma16bf(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A word that the kernel reads through the scalar cache (constant while it runs):
// a vector load here would wait for the tile loads in flight.
__device__ __forceinline__ int scalar_word(const int32_t *p, int64_t i) {
  return ((const __attribute__((address_space(4))) int32_t *)(uintptr_t)p)[i];
}

// This lane's value and that of lane l ^ 32, in the order of the halves.
struct Two {
  float lo, hi;
};
__device__ __forceinline__ Two halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return Two{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ float halves_max(float v) {
  const Two t = halves(v);
  return fmaxf(t.lo, t.hi);
}
__device__ __forceinline__ float halves_sum(float v) {
  const Two t = halves(v);
  return t.lo + t.hi;
}
// Largest of the four 16-lane groups' values, and their sum, in every lane.
__device__ __forceinline__ float groups_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return halves_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float groups_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return halves_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Eight codes as bf16, exactly.
template <int kFormat>
__device__ __forceinline__ v8bf code8_bf16(int lo, int hi) {
  if constexpr (kFormat == MOE_W8A8_FORMAT_FP8) return codes_bf16(lo, hi);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = i < 2 ? lo : hi, at = 16 * (i & 1);
    const float a = (float)(int8_t)(s >> at), b = (float)(int8_t)(s >> (at + 8));
    // 8 bits of an integer fit bf16's significand: the upper halves are the values
    w[i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  }
  return __builtin_bit_cast(v8bf, v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]});
}

// Values that are not finite: whether a fragment holds one, the fragment with those
// zeroed, and marks of them. A sum of marks of up to 63 keys says how many of each
// kind there were: +inf counts 1, -inf 64, NaN 4096.
__device__ __forceinline__ bool any_odd(v8bf v) {
  const v4i w = __builtin_bit_cast(v4i, v);
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r |= (w[i] & 0x7f80) == 0x7f80 || (w[i] & 0x7f800000) == 0x7f800000;
  return r;
}
template <bool kMarks>
__device__ __forceinline__ v8bf odd_part(v8bf v) {
  const v4i w = __builtin_bit_cast(v4i, v);
  v4i r = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int h = w[j / 2] >> 16 * (j & 1) & 0xffff;
    const bool odd = (h & 0x7f80) == 0x7f80;
    const int mark = h & 0x7f ? 0x4580 : h & 0x8000 ? 0x4280 : 0x3f80;  // 4096, 64, 1
    const int x = kMarks ? (odd ? mark : 0) : (odd ? 0 : h);
    r[j / 2] |= x << 16 * (j & 1);
  }
  return __builtin_bit_cast(v8bf, r);
}
// A result with the kinds that a sum of marks counts added to it.
__device__ __forceinline__ float add_odd(float v, float marks) {
  const int n = (int)marks;
  if (n & 63) v += INFINITY;
  if (n >> 6 & 63) v -= INFINITY;
  return n >> 12 ? NAN : v;
}

// A tile of kKeys keys (or values) of one kv head in LDS: rows of D elements, as
// they lie in the cache, but with the 16-byte chunks of a row exchanged among
// themselves so that the lanes of a fragment load meet different banks. Keys are read
// a chunk from each of 16 rows; values transposed, 16 elements of 4 (8-bit: 8) rows.
template <int D, int kFormat, int kKeys_ = 32>
struct Tile {
  static constexpr int kKeys = kKeys_;
  static constexpr bool k8 = kFormat != kBf16Cache;
  static constexpr int kRow = D * (k8 ? 1 : 2);  // bytes
  static constexpr int kChunks = kRow / 16;
  static constexpr int kBytes = kKeys * kRow;
  static constexpr int kLoads = kBytes / 1024;  // wavefront loads of 1 KB

  // Chunk position of chunk c of row r (its own inverse: c from the position). LDS serves
  // 256 bytes at once, 16 chunks in different columns of that width: of keys, one chunk of
  // each of 16 rows; of 16-bit values, two (kWide: four) neighbours of each of 8 (4) rows;
  // of 8-bit values, one of each of the 16 rows that two lane groups take.
  static constexpr int kWin = kChunks < 16 ? 16 / kChunks : 1;  // rows of such a width
  static constexpr int kMask = kChunks < 16 ? kChunks - 1 : 15;
  static __device__ __forceinline__ int key_chunk(int r, int c) { return c ^ (r / kWin & kMask); }
  template <bool kWide = false>
  static __device__ __forceinline__ int value_chunk(int r, int c) {
    if constexpr (k8) return c ^ (((r & 7) / kWin | (r >> 4 & 1) * (8 / kWin)) & kMask);
    if constexpr (kWide) return c ^ ((r & 3) / kWin << 2);
    return c ^ ((r & 7) / kWin << 1);
  }
  // Key fragment (A operand of 16 keys x 32 elements): lane l has key t16 + l % 16.
  // Which elements step s holds is the same for the queries: query_at.
  static __device__ __forceinline__ v8bf key(const char *tile, int t16, int s, int lane) {
    const int r = t16 + (lane & 15), g = lane >> 4;
    return *reinterpret_cast<const v8bf *>(tile + r * kRow + key_chunk(r, 4 * s + g) * 16);
  }
  // two steps' fragments from one chunk of codes
  static __device__ __forceinline__ void key2(const char *tile, int t16, int s2, int lane, v8bf *f) {
    const int r = t16 + (lane & 15), g = lane >> 4;
    const v4i w = *reinterpret_cast<const v4i *>(tile + r * kRow + key_chunk(r, 4 * s2 + g) * 16);
    f[0] = code8_bf16<kFormat>(w[0], w[1]);
    f[1] = code8_bf16<kFormat>(w[2], w[3]);
  }
  static __device__ __forceinline__ int query_at(int s, int lane) {
    const int g = lane >> 4;
    return k8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
  }
  // Value fragment (A operand of 16 elements x 32 keys, of keys r0 .. r0 + 31): lane l
  // has element 16 dt + l % 16; its eight keys are 4g .. 4g+3 and 16+4g .. 16+4g+3
  // (g = l / 16), which are the keys whose scores the lane holds after the first
  // product, so that probabilities go from one product to the next in place.
  static __device__ __forceinline__ v8bf value(const char *tile, int r0, int dt, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (k8) {
      typedef __attribute__((address_space(3))) v2i L;
      const int j = i >> 1, r = r0 + 4 * g + (j & 3) + 16 * (j >> 2);
      const v2i w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (L *)(tile + r * kRow + value_chunk(r, dt) * 16 + (i & 1) * 8));
      return code8_bf16<kFormat>(w[0], w[1]);
    } else {
      typedef __attribute__((address_space(3))) v4s L;
      const int r = r0 + 4 * g + (i >> 2), c = 2 * dt + ((i >> 1) & 1), o = (i & 1) * 8;
      const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (L *)(tile + r * kRow + value_chunk(r, c) * 16 + o));
      const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (L *)(tile + (r + 16) * kRow + value_chunk(r + 16, c) * 16 + o));
      return __builtin_bit_cast(
          v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

}  // namespace moe
