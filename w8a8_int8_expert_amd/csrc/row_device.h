// row_device.h -- device building blocks of the row operators: loads and
// stores of eight consecutive elements at any element alignment, and the
// per-token code rule of the block operators. Included by the HIP sources only.
#pragma once

#include "lds_dma.h"
#include "block_internal.h"

namespace moe {

// 16 and 8 bytes at the alignment of their elements. Rows may start anywhere
// (odd widths, strides): global memory takes such an access in one
// instruction, so an odd row moves as few instructions as an aligned one.
typedef v4i v4i_a2 __attribute__((aligned(2)));
typedef v2i v2i_a2 __attribute__((aligned(2)));
typedef v4f v4f_a4 __attribute__((aligned(4)));

// Eight elements c .. c+7 of a row of n (those past it are 0), in two steps: the
// load, and what becomes of it. A chunk that ends past the row is loaded from
// the row's last eight elements and moved down, so that a row's odd end costs one
// load like any other chunk (element by element it held a whole block back:
// add_norm of 8192 rows of 4095 took 93 us, 4096 columns 46). Only a row of
// fewer than eight elements is loaded one by one. kOdd false: n is a multiple of
// eight, and nothing of this is needed (8192 x 4096, both norms, codes: 80 us, 87
// with it).
template <bool kOdd = true>
__device__ __forceinline__ v4i fetch8(const uint16_t *row, int c, int n) {
  if constexpr (!kOdd)
    return c < n ? *reinterpret_cast<const v4i_a2 *>(row + c) : v4i{0, 0, 0, 0};
  if (n >= 8) return *reinterpret_cast<const v4i_a2 *>(row + (c < n - 8 ? c : n - 8));
  v4i r = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < n) r[j / 2] |= (int)((uint32_t)row[c + j] << (16 * (j & 1)));
  return r;
}
template <bool kOdd = true>
__device__ __forceinline__ void unpack8(v4i r, int c, int n, float *o) {
  const int over = c + 8 - n;  // elements past the row
  if (kOdd && over > 0 && n >= 8) {
    if (over & 4) r = v4i{r[2], r[3], 0, 0};
    if (over & 2) r = v4i{r[1], r[2], r[3], 0};
    if (over & 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = (int)(((uint32_t)r[i] >> 16) | (i < 3 ? (uint32_t)r[i + 1] << 16 : 0u));
    }
    if (over >= 8) r = v4i{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float((uint32_t)r[i] << 16);
    o[2 * i + 1] = __uint_as_float((uint32_t)r[i] & 0xffff0000u);
  }
}
struct Floats8 {
  v4f a, b;
};
template <bool kOdd = true>
__device__ __forceinline__ Floats8 fetch8(const float *row, int c, int n) {
  Floats8 r;
  if constexpr (!kOdd) {
    r = Floats8{v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
    if (c < n) {
      r.a = *reinterpret_cast<const v4f_a4 *>(row + c);
      r.b = *reinterpret_cast<const v4f_a4 *>(row + c + 4);
    }
    return r;
  }
  if (n >= 8) {
    const float *p = row + (c < n - 8 ? c : n - 8);
    r.a = *reinterpret_cast<const v4f_a4 *>(p);
    r.b = *reinterpret_cast<const v4f_a4 *>(p + 4);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.a[j] = c + j < n ? row[c + j] : 0.0f;
      r.b[j] = c + 4 + j < n ? row[c + 4 + j] : 0.0f;
    }
  }
  return r;
}
template <bool kOdd = true>
__device__ __forceinline__ void unpack8(Floats8 r, int c, int n, float *o) {
  const int over = c + 8 - n;
  if (kOdd && over > 0 && n >= 8) {
    if (over & 4) r = Floats8{r.b, v4f{0, 0, 0, 0}};
    if (over & 2) r = Floats8{v4f{r.a[2], r.a[3], r.b[0], r.b[1]}, v4f{r.b[2], r.b[3], 0, 0}};
    if (over & 1) r = Floats8{v4f{r.a[1], r.a[2], r.a[3], r.b[0]}, v4f{r.b[1], r.b[2], r.b[3], 0}};
    if (over >= 8) r = Floats8{v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[j] = r.a[j];
    o[4 + j] = r.b[j];
  }
}
template <bool kOdd = true, typename T>
__device__ __forceinline__ void load8(const T *row, int c, int n, float *o) {
  unpack8<kOdd>(fetch8<kOdd>(row, c, n), c, n, o);
}
// Two values rounded to bf16 (nearest, ties to even; NaN stays NaN) by the one
// hardware instruction.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2bf));
}
// Elements c .. c+7 of a row of n; a row's odd end in pieces of 4, 2 and 1.
template <bool kOdd = true>
__device__ __forceinline__ void store8(uint16_t *row, int c, int n, const float *v) {
  typedef uint32_t u32_a2 __attribute__((aligned(2)));
  uint16_t *p = row + c;
  const int rem = n - c;
  int w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = (int)bf16x2(v[2 * i], v[2 * i + 1]);
  if (rem >= 8) {
    *reinterpret_cast<v4i_a2 *>(p) = v4i{w[0], w[1], w[2], w[3]};
  } else if (kOdd && rem > 0) {
    if (rem & 4) {
      *reinterpret_cast<v2i_a2 *>(p) = v2i{w[0], w[1]};
      p += 4; w[0] = w[2]; w[1] = w[3];
    }
    if (rem & 2) {
      *reinterpret_cast<u32_a2 *>(p) = (uint32_t)w[0];
      p += 2; w[0] = w[1];
    }
    if (rem & 1) *p = (uint16_t)w[0];
  }
}
template <bool kOdd = true>
__device__ __forceinline__ void store8(float *row, int c, int n, const float *v) {
  typedef float v2f_a4 __attribute__((ext_vector_type(2), aligned(4)));
  float *p = row + c;
  const int rem = n - c;
  if (rem >= 8) {
    *reinterpret_cast<v4f_a4 *>(p) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f_a4 *>(p + 4) = v4f{v[4], v[5], v[6], v[7]};
  } else if (kOdd && rem > 0) {
    float w[4] = {v[0], v[1], v[2], v[3]};
    if (rem & 4) {
      *reinterpret_cast<v4f_a4 *>(p) = v4f{v[0], v[1], v[2], v[3]};
      p += 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = v[4 + i];
    }
    if (rem & 2) {
      *reinterpret_cast<v2f_a4 *>(p) = v2f_a4{w[0], w[1]};
      p += 2; w[0] = w[2];
    }
    if (rem & 1) *p = w[0];
  }
}

// |v| as its bits: NaN orders above infinity, infinity above every number, so
// an unsigned maximum keeps what is not finite.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Code rule of a row with largest |v| of bits `amax`: code = round(v * pre * rr),
// row scale `scale`; `ok` is false for a row that is not finite (codes 0,
// scale NaN). Below 2^-64 the row is lifted by 2^64 first (exact), where
// qmax / a would overflow or lose bits to a subnormal.
struct RowCode {
  float pre, rr, scale;
  bool ok;
};
__device__ __forceinline__ RowCode row_code(uint32_t amax, bool fp8) {
  const float qmax = fp8 ? kFp8Max : 127.0f;
  RowCode c;
  c.ok = amax < 0x7f800000u;
  const float a = __uint_as_float(amax);
  const bool tiny = a < 0x1p-64f;
  c.pre = tiny ? 0x1p64f : 1.0f;
  const float al = a * c.pre;
  c.rr = a > 0.0f ? qmax / al : 0.0f;
  c.scale = al / qmax * (tiny ? 0x1p-64f : 1.0f);
  if (!c.ok) c.scale = __uint_as_float(0x7fc00000u);
  return c;
}
__device__ __forceinline__ uint32_t row_codes4(const float *v, const RowCode &c, bool fp8) {
  const float t[4] = {v[0] * c.pre, v[1] * c.pre, v[2] * c.pre, v[3] * c.pre};
  return c.ok ? codes4(t, c.rr, fp8) : 0u;
}

// Sum over the wavefront in every lane, in a fixed order (DPP row shifts and
// broadcasts as wave_incl_scan; lane 63 holds the total).
__device__ __forceinline__ float wave_sum_f32(float v) {
  auto add = [](float x, int moved) { return x + __int_as_float(moved); };
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xF, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xF, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xF, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xF, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xA, 0xF, false));
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xC, 0xF, false));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ uint32_t wave_max_bits(uint32_t m) {
  return __float_as_uint(wave_max(__uint_as_float(m)));
}

// Hidden values h = silu(g) u of columns c .. c+7 (c a multiple of 8, `rem` of
// them exist, 0 past them) from a row of gate and up values in packed order:
// alternating runs of 32, whole ones also at the end.
__device__ __forceinline__ void hidden8(const float *gu, int c, int rem, float *o) {
  if (rem <= 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = 0.0f;
    return;
  }
  const v4f *p = reinterpret_cast<const v4f *>(gu + c / 32 * 64 + c % 32);
  const v4f g[2] = {p[0], p[1]}, u[2] = {p[8], p[9]};
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = j < rem ? swiglu(g[j / 4][j % 4], u[j / 4][j % 4]) : 0.0f;
}

}  // namespace moe
