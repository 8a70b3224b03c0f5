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

// Eight elements from p, the first `rem` of which exist (the rest read as 0).
__device__ __forceinline__ void load8(const uint16_t *p, int rem, float *o) {
  if (rem >= 8) {
    const v4i r = *reinterpret_cast<const v4i_a2 *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float((uint32_t)r[i] << 16);
      o[2 * i + 1] = __uint_as_float((uint32_t)r[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = i < rem ? bf16_to_f32(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float *p, int rem, float *o) {
  if (rem >= 8) {
    const v4f a = *reinterpret_cast<const v4f_a4 *>(p);
    const v4f b = *reinterpret_cast<const v4f_a4 *>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = a[i];
      o[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = i < rem ? p[i] : 0.0f;
  }
}
// Two values rounded to bf16 (nearest, ties to even; NaN stays NaN) by the one
// hardware instruction.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2bf));
}
__device__ __forceinline__ void store8(uint16_t *p, int rem, const float *v) {
  if (rem >= 8) {
    v4i r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (int)bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<v4i_a2 *>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < rem) p[i] = f32_to_bf16(v[i]);
  }
}
__device__ __forceinline__ void store8(float *p, int rem, const float *v) {
  if (rem >= 8) {
    *reinterpret_cast<v4f_a4 *>(p) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f_a4 *>(p + 4) = v4f{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < rem) p[i] = v[i];
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
// them exist) from a row of gate and up values in packed order: alternating
// runs of 32.
__device__ __forceinline__ void hidden8(const float *gu, int c, int rem, float *o) {
  if (rem <= 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = 0.0f;
    return;
  }
  float u[8];
  const float *p = gu + c / 32 * 64 + c % 32;
  load8(p, rem, o);
  load8(p + 32, rem, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = swiglu(o[j], u[j]);
}

}  // namespace moe
