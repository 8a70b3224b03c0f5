// lds_dma.h -- device building blocks shared by the tiled matrix products: direct
// global -> LDS loads, the wait that goes with them, the epilogue's SwiGLU and
// row maximum, and the conversion of e4m3 codes. Included by the HIP sources only.
#pragma once

#include "moe_internal.h"

// The direct-to-LDS loads are issued from inline assembly: the compiler's own
// intrinsic makes every later LDS read wait for all outstanding loads, which
// would drain the stage ring on each step. The assembly sets M0 (the LDS base
// of the wavefront's 1 KB) itself, and the waits are explicit.
#pragma clang diagnostic ignored "-Winline-asm"

namespace moe {

__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return (uint32_t)(uintptr_t)((__attribute__((address_space(3))) const void *)p);
}
// 16 bytes per lane from global memory into LDS at lds_base + 16*lane. An
// LDS-DMA load needs one wait state after M0 is written.
__device__ __forceinline__ void dma16(const void *g, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(g), "s"(lds_base)
               : "memory", "m0");
}
// 4 bytes per lane into LDS at lds_base + 4*lane.
__device__ __forceinline__ void dma4(const void *g, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(g), "s"(lds_base)
               : "memory", "m0");
}
// Wait until at most N of this wavefront's loads are in flight and its LDS
// accesses are done, then meet the other wavefronts of the block.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// Maximum of a non-negative value over each 32-lane half of the wavefront,
// by DPP moves (no LDS round trip): row_shr 1, 2, 4, 8 leave each 16-lane
// row's maximum in its lane 15, and row_bcast15 into rows 1 and 3 adds the
// row below. The results land in lanes 31 and 63. Non-negative floats order
// as their bit patterns, so the maximum is taken on those.
__device__ __forceinline__ uint32_t half_wave_max(uint32_t m) {
  auto step = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
  m = step(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x111, 0xF, 0xF, false));
  m = step(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x112, 0xF, 0xF, false));
  m = step(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x114, 0xF, 0xF, false));
  m = step(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x118, 0xF, 0xF, false));
  m = step(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x142, 0xA, 0xF, false));
  return m;
}

// silu(g) * u with the hardware exponential and reciprocal.
__device__ __forceinline__ float swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
// Eight e4m3 codes as bf16 (exact: three mantissa bits, exponents of -9 to 8).
__device__ __forceinline__ v8bf codes_bf16(int lo, int hi) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Accumulators: INT32 for INT8 codes, fp32 for FP8 codes.
template <bool kF8> struct Acc32 { typedef v16i T; };
template <> struct Acc32<true> { typedef v16f T; };

}  // namespace moe
