// epilogue_device.h -- what the W8A8 products of the decoder block do with a
// dequantised value: bias, gate per token, add, one rounding to the output
// type. Included by the HIP sources only.
#pragma once

#include "lds_dma.h"
#include "row_device.h"

namespace moe {

// Columns n0 .. n0+VN-1 of row t (those below ep.N exist), gated values in v:
// add, rounding, store.
template <int VN>
__device__ __forceinline__ void store_columns(const Epilogue &ep, int64_t t, int n0, float *v) {
  const int rem = ep.N - n0;
  if (rem <= 0) return;
  if (ep.add) {
    const uint16_t *row = ep.add + t * ep.ld_add;
    if constexpr (VN == 8) {
      float b[8];
      load8(row, n0, ep.N, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += b[i];
    } else {  // (one 8-byte load where all four exist: 5.4 us for a single token, 5.2 so)
#pragma unroll
      for (int i = 0; i < VN; ++i)
        if (i < rem) v[i] += bf16_to_f32(row[n0 + i]);
    }
  }
  if (ep.out_f32) {
    float *row = static_cast<float *>(ep.out) + t * ep.ld_out;
    if constexpr (VN == 8) {
      store8(row, n0, ep.N, v);
    } else if (rem >= VN) {
      *reinterpret_cast<v4f_a4 *>(row + n0) = v4f{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < VN; ++i)
        if (i < rem) row[n0 + i] = v[i];
    }
  } else {
    uint16_t *row = static_cast<uint16_t *>(ep.out) + t * ep.ld_out;
    if constexpr (VN == 8) {
      store8(row, n0, ep.N, v);
    } else if (rem >= VN) {
      *reinterpret_cast<v2i_a2 *>(row + n0) = v2i{(int)bf16x2(v[0], v[1]), (int)bf16x2(v[2], v[3])};
    } else {
#pragma unroll
      for (int i = 0; i < VN; ++i)
        if (i < rem) row[n0 + i] = f32_to_bf16(v[i]);
    }
  }
}

// The same from the dequantised sums: bias and gate first.
template <int VN>
__device__ __forceinline__ void finish_columns(const Epilogue &ep, int64_t t, int n0, float *v) {
  if (ep.bias) {
#pragma unroll
    for (int i = 0; i < VN; ++i)
      if (n0 + i < ep.N) v[i] += ep.bias[n0 + i];
  }
  if (ep.gate) {
    const float g = ep.gate[t];
#pragma unroll
    for (int i = 0; i < VN; ++i) v[i] *= g;
  }
  store_columns<VN>(ep, t, n0, v);
}

}  // namespace moe
