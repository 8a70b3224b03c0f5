// host_checks.h -- argument checks shared by the host sides of the operators:
// alignment, pitches, and whether two matrices in memory may share a byte.
#pragma once

#include "block_internal.h"

namespace moe {

constexpr int64_t kMaxRows = ((int64_t)1 << 22) - 1;  // a launch counts rows x threads in 32 bits
// Rows a distance of ld elements apart stay addressable (2^48 elements in all).
constexpr int64_t kMaxPitch = (int64_t)1 << 26;

inline bool al(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
inline bool width_ok(int64_t k) { return k >= 1 && k <= kMaxWidth; }
inline bool outputs_ok(int64_t n) { return n >= 1 && n <= kMaxOutputs; }
inline bool format_ok(int32_t f) { return f == MOE_W8A8_FORMAT_INT8 || f == MOE_W8A8_FORMAT_FP8; }
inline bool type_ok(int32_t t) { return t == MOE_W8A8_BF16 || t == MOE_W8A8_F32; }
inline bool pitch_ok(int64_t ld, int64_t width) { return ld >= width && ld <= kMaxPitch; }
// A strided matrix in memory: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Mat {
  const void *p;
  size_t rows, pitch, width;
};
inline Mat mat(const void *p, int64_t rows, int64_t ld, int64_t width, size_t size) {
  return Mat{rows > 0 ? p : nullptr, (size_t)rows, (size_t)ld * size, (size_t)width * size};
}
inline Mat flat(const void *p, size_t bytes) { return Mat{bytes ? p : nullptr, 1, bytes, bytes}; }
// Whether two matrices may share a byte. Column blocks of one buffer (the same
// pitch) are told apart by their columns; anything else by the ranges they span.
inline bool overlap(const Mat &a, const Mat &b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x >= y + (b.rows - 1) * b.pitch + b.width || y >= x + (a.rows - 1) * a.pitch + a.width)
    return false;
  if (a.pitch != b.pitch) return true;
  const size_t d = y >= x ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
  return d < a.width || d + b.width > a.pitch;
}

}  // namespace moe

#define MOE_CHECK(expr)                                \
  do {                                                 \
    if ((expr) != hipSuccess) return MOE_W8A8_ERR_HIP; \
  } while (0)
#define MOE_TRY(expr)              \
  do {                             \
    const int rc_ = (expr);        \
    if (rc_ != MOE_W8A8_OK) return rc_; \
  } while (0)
