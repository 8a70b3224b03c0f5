// logprobs.hip -- log probabilities of given tokens, entropy and top alternatives of
// rows of logits. With m the row's largest logit, s = sum exp(x - m) and
// e = sum (x - m) exp(x - m):  z - m = log s,  entropy = log s - e / s,  so that
// every sum is of numbers near the row's largest, whatever the logits' offset.
#include "attention_internal.h"
#include "row_device.h"

namespace moe {
namespace {

constexpr int kThreads = 1024;

__device__ __forceinline__ float logit(const float *x, int i) { return x[i]; }
__device__ __forceinline__ float logit(const uint16_t *x, int i) { return bf16_to_f32(x[i]); }

// Order of the alternatives as one number: the larger logit first (NaN above
// everything, -0 as 0), of equal ones the lower token. Never 0.
__device__ __forceinline__ uint64_t rank_of(float v, int i) {
  uint32_t u = v == v ? __float_as_uint(v + 0.0f) : 0x7fffffffu;
  u = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (uint64_t)u << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float rank_value(uint64_t r) {
  uint32_t u = (uint32_t)(r >> 32);
  u = u & 0x80000000u ? u & 0x7fffffffu : ~u;
  return __uint_as_float(u);
}

// Running largest value, and the two sums relative to it.
struct Sums {
  float m, s, e;
};
__device__ __forceinline__ void join(Sums &a, const Sums &b) {
  const float m = fmaxf(a.m, b.m);
  auto part = [&](const Sums &p, float &s, float &e) {
    if (p.m == -INFINITY) {  // nothing, or nothing but -inf (or NaN: kept in s)
      s = p.s;
      e = p.e;
      return;
    }
    const float d = p.m - m, f = expf(d);
    s = p.s * f;
    e = f > 0.0f ? (p.e + p.s * d) * f : 0.0f;  // (d may be past the fp32 range)
  };
  float s0, e0, s1, e1;
  part(a, s0, e0);
  part(b, s1, e1);
  a = Sums{m, s0 + s1, e0 + e1};
}

template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobArgs a) {
  __shared__ float red[3][kThreads / 64];
  __shared__ uint64_t best[kThreads / 64];
  const int64_t t = blockIdx.x;
  const T *x = reinterpret_cast<const T *>(a.x) + t * a.ld;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float m = -INFINITY;
  bool nan = false;
  for (int i = tid; i < a.V; i += kThreads) {
    const float v = logit(x, i);
    nan |= v != v;
    m = fmaxf(m, v);
  }
  Sums p{m, 0.0f, 0.0f};
  for (int i = tid; i < a.V; i += kThreads) {
    const float v = logit(x, i);
    if (v == -INFINITY) continue;
    const float d = v - m, f = expf(d);
    p.s += f;
    p.e += f > 0.0f ? d * f : 0.0f;
  }
  if (nan) p.s = NAN;
  for (int o = 32; o > 0; o >>= 1)
    join(p, Sums{__shfl_xor(p.m, o), __shfl_xor(p.s, o), __shfl_xor(p.e, o)});
  if (lane == 0) {
    red[0][wave] = p.m;
    red[1][wave] = p.s;
    red[2][wave] = p.e;
  }
  __syncthreads();
  p = Sums{red[0][0], red[1][0], red[2][0]};
  for (int w = 1; w < kThreads / 64; ++w) join(p, Sums{red[0][w], red[1][w], red[2][w]});
  const float z = p.m == -INFINITY ? NAN : logf(p.s);
  if (tid == 0) {
    if (a.logprobs) {
      const int64_t k = a.tokens[t];
      a.logprobs[t] = k >= 0 && k < a.V ? logit(x, (int)k) - p.m - z : NAN;
    }
    if (a.entropy) a.entropy[t] = z - p.e / p.s;
  }
  uint64_t last = ~0ull;
  for (int n = 0; n < a.top; ++n) {
    uint64_t r = 0;
    for (int i = tid; i < a.V; i += kThreads) {
      const uint64_t k = rank_of(logit(x, i), i);
      if (k < last && k > r) r = k;
    }
    r = wave_max_u64(r);
    if (lane == 0) best[wave] = r;
    __syncthreads();
    last = 0;
    for (int w = 0; w < kThreads / 64; ++w) last = best[w] > last ? best[w] : last;
    __syncthreads();
    if (tid == 0) {
      a.top_tokens[t * a.top + n] = (int)~(uint32_t)last;
      a.top_logprobs[t * a.top + n] = rank_value(last) - p.m - z;
    }
  }
}

}  // namespace

hipError_t launch_token_logprobs(const LogprobArgs &a, bool f32, int64_t T, hipStream_t st) {
  const dim3 grid((unsigned)T), block(kThreads);
  if (f32) return launch_kernel(logprobs_kernel<float>, grid, block, st, {}, a);
  return launch_kernel(logprobs_kernel<uint16_t>, grid, block, st, {}, a);
}

}  // namespace moe
