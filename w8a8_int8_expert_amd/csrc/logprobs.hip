// logprobs.hip -- log probabilities of given tokens, entropy and top alternatives of
// rows of logits, in one pass over them. With m the row's largest logit,
// s = sum exp(x - m) and e = sum (x - m) exp(x - m):  z - m = log s and
// entropy = log s - e / s, so that every sum is of numbers near the row's largest,
// whatever the logits' offset. Each thread keeps its own (m, s, e) and takes the sums
// along when its m grows.
//
// The alternatives are found in the same pass. The n-th largest of the first chunk's
// thread maxima is a bound that at least n elements reach; only elements past it go
// into a list in LDS (about n V / 2048 of a row in random order), which is cut back to
// its n best, and the bound raised, when it fills up: an order in which every element is
// a candidate costs time, not room. The bound is found by halving over wavefront ballots, and
// a wavefront's candidates take one atomic: 32 rows of 32003 in 9 us (12 when each maximum
// counted those above it and each candidate took its own atomic).
//
// Bound by memory for many rows and few alternatives: 4096 rows of 32003 fp32 logits, top 1, in
// 107 us, 4.9 TB/s; 1024 of 128256 bf16, 263 MB, top 1, in 126, 2.1 TB/s. The lists cost two
// barriers for each place whenever they fill up: 4096 rows of 32003 fp32 with 0, 5, 20, 64
// alternatives 94, 125, 174, 405 us, in bf16 44, 116, 172, 396 (top 1: 94); in rising order, where
// every chunk fills them, top 20 958, top 64 2970. A row with a NaN takes a pass over itself for
// each place: one among 4096 rows, top 20, 459 us. Few rows are cut into parts of at least 4096
// elements, one to a block, and joined by a second launch.
#include "attention_internal.h"
#include "row_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kChunk = 8 * kThreads;
constexpr int kKeep = 256;              // candidates that may wait between two chunks
constexpr int kRoom = kKeep + kChunk;   // and what one chunk may add
constexpr int kMostParts = 64;          // one lane each where they are joined
constexpr float kFar = -200.0f;         // exp of it is 0 in fp32

__device__ __forceinline__ float logit(const float *x, int i) { return x[i]; }
__device__ __forceinline__ float logit(const uint16_t *x, int i) { return bf16_to_f32(x[i]); }

// Order of the alternatives as one number: the larger logit first (NaN above
// everything, -0 as 0), of equal ones the lower token. Never 0.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = v == v ? __float_as_uint(v + 0.0f) : 0x7fffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint64_t rank_of(float v, int i) {
  return (uint64_t)order_of(v) << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float rank_value(uint64_t r) { return order_value((uint32_t)(r >> 32)); }
__device__ __forceinline__ int rank_token(uint64_t r) { return (int)~(uint32_t)r; }

// Largest value so far and the two sums relative to it. A row with a NaN has s = NaN
// in the end; +inf is seen in m, nothing but -inf in s = 0.
struct Sums {
  float m, s, e;
};
constexpr float kLowest = -3.402823466e38f;
__device__ __forceinline__ void rescale(Sums &a, float m) {
  const float d = fmaxf(a.m - m, kFar), f = expf(d);
  a.e = (a.e + a.s * d) * f;
  a.s *= f;
  a.m = m;
}
__device__ __forceinline__ void join(Sums &a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  rescale(a, m);
  rescale(b, m);
  a.s += b.s;
  a.e += b.e;
}

// What a part hands to the join: its sums, and its best candidates in order.
struct Parts {
  Sums *sums;      // [T][parts]
  uint64_t *best;  // [T][parts][top], 0 past the part's end
  int parts;
};
struct Result {
  float z, h;  // z - m and the entropy, NaN where the row has none
};
__device__ __forceinline__ Result result_of(const Sums &a) {
  const bool none = a.s == 0.0f || a.m == INFINITY;
  const float z = none ? NAN : logf(a.s);
  return Result{z, z - a.e / a.s};
}
template <typename T>
__device__ __forceinline__ void write_sums(const LogprobArgs &a, int64_t t, const T *x,
                                           const Sums &s, const Result &r) {
  if (a.logprobs) {
    const int64_t k = a.tokens[t];
    a.logprobs[t] = k >= 0 && k < a.V ? logit(x, (int)k) - s.m - r.z : NAN;
  }
  if (a.entropy) a.entropy[t] = r.h;
}
__device__ __forceinline__ void write_top(const LogprobArgs &a, int64_t t, int n, uint64_t k,
                                          const Sums &s, const Result &r) {
  a.top_tokens[t * a.top + n] = rank_token(k);
  a.top_logprobs[t * a.top + n] = rank_value(k) - s.m - r.z;
}

template <typename T, bool kTop>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobArgs a, Parts parts, int per) {
  __shared__ uint64_t list[kTop ? kRoom : 1], best[64];
  __shared__ uint64_t wave_best[kWaves];
  __shared__ Sums red[kWaves];
  __shared__ int count;
  __shared__ uint32_t maxima[kTop ? kThreads : 1];
  const int64_t t = blockIdx.x / parts.parts;
  const int part = blockIdx.x % parts.parts;
  const T *x = reinterpret_cast<const T *>(a.x) + t * a.ld;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c0 = part * per, c1 = c0 + per < a.V ? c0 + per : a.V;
  const int top = a.top;
  Sums p{kLowest, 0.0f, 0.0f};
  bool nan = false;
  uint32_t bar = 0;  // order of the bound that candidates reach
  if (kTop && tid == 0) count = 0;

  // The `n` best of the list, in order, in `best`; the list is spent (every thread).
  auto take_best = [&](int n, int have) {
    uint64_t mine[(kRoom + kThreads - 1) / kThreads];
#pragma unroll
    for (int i = 0; i < (kRoom + kThreads - 1) / kThreads; ++i)
      mine[i] = i * kThreads + tid < have ? list[i * kThreads + tid] : 0;
    for (int k = 0; k < n; ++k) {
      uint64_t r = 0;
#pragma unroll
      for (int i = 0; i < (kRoom + kThreads - 1) / kThreads; ++i) r = mine[i] > r ? mine[i] : r;
      r = wave_max_u64(r);
      if (lane == 0) wave_best[wave] = r;
      __syncthreads();
      r = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) r = wave_best[w] > r ? wave_best[w] : r;
      __syncthreads();
      if (tid == 0) best[k] = r;
#pragma unroll
      for (int i = 0; i < (kRoom + kThreads - 1) / kThreads; ++i) mine[i] = mine[i] == r ? 0 : mine[i];
    }
    __syncthreads();
  };

  auto raw = fetch8(x, c0 + 8 * tid, a.V);
  for (int c = c0; c < c1; c += kChunk) {
    float v[8];
    const int at = c + 8 * tid;
    unpack8(raw, at, a.V, v);
    if (c + kChunk < c1) raw = fetch8(x, at + kChunk, a.V);
    if (at + 8 > c1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = at + j < c1 ? v[j] : -INFINITY;
    }
    float big = v[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) big = fmaxf(big, v[j]);
#pragma unroll
    for (int j = 0; j < 8; j += 2) nan |= __builtin_isunordered(v[j], v[j + 1]);
    if (big > p.m) rescale(p, big);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = fmaxf(v[j] - p.m, kFar), f = __expf(d);
      p.s += f;
      p.e = __builtin_fmaf(d, f, p.e);
    }
    if constexpr (kTop) {
      if (c == c0) {
        // the bound, bit by bit: the largest number that `top` of the threads' maxima
        // reach (0 if fewer have any), or the first one met that just so many do
        maxima[tid] = at < c1 ? order_of(big) : 0;
        __syncthreads();
        uint32_t o[kWaves], bound = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) o[w] = maxima[w * 64 + lane];
        for (int bit = 31; bit >= 0; --bit) {
          const uint32_t next = bound | 1u << bit;
          int n = 0;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) n += __popcll(__ballot(o[w] >= next));
          if (n >= top) bound = next;
          if (n == top) break;
        }
        bar = bound;
      }
      // candidates reach the bound; each takes its place behind those of lower lanes
      const bool added = __any(at < c1 && order_of(big) >= bar);
      if (added) {
        uint64_t past[8];
        int n = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          past[j] = __ballot(at + j < c1 && order_of(v[j]) >= bar);
          n += __popcll(past[j]);
        }
        int to = 0;
        if (lane == 0) to = atomicAdd(&count, n);
        to = __builtin_amdgcn_readfirstlane(to);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (past[j] >> lane & 1)
            list[to + __builtin_amdgcn_mbcnt_hi((uint32_t)(past[j] >> 32),
                                                __builtin_amdgcn_mbcnt_lo((uint32_t)past[j], 0))] =
                rank_of(v[j], at + j);
          to += __popcll(past[j]);
        }
      }
      if (c == c0 && bar != 0) ++bar;  // of equal ones those of lower tokens come first
      if (__syncthreads_or(added)) {
        const int have = count;
        __syncthreads();
        if (have > kKeep) {
          take_best(top, have);
          if (tid < top) list[tid] = best[tid];
          if (tid == 0) count = top;
          bar = (uint32_t)(best[top - 1] >> 32) + 1;
          __syncthreads();
        }
      }
    }
  }

  // to the block's largest first, then the sums
  float m = order_value(wave_max_bits(order_of(p.m)));
  if (lane == 0) red[wave].m = m;
  nan = __syncthreads_or(nan);
  m = red[0].m;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) m = fmaxf(m, red[w].m);
  rescale(p, m);
  p.s = wave_sum_f32(p.s);
  p.e = wave_sum_f32(p.e);
  if (lane == 0) red[wave].s = p.s, red[wave].e = p.e;
  __syncthreads();
  p = Sums{m, nan ? NAN : 0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) p.s += red[w].s, p.e += red[w].e;
  const bool whole = parts.parts == 1;
  const Result r = result_of(p);
  if (tid == 0) {
    if (whole) write_sums(a, t, x, p, r);
    else parts.sums[blockIdx.x] = p;
  }
  if constexpr (kTop) {
    auto put = [&](int n, uint64_t k) {
      if (whole) write_top(a, t, n, k, p, r);
      else parts.best[(int64_t)blockIdx.x * top + n] = k;
    };
    if (p.s != p.s) {
      // a NaN compares with nothing: such a row takes one round over it for each place
      uint64_t last = ~0ull;
      for (int n = 0; n < top; ++n) {
        uint64_t k = 0;
        for (int i = c0 + tid; i < c1; i += kThreads) {
          const uint64_t o = rank_of(logit(x, i), i);
          if (o < last && o > k) k = o;
        }
        k = wave_max_u64(k);
        if (lane == 0) wave_best[wave] = k;
        __syncthreads();
        k = 0;
        for (int w = 0; w < kWaves; ++w) k = wave_best[w] > k ? wave_best[w] : k;
        __syncthreads();
        if (tid == 0) put(n, k);
        last = k;
      }
      return;
    }
    // every candidate counts those above it: its place
    const int have = count;
    for (int i = tid; i < have; i += kThreads) {
      const uint64_t mine = list[i];
      int above = 0;
#pragma unroll 8
      for (int j = 0; j < have; ++j) above += list[j] > mine;
      if (above < top) put(above, mine);
    }
    for (int n = have + tid; n < top; n += kThreads) put(n, 0);  // (a short last part)
  }
}

// Joins a row's parts, whose lists are in order. The candidates of few parts each count
// those above them; of more parts, a wavefront with a list to a lane gives each place to the
// largest of the heads. That takes 3 + 0.2 top us, counting 1 + 0.03 parts top us: 20 places
// of 8 parts 5.2 us counted, 7.6 us from the heads; 16 of 32 parts 16 us counted, 6 from
// the heads.
constexpr int kJoinThreads = 256;
constexpr int kCountedParts = 8;
template <typename T>
__global__ __launch_bounds__(kJoinThreads) void logprobs_join_kernel(LogprobArgs a, Parts parts) {
  __shared__ uint64_t lists[kMostParts * 64];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, n = parts.parts, top = a.top;
  Sums p{kLowest, 0.0f, 0.0f};
  if (lane < n) p = parts.sums[t * n + lane];
  for (int i = tid; i < n * top; i += kJoinThreads) lists[i] = parts.best[t * n * top + i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
    join(p, Sums{__shfl_xor(p.m, o), __shfl_xor(p.s, o), __shfl_xor(p.e, o)});
  const Result r = result_of(p);
  if (tid == 0) write_sums(a, t, reinterpret_cast<const T *>(a.x) + t * a.ld, p, r);
  __syncthreads();
  if (n <= kCountedParts) {
    for (int i = tid; i < n * top; i += kJoinThreads) {
      const uint64_t mine = lists[i];
      int above = 0;
#pragma unroll 8
      for (int j = 0; j < n * top; ++j) above += lists[j] > mine;
      if (mine != 0 && above < top) write_top(a, t, above, mine, p, r);
    }
    return;
  }
  if (tid >= 64) return;
  int head = 0;
  uint64_t mine = lane < n ? lists[lane * top] : 0, got = 0;
  for (int k = 0; k < top; ++k) {
    const uint64_t big = wave_max_u64(mine);
    if (lane == k) got = big;
    if (mine == big && lane < n) mine = ++head < top ? lists[lane * top + head] : 0;
  }
  if (lane < top) write_top(a, t, lane, got, p, r);
}

// Parts of a row: about 1024 blocks in all.
int parts_of(int V, int64_t T) {
  const int64_t want = (1024 + T - 1) / T;
  const int most = (V + 2 * kChunk - 1) / (2 * kChunk);
  const int n = (int)(want < most ? want : most);
  return n < kMostParts ? n : kMostParts;
}
size_t sums_bytes(int parts, int64_t T) { return ((size_t)T * parts * sizeof(Sums) + 255) / 256 * 256; }

template <typename T>
hipError_t launch(const LogprobArgs &a, int64_t T_, void *ws, hipStream_t st) {
  const int want = parts_of(a.V, T_);
  const int per = ((a.V + want - 1) / want + kChunk - 1) / kChunk * kChunk;
  const int n = (a.V + per - 1) / per;
  Parts p{(Sums *)ws, nullptr, n};
  p.best = reinterpret_cast<uint64_t *>((char *)ws + sums_bytes(n, T_));
  const dim3 grid((unsigned)(T_ * n)), block(kThreads);
  const hipError_t e = a.top ? launch_kernel(logprobs_kernel<T, true>, grid, block, st, {}, a, p, per)
                             : launch_kernel(logprobs_kernel<T, false>, grid, block, st, {}, a, p, per);
  if (e != hipSuccess || n == 1) return e;
  return launch_kernel(logprobs_join_kernel<T>, dim3((unsigned)T_), dim3(kJoinThreads), st, {}, a, p);
}

}  // namespace

size_t token_logprobs_workspace(int V, int top, int64_t T) {
  const int n = parts_of(V, T);
  return n > 1 ? sums_bytes(n, T) + (size_t)T * n * top * sizeof(uint64_t) : 0;
}
hipError_t launch_token_logprobs(const LogprobArgs &a, bool f32, int64_t T, void *ws,
                                 hipStream_t st) {
  return f32 ? launch<float>(a, T, ws, st) : launch<uint16_t>(a, T, ws, st);
}

}  // namespace moe
