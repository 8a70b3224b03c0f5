// attention_tiles.hip -- attention of many query rows of each kv head over the paged
// cache (chunks of a prefill). A row is one query head of one token; the rows of the
// heads that share a kv head follow each other token by token, 128 to a block.
//
// Each wavefront has 32 rows, the block's four share tiles of keys and values in LDS.
// Scores are taken with keys as the matrix instruction's rows and queries as its
// columns: lane l holds query l % 32 and half of the keys, so that a row's maximum and
// sum stay in the lane but for one exchange with lane l ^ 32, and the probabilities
// are where the second product takes them from, with the values transposed by the LDS
// reads. The running maximum is raised only when a row's grows by more than 2^8, so
// that most tiles leave the results alone: a probability may be as large as that, which
// neither its bf16 rounding nor the fp32 sums mind.
//
// Bound by the matrix instructions together with the exponentials: of 64 keys, 32
// matrix instructions of 32 cycles against about 1000 cycles of vector instructions.
// Two blocks share a compute unit, one's softmax under the other's products. 8192 tokens of 32
// heads over 8 of 128, causal: 532 to 565 us with the card's clocks, 1.0 PFLOP/s.
//
// Nothing between a tile's barriers diverges (loops run by shared counts, conditions of
// single lanes select): the compiler has been seen to put a copy of a live register,
// where registers are short, before the restore of the lanes that such a branch left.
#include <type_traits>

#include "attention_device.h"
#include "attention_work.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr float kGrow = 8.0f;  // log2 of what a row's maximum may grow unseen

template <int D, int kFormat>
struct Cfg {
  static constexpr bool k8 = kFormat != kBf16Cache;
  static constexpr int kKeys = kManyKeys<D>;  // of a tile
  static constexpr int kSub = kKeys / 16;           // runs of 16 keys: each in one page
  static constexpr int kRow = 2 * D;                // bytes of a row in LDS (bf16)
  static constexpr int kTile = kKeys * kRow;
  static constexpr int kScales = k8 ? 2 * kKeys * 4 : 0;
  static constexpr int kStage = 2 * kTile + kScales;
  static constexpr int kLds = 2 * kStage;
  static constexpr int kBlocks = kKeys / 32;  // of 32 keys
  static constexpr int kSteps = D / 16;       // matrix instructions of a score block
  static constexpr int kOut = D / 32;
  // Blocks on a compute unit, which share its registers. 8-bit heads of 128 keep some of their
  // state in memory for two (32 registers), and win: 4 sequences of 2048 tokens, INT8, 230 us,
  // one block 322. 256-wide heads have room for one: no other products run under its softmax.
  // A third block of 64-wide heads: 8192 tokens, bf16, 321 us, two 346; INT8 ones lose as much
  // in short chunks (47 us for 42) as they win in long ones (405 for 435).
  static constexpr int kPerUnit = D == 256 ? 1 : D == 64 && !k8 ? 3 : 2;
};

// Order for the scheduler: the next N instructions of a kind.
enum { kVector = 2, kMatrix = 8 };
template <int kKind, int N>
__device__ __forceinline__ void sched() {
  __builtin_amdgcn_sched_group_barrier(kKind, N, 0);
}

__device__ __forceinline__ v16f mfma32bf(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// Rows of a tile of bf16 elements in LDS, chunks of 16 bytes exchanged as Tile has them.
template <int D>
__device__ __forceinline__ int key_at(int r, int c) {
  return r * 2 * D + Tile<D, kBf16Cache>::key_chunk(r, c) * 16;
}
template <int D>
__device__ __forceinline__ int value_at(int r, int c) {
  return r * 2 * D + Tile<D, kBf16Cache>::template value_chunk<true>(r, c) * 16;
}
// A operand of 32 elements x 16 keys (keys r0 + 8 e + 4 (l / 32) + 0..3, e = 0, 1):
// lane l has element 32 dt + l % 32.
template <int D>
__device__ __forceinline__ v8bf value_frag(const char *tile, int r0, int dt, int lane) {
  typedef __attribute__((address_space(3))) v4s L;
  const int i = lane & 15, r = r0 + 4 * (lane >> 5) + (i >> 2);
  const int c = 4 * dt + 2 * ((lane >> 4) & 1) + ((i >> 1) & 1), o = (i & 1) * 8;
  const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)(tile + value_at<D>(r, c) + o));
  const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L *)(tile + value_at<D>(r + 8, c) + o));
  return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int D, int kFormat>
__global__ __launch_bounds__(kThreads, (Cfg<D, kFormat>::kPerUnit)) void tiles_kernel(
    AttnArgs a, CacheView c, BatchView bt, int target, Partial part) {
  typedef Cfg<D, kFormat> C;
  constexpr int K = C::kKeys, NB = C::kBlocks;
  __shared__ __attribute__((aligned(1024))) char lds[C::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  const int h = blockIdx.x % c.kv_heads;
  const Schedule<false, K> work(a, bt, target, kLeastMany<D>, 1);
  const int chunk = work.chunk;
  const int page_size = 1 << c.log2_page;
  const uint32_t page16 = (uint32_t)(c.page_bytes >> 4);
  const uint32_t lds_at = __builtin_amdgcn_readfirstlane(lds_addr(lds));
  const float scale2 = fabsf(a.scale2);
  const uint32_t flip = a.scale2 < 0.0f ? 0x80008000u : 0u;  // (queries take the sign)

  // Direct loads: a wavefront's kEach loads of 1 KB take consecutive rows; which chunk
  // a lane reads depends on its row and the exchange, the same for loads 16 rows apart.
  constexpr int kEach = C::kTile / 1024 / kWaves, kLoadRows = 1024 / C::kRow;
  constexpr int kKinds = kLoadRows >= 16 ? 1 : 16 / kLoadRows < kEach ? 16 / kLoadRows : kEach;
  uint32_t lane_at[2][kKinds];
#pragma unroll
  for (int i = 0; i < kKinds; ++i) {
    const int r = wave * kEach * kLoadRows + i * kLoadRows + lane * 16 / C::kRow;
    const int ch = lane * 16 % C::kRow / 16, in = lane * 16 / C::kRow * C::kRow;
    lane_at[0][i] = in + Tile<D, kBf16Cache>::key_chunk(r, ch) * 16;
    lane_at[1][i] = in + Tile<D, kBf16Cache>::template value_chunk<true>(r, ch) * 16;
  }

  for (int64_t u = blockIdx.x / c.kv_heads;; u += gridDim.x / c.kv_heads) {
    const Unit un = work.find(a, bt, u);
    if (un.b < 0) break;
    const int r0 = un.block * kTileRows;
    const int r1 = un.w.rows < r0 + kTileRows ? un.w.rows : r0 + kTileRows;
    const int len = un.w.s.len, first = len - un.w.s.n;
    const int p0 = first + r0 / a.group, p1 = first + (r1 - 1) / a.group;
    const int any_lo = seen_lo(p0, a.window), any_hi = seen_hi(p1, len, a.causal);
    const int all_lo = seen_lo(p1, a.window), all_hi = seen_hi(p0, len, a.causal);
    const int end = any_hi > any_lo ? (any_hi + K - 1) / K : any_lo / K;
    const int t0 = any_lo / K + un.piece * chunk;
    const int t1 = un.piece + 1 < un.pieces && t0 + chunk < end ? t0 + chunk : end;

    // (a lane past the last row computes that one again and sees nothing)
    const int row_ = r0 + 32 * wave + col;
    const bool there = row_ < r1;
    const int row = there ? row_ : r1 - 1, tok = row / a.group;
    const int lo = seen_lo(first + tok, a.window);
    const int hi = there ? seen_hi(first + tok, len, a.causal) : 0;
    v8bf q[C::kSteps];
    {
      const uint16_t *src = a.q + (int64_t)(un.w.s.start + tok) * a.ld_q +
                            (h * a.group + row % a.group) * D + 8 * half;
#pragma unroll
      for (int s = 0; s < C::kSteps; ++s) {
        v4i w = *reinterpret_cast<const v4i_a2 *>(src + 16 * s);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] ^= (int)flip;
        q[s] = __builtin_bit_cast(v8bf, w);
      }
    }

    // Pages. A wavefront brings kMine consecutive rows of each tile, which lie in one page.
    // Whether pages are missing at all is found out once, lanes reading 64 at a time.
    constexpr int kMine = K / kWaves;
    const int32_t *const table = bt.table + (int64_t)un.b * bt.ld_table;
    auto exists = [&](int p) { return (uint32_t)p < (uint32_t)c.num_pages; };
    bool holes = false;
    if (t0 < t1) {
      const int last = ((t1 * K < any_hi ? t1 * K : any_hi) - 1) >> c.log2_page;
      for (int i = t0 * K >> c.log2_page; i <= last; i += 64)
        holes = holes || __any(!exists(table[i + lane < last ? i + lane : last]));
    }
    // of run x of 16 keys of tile t (where there are holes)
    auto run_exists = [&](int t, int x) {
      const int key = t * K + 16 * x;
      return key < any_hi && exists(scalar_word(table, key >> c.log2_page));
    };
    // this wavefront's page of tile t (past the last key: of that)
    auto my_page = [&](int t) {
      const int key = t * K + wave * kMine;
      return scalar_word(table, (key < any_hi ? key : any_hi - 1) >> c.log2_page);
    };
    // a tile on its way: direct loads (bf16), or codes in registers, converted when they are
    // put into LDS. A page that does not exist is read as page 0, and masked.
    constexpr int kPer = C::k8 ? kMine * D / 16 / 64 : 1;
    v4i codes[2][kPer];
    float scl = 0.0f;
    int page = t0 < t1 ? my_page(t0) : 0;  // of the next tile to be fetched
    auto fetch = [&](int buf, int t) __attribute__((always_inline)) {
      const uint32_t p = exists(page) ? page : 0;
      page = my_page(t + 1);
      const uint32_t row = ((uint32_t)h << c.log2_page) + ((t * K + wave * kMine) & (page_size - 1));
      if constexpr (!C::k8) {
        const uint64_t from = ((uint64_t)p * page16 << 4) + (uint64_t)row * C::kRow;
        const uint32_t to = lds_at + buf * C::kStage + wave * kEach * 1024;
        dma16_run<kEach, kKinds>(c.k + from, lane_at[0], to);
        dma16_run<kEach, kKinds>(c.v + from, lane_at[1], to + C::kTile);
      } else {
        const uint64_t from = ((uint64_t)p * page16 << 4) + (uint64_t)row * D;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          codes[0][i] = *reinterpret_cast<const v4i *>(c.k + from + (i * 64 + lane) * 16);
          codes[1][i] = *reinterpret_cast<const v4i *>(c.v + from + (i * 64 + lane) * 16);
        }
        // (the scales of kMine keys, then values, by all lanes: the same one more than once)
        const float *const sc = lane & kMine ? c.v_scale : c.k_scale;
        scl = sc[(int64_t)p * c.scale_stride + row + lane % kMine];
      }
    };
    auto put = [&](int buf) {
      if constexpr (C::k8) {
        char *const st = lds + buf * C::kStage;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int piece = wave * kPer * 64 + i * 64 + lane;
          const int r = piece / (D / 16), ch = piece % (D / 16) * 2;
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const v8bf x = code8_bf16<kFormat>(codes[v][i][2 * e], codes[v][i][2 * e + 1]);
              *reinterpret_cast<v8bf *>(st + v * C::kTile + (v ? value_at<D>(r, ch + e)
                                                               : key_at<D>(r, ch + e))) = x;
            }
        }
        reinterpret_cast<float *>(st + 2 * C::kTile)[(lane & kMine ? K : 0) + wave * kMine +
                                                      lane % kMine] =
            lane & kMine ? scl : scl * scale2;  // (scores come out scaled)
      }
    };

    v16f o[C::kOut];
#pragma unroll
    for (int d = 0; d < C::kOut; ++d) o[d] = v16f{};
    float m = kNoMax, l = 0.0f;
    bool some_odd = false;

    // values of a tile in LDS that no row of the block sees count as zeros, whatever lies
    // there
    auto clear_unseen = [&](char *vt, int key0, const bool *ok) {
      for (int y = 0; y < C::kTile / 16 / kThreads; ++y) {
        const int i = y * kThreads + tid, r = i / (C::kRow / 16), key = key0 + r;
        int gone = (key < any_lo) | (key >= any_hi);
#pragma unroll
        for (int x = 0; x < C::kSub; ++x) gone |= (r >> 4 == x) & !ok[x];
        v4i v = reinterpret_cast<const v4i *>(vt)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = gone ? 0 : v[j];
        reinterpret_cast<v4i *>(vt)[i] = v;
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
    // scores, softmax and product of the tile in stage buf
    auto step = [&](auto kind, int buf, int key0, const bool *ok) __attribute__((always_inline)) {
      constexpr bool kMasked = decltype(kind)::value;
      char *const kt = lds + buf * C::kStage, *const vt = kt + C::kTile;
      const float *const sc = reinterpret_cast<const float *>(vt + C::kTile);
      if constexpr (kMasked) clear_unseen(vt, key0, ok);

      // scores: block n, register i: key 32 n + 8 (i / 4) + 4 half + i % 4. The fragments of
      // four instructions are on their way while the four before are at work: an LDS read
      // takes as long as three (left to the compiler, which reads each where it is needed,
      // 8192 tokens of 32 heads of 128 take 549 us instead of 538).
      v16f s[NB];
      v8bf f[2][4];
      // (of wide bf16 heads, places in LDS are worked out again for each tile: there are no
      // registers to keep them in, and one read back from memory waits for the loads in
      // flight. 8192 tokens, 16 heads of 256, bf16: 910 us, 1147 with what the compiler kept)
      int at_ = lane;
      if constexpr (D == 256 && !C::k8) asm volatile("" : "+v"(at_));
      auto keys = [&](int i, v8bf *to) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          to[j] = *reinterpret_cast<const v8bf *>(
              kt + key_at<D>(32 * ((i + j) % NB) + (at_ & 31), 2 * ((i + j) / NB) + (at_ >> 5)));
      };
      keys(0, f[0]);
#pragma unroll
      for (int n = 0; n < NB; ++n) s[n] = v16f{};
#pragma unroll
      for (int i = 0; i < NB * C::kSteps; i += 4) {
        if (i + 4 < NB * C::kSteps) keys(i + 4, f[(i / 4 + 1) % 2]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[(i + j) % NB] = mfma32bf(f[i / 4 % 2][j], q[(i + j) / NB], s[(i + j) % NB]);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (C::k8) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const v4f ks = *reinterpret_cast<const v4f *>(sc + 32 * n + 8 * i + 4 * half);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[n][4 * i + j] *= ks[j];
          }
      }
      uint32_t seen = 0xffffffffu;
      if constexpr (kMasked) {
        seen = 0;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = 32 * n + 8 * (i / 4) + 4 * half + i % 4, key = key0 + at;
            const bool see = key >= lo && key < hi && ok[2 * n + i / 8];
            s[n][i] = see ? s[n][i] : -INFINITY;
            if (see) seen |= 1u << (16 * n + i);
          }
      }
      float big = s[0][0];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) big = fmaxf(big, s[n][i]);
      big = C::k8 ? halves_max(big) : halves_max(big) * scale2;
      // Of scores past 2^24 the largest one's rounding is no small part of an exponent any more:
      // all are rounded as it is.
      float times = C::k8 ? 1.0f : scale2;
      if (!C::k8 && __any(fabsf(big) > 0x1p24f)) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[n][i] *= scale2;
        times = 1.0f;
      }
      if (__any(big > m + kGrow)) {
        const float mm = fmaxf(m, big), f = __builtin_amdgcn_exp2f(m - mm);
        m = mm;
        l *= f;
#pragma unroll
        for (int d = 0; d < C::kOut; ++d) o[d] *= f;
      }
      // Values that are not finite, in a tile of which some rows do not see all: an unseen
      // one must not reach a row through 0 times infinity. They are taken out here, and
      // put back behind the loop. (Every wavefront looks at the whole tile, so that all
      // come to the same.)
      if constexpr (kMasked) {
        bool odd = false;
        for (int y = 0; y < C::kTile / 16 / 64; ++y)
          odd |= any_odd(reinterpret_cast<const v8bf *>(vt)[y * 64 + lane]);
        if (__any(odd)) {
          some_odd = true;
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          for (int y = 0; y < C::kTile / 16 / kThreads; ++y) {
            v8bf *const v = reinterpret_cast<v8bf *>(vt) + y * kThreads + tid;
            *v = odd_part<false>(*v);
          }
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
      }
      // The probabilities of 16 keys after the other: those of the next 16 are taken, and
      // their values read, while the matrix instructions of the last are at work.
      auto probabilities = [&](int x) __attribute__((always_inline)) {
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x / 2][8 * (x % 2) + j], times, -m));
          if constexpr (kMasked) e[j] = seen >> (8 * x + j) & 1 ? e[j] : 0.0f;  // (-inf times 0)
          l += e[j];
        }
        if constexpr (C::k8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const v4f vs = *reinterpret_cast<const v4f *>(sc + K + 16 * x + 8 * i + 4 * half);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool see = !kMasked || (seen >> (8 * x + 4 * i + j) & 1);
              e[4 * i + j] = see ? e[4 * i + j] * vs[j] : 0.0f;
            }
          }
        }
        // rounded to bf16 for the second product: half a step of 2^-8 each, which the result,
        // itself rounded so, averages over its keys; the row's sum is of the unrounded ones. The
        // result is off by 0.0021 to 0.0023 of its size (root mean square), by its own rounding
        // alone 0.0016 to 0.0017. A second term, which the few rows of a decode step have, brings
        // it there for half again the matrix instructions: 8192 tokens, 32 heads of 128, 705 us
        // instead of 541, 16 heads of 256 1058 instead of 919, the mixed batch of 12 sequences
        // 482 instead of 384, 9 windowed chunks of 64-wide INT8 heads 45 instead of 42.
        return __builtin_bit_cast(
            v8bf, v4i{(int)bf16x2(e[0], e[1]), (int)bf16x2(e[2], e[3]), (int)bf16x2(e[4], e[5]),
                      (int)bf16x2(e[6], e[7])});
      };
      v8bf p[2], v[2][C::kOut];
      auto values = [&](int x) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < C::kOut; ++d) v[x % 2][d] = value_frag<D>(vt, 16 * x, d, at_);
      };
      values(0);
      p[0] = probabilities(0);
#pragma unroll
      for (int x = 0; x < 2 * NB; ++x) {
        if (x + 1 < 2 * NB) values(x + 1);
        __builtin_amdgcn_sched_barrier(0);
        if (x + 1 < 2 * NB) p[(x + 1) % 2] = probabilities(x + 1);
#pragma unroll
        for (int d = 0; d < C::kOut; ++d) o[d] = mfma32bf(v[x % 2][d], p[x % 2], o[d]);
        if (x + 1 < 2 * NB)
#pragma unroll
          for (int d = 0; d < C::kOut; ++d) {
            sched<kMatrix, 1>();
            sched<kVector, 28 / C::kOut>();
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    if (t0 < t1) {
      fetch(0, t0);
      put(0);
    }
    int t = t0, buf = 0;
    bool ok[C::kSub];  // (without holes all true: places past the last key are masked anyway)
#pragma unroll
    for (int x = 0; x < C::kSub; ++x) ok[x] = true;
    // tile t is in LDS and every wavefront done with the one before: the next one is set
    // on its way; whether every row sees all of this one
    auto open = [&]() __attribute__((always_inline)) {
      if constexpr (C::k8) __syncthreads();
      else wait_barrier<0>();
      if (t + 1 < t1) fetch(buf ^ 1, t + 1);
      bool whole = t * K >= all_lo && t * K + K <= all_hi;
      if (holes) {
#pragma unroll
        for (int x = 0; x < C::kSub; ++x) {
          ok[x] = run_exists(t, x);
          whole = whole && ok[x];
        }
      }
      return whole;
    };
    auto close = [&]() __attribute__((always_inline)) {
      if (t + 1 < t1) put(buf ^ 1);
      ++t;
      buf ^= 1;
    };
    // (two loops, so that the results keep their registers from one whole tile to the next)
    if (t < t1) {
      bool whole = open();
      for (;;) {
        while (whole) {
          step(std::false_type{}, buf, t * K, ok);
          close();
          if (t >= t1) break;
          whole = open();
        }
        if (t >= t1) break;
        step(std::true_type{}, buf, t * K, ok);
        close();
        if (t >= t1) break;
        whole = open();
      }
    }

    // what was taken out, as marks times the keys that a row sees
    for (t = t0; some_odd && t < t1; ++t) {
      const int key0 = t * K;
      bool whole = key0 >= all_lo && key0 + K <= all_hi;
#pragma unroll
      for (int x = 0; x < C::kSub; ++x) {
        ok[x] = !holes || run_exists(t, x);
        whole = whole && ok[x];
      }
      if (whole) continue;
      __syncthreads();
      page = my_page(t);
      fetch(0, t);
      put(0);
      if constexpr (C::k8) __syncthreads();
      else wait_barrier<0>();
      char *const vt = lds + C::kTile;
      clear_unseen(vt, key0, ok);
      for (int y = 0; y < C::kTile / 16 / kThreads; ++y) {
        v8bf *const v = reinterpret_cast<v8bf *>(vt) + y * kThreads + tid;
        *v = odd_part<true>(*v);
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll 1
      for (int x = 0; x < 2 * NB; ++x) {  // 16 keys: a sum of marks can count them
        bool there_x = ok[0];
#pragma unroll
        for (int j = 1; j < C::kSub; ++j) there_x = x == j ? ok[j] : there_x;
        v4i one = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int key = key0 + 16 * x + 8 * (j / 4) + 4 * half + j % 4;
          one[j / 2] |= key >= lo && key < hi && there_x ? 0x3f80 << 16 * (j & 1) : 0;
        }
#pragma unroll
        for (int d = 0; d < C::kOut; ++d) {
          const v16f marks = mfma32bf(value_frag<D>(vt, 16 * x, d, lane),
                                      __builtin_bit_cast(v8bf, one), v16f{});
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] = add_odd(o[d][i], marks[i]);
        }
      }
    }

    l = halves_sum(l);
    if (there) {
      m = seen_max(m, l, c, table, lo > t0 * K ? lo : t0 * K, hi < t1 * K ? hi : t1 * K);
      if (un.pieces == 1) {
        const float inv = inverse_sum(l, m);
        uint16_t *dst = a.out + (int64_t)(un.w.s.start + tok) * a.ld_out +
                        (h * a.group + row % a.group) * D + 4 * half;
#pragma unroll
        for (int d = 0; d < C::kOut; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<v2i_e2 *>(dst + 32 * d + 8 * i) =
                v2i{(int)bf16x2(o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                    (int)bf16x2(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
      } else {
        const int64_t at = ((int64_t)h * part.slots + un.slot) * kTileRows + (row - r0);
#pragma unroll
        for (int d = 0; d < C::kOut; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<v4f *>(part.o + at * D + 32 * d + 8 * i + 4 * half) =
                v4f{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        if (half == 0) {
          part.ml[2 * at] = m;
          part.ml[2 * at + 1] = l;
        }
      }
    }
    __syncthreads();  // LDS is the next unit's
  }
}

template <int D, int kFormat>
hipError_t launch(const AttnArgs &a, const CacheView &c, const BatchView &b, const AttnPlan &p,
                  float *partial, hipStream_t st) {
  return launch_kernel(tiles_kernel<D, kFormat>, dim3(p.tile_grid * c.kv_heads), dim3(kThreads), st,
                       {}, a, c, b, p.tile_target, partial_many(p, c.kv_heads, D, partial));
}
template <int D>
hipError_t launch(const AttnArgs &a, const CacheView &c, int format, const BatchView &b,
                  const AttnPlan &p, float *partial, hipStream_t st) {
  if (format == kBf16Cache) return launch<D, kBf16Cache>(a, c, b, p, partial, st);
  if (format == MOE_W8A8_FORMAT_FP8)
    return launch<D, MOE_W8A8_FORMAT_FP8>(a, c, b, p, partial, st);
  return launch<D, MOE_W8A8_FORMAT_INT8>(a, c, b, p, partial, st);
}

}  // namespace

hipError_t launch_attention_tiles(const AttnArgs &a, const CacheView &c, int D, int format,
                                  const BatchView &b, const AttnPlan &p, float *partial,
                                  hipStream_t st) {
  if (D == 64) return launch<64>(a, c, format, b, p, partial, st);
  if (D == 128) return launch<128>(a, c, format, b, p, partial, st);
  return launch<256>(a, c, format, b, p, partial, st);
}

}  // namespace moe
