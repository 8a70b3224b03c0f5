// attention_rows.hip -- attention of few query rows of each kv head over the paged
// cache (decode steps). A row is one query head of one token; the rows of the heads
// that share a kv head are taken together, 16 to a matrix instruction.
//
// With keys as the instruction's rows and queries as its columns, lane l holds the
// scores of query l % 16 and of the keys 4 (l / 16) + 0..3: the softmax runs inside
// lanes but for one exchange over the four lane groups, and the probabilities are
// where the second product (values transposed by the LDS reads) takes them from.
// Bound by the cache's bytes (8 sequences of 65536 keys, 8 kv heads of 128, FP8: 1.1 GB in
// 196 us, 5.7 TB/s; 32 ragged ones of 1 to 8192, INT8: 174 MB in 48, of which about 6 are its
// beginning and end). Every wavefront brings its own tiles of 32 keys into
// LDS by direct loads, the next in flight while one is worked on, and no two of them
// meet until the end.
#include "attention_device.h"
#include "attention_work.h"

namespace moe {
namespace {

constexpr int kKeys = kFewKeys;

template <int D, int kFormat, int NQ>
struct Rows {
  typedef Tile<D, kFormat, kKeys> TL;
  static constexpr int kScaleBytes = TL::k8 ? 256 : 0;
  static constexpr int kStage = 2 * TL::kBytes + kScaleBytes;
  static constexpr int kWaves = 4 * 2 * kStage <= 150 * 1024 ? 4 : 2;
  static constexpr int kRows = 16 * NQ;
  static constexpr int kLoads = 2 * TL::kLoads + (TL::k8 ? 1 : 0);
  // joining the wavefronts: their results of 16 rows each, and (m, l) of all rows
  static constexpr int kPad = D + 4;
  static constexpr int kJoin = kWaves * 16 * kPad * 4;
  static constexpr int kStages = kWaves * 2 * kStage;
  static constexpr int kLds = kStages > kJoin ? kStages : kJoin;
};

template <int D, int kFormat, int NQ>
__global__ __launch_bounds__((64 * Rows<D, kFormat, NQ>::kWaves)) void rows_kernel(
    AttnArgs a, CacheView c, BatchView bt, int target, Partial part) {
  typedef Rows<D, kFormat, NQ> C;
  typedef typename C::TL TL;
  constexpr int W = C::kWaves, kSteps = D / 32, kOut = D / 16;
  __shared__ __attribute__((aligned(1024))) char lds[C::kLds];
  __shared__ float ml[W][C::kRows][2];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
  const int h = blockIdx.x % c.kv_heads;
  const Schedule<true, kKeys> work(a, bt, target, kLeastFew, kLeastFew);
  const int chunk = work.chunk;
  const int page_size = 1 << c.log2_page;
  char *const mine = lds + wave * 2 * C::kStage;
  const uint32_t mine_at = __builtin_amdgcn_readfirstlane(lds_addr(mine));

  // Direct loads of 1 KB: which chunks the lanes read depends on the load's rows, the
  // same 16 rows on (but for 8-bit values).
  constexpr int kHalf = TL::kLoads / 2, kValueKinds = TL::k8 ? TL::kLoads : kHalf;
  uint32_t key_lane[kHalf], value_lane[kValueKinds];
#pragma unroll
  for (int i = 0; i < TL::kLoads; ++i) {
    const int in = i * 1024 + lane * 16, r = in / TL::kRow, p = in % TL::kRow / 16;
    const int row = lane * 16 / TL::kRow * TL::kRow;
    if (i < kHalf) key_lane[i] = row + TL::key_chunk(r, p) * 16;
    if (i < kValueKinds) value_lane[i] = row + TL::value_chunk(r, p) * 16;
  }

  for (int u = blockIdx.x / c.kv_heads;; u += gridDim.x / c.kv_heads) {
    const Unit un = work.find(a, bt, u);
    if (un.b < 0) break;
    const int len = un.w.s.len, first = len - un.w.s.n;
    // keys that some row, and that every row sees
    const int rows = un.w.rows, p0 = first, p1 = first + (rows - 1) / a.group;
    const int any_lo = seen_lo(p0, a.window), any_hi = seen_hi(p1, len, a.causal);
    const int all_lo = seen_lo(p1, a.window), all_hi = seen_hi(p0, len, a.causal);
    const int t0 = un.w.t0 + un.piece * chunk;
    const int end = un.w.t0 + un.w.keys, t1 = t0 + chunk < end ? t0 + chunk : end;

    // queries, and what each sees
    v8bf q[NQ][kSteps];
    int lo[NQ], hi[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      // (a lane past the last row takes that one again and sees nothing)
      const bool there = n * 16 + col < rows;
      const int r = there ? n * 16 + col : rows - 1, i = r / a.group;
      lo[n] = seen_lo(first + i, a.window);
      hi[n] = there ? seen_hi(first + i, len, a.causal) : 0;
      const uint16_t *src =
          a.q + (int64_t)(un.w.s.start + i) * a.ld_q + (h * a.group + r % a.group) * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        q[n][s] = __builtin_bit_cast(
            v8bf, (v4i)*reinterpret_cast<const v4i_a2 *>(src + TL::query_at(s, lane)));
    }

    // direct loads of tile t into a stage; a page that does not exist is read as page 0
    // and masked
    auto page_of = [&](int key) {
      const int i = key >> c.log2_page;
      return key < any_hi ? scalar_word(bt.table, (int64_t)un.b * bt.ld_table + i) : -1;
    };
    auto issue = [&](int stage, int t, int pg0, int pg1) {
      const int64_t in0 = ((int64_t)h * page_size + (t * kKeys & (page_size - 1)));
      const int64_t in1 = ((int64_t)h * page_size + ((t * kKeys + 16) & (page_size - 1)));
      const int64_t s0 = (uint32_t)pg0 < (uint32_t)c.num_pages ? pg0 : 0;
      const int64_t s1 = (uint32_t)pg1 < (uint32_t)c.num_pages ? pg1 : 0;
      const int64_t b0 = s0 * c.page_bytes + in0 * TL::kRow, b1 = s1 * c.page_bytes + in1 * TL::kRow;
      const uint32_t at = mine_at + stage * C::kStage;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < TL::kLoads; ++i)
          dma16((x ? c.v : c.k) + (i < kHalf ? b0 + i * 1024 : b1 + (i - kHalf) * 1024),
                x ? value_lane[i % kValueKinds] : key_lane[i % kHalf],
                at + x * TL::kBytes + i * 1024);
      if constexpr (TL::k8) {
        const float *sc = lane < 32 ? c.k_scale : c.v_scale;
        const int r = lane & 31;
        dma4(sc + (r < 16 ? s0 * c.scale_stride + in0 : s1 * c.scale_stride + in1) + (r & 15),
             at + 2 * TL::kBytes);
      }
    };

    v4f o[NQ][kOut];
    float m[NQ], l[NQ];
    uint32_t some[NQ];  // whether this lane's keys of a row are seen at all
    int t, stage, pg0, pg1, ng0, ng1;
    auto begin = [&]() __attribute__((always_inline)) {
      t = t0 + wave;
      stage = 0;
      pg0 = pg1 = ng0 = ng1 = -1;
      if (t < t1) {
        pg0 = page_of(t * kKeys);
        pg1 = page_of(t * kKeys + 16);
        issue(0, t, pg0, pg1);
        ng0 = page_of((t + W) * kKeys);
        ng1 = page_of((t + W) * kKeys + 16);
      }
    };
    begin();
    // Tiles that all rows see are not searched for values that are not finite: one of those
    // shows in a result, and the wavefront takes its tiles again, searching all. (Of codes
    // only the scales can be infinite, whose rests are 0.)
    for (bool careful = false;; careful = true) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = kNoMax;
        l[n] = 0.0f;
        some[n] = 0;
#pragma unroll
        for (int d = 0; d < kOut; ++d) o[n][d] = v4f{0, 0, 0, 0};
      }
      for (; t < t1; t += W, stage ^= 1) {
        // the stage of the tile before this one has been read to its end
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (t + W < t1) {
          issue(stage ^ 1, t + W, ng0, ng1);
          asm volatile("s_waitcnt vmcnt(%0)" ::"n"(C::kLoads) : "memory");
        } else {
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        char *const kt = mine + stage * C::kStage, *const vt = kt + TL::kBytes;
        const float *const sc = reinterpret_cast<const float *>(vt + TL::kBytes);
        const int key0 = t * kKeys;
        const bool ok0 = (uint32_t)pg0 < (uint32_t)c.num_pages,
                   ok1 = (uint32_t)pg1 < (uint32_t)c.num_pages;
        const bool masked = !(key0 >= all_lo && key0 + kKeys <= all_hi && ok0 && ok1);
        pg0 = ng0;
        pg1 = ng1;
        ng0 = page_of((t + 2 * W) * kKeys);
        ng1 = page_of((t + 2 * W) * kKeys + 16);
        if (masked) {
          // values that no row sees count as zeros, whatever lies there
          for (int y = 0; y < TL::kBytes / 1024; ++y) {
            const int i = y * 64 + lane, r = i / TL::kChunks, key = key0 + r;
            const bool gone = (key < any_lo) | (key >= any_hi) | !(r < 16 ? ok0 : ok1);
            v4i v = reinterpret_cast<const v4i *>(vt)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = gone ? 0 : v[j];
            reinterpret_cast<v4i *>(vt)[i] = v;
          }
        }

        // scores: keys 16 x + 4 g + i of column col
        v4f s[NQ][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[n][0] = s[n][1] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if constexpr (TL::k8) {
#pragma unroll
            for (int s2 = 0; s2 < kSteps / 2; ++s2) {
              v8bf f[2];
              TL::key2(kt, 16 * x, s2, lane, f);
#pragma unroll
              for (int n = 0; n < NQ; ++n) {
                s[n][x] = mfma16bf(f[0], q[n][2 * s2], s[n][x]);
                s[n][x] = mfma16bf(f[1], q[n][2 * s2 + 1], s[n][x]);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
              const v8bf f = TL::key(kt, 16 * x, i, lane);
#pragma unroll
              for (int n = 0; n < NQ; ++n) s[n][x] = mfma16bf(f, q[n][i], s[n][x]);
            }
          }
        }
        v4f ks[2], vs[2];
        if constexpr (TL::k8) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            ks[x] = *reinterpret_cast<const v4f *>(sc + 16 * x + 4 * g);
            vs[x] = *reinterpret_cast<const v4f *>(sc + 32 + 16 * x + 4 * g);
          }
        }
        v8bf p[NQ], rest[NQ];
        uint32_t seen[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float mx = kNoMax;
          seen[n] = 0xffu;
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v = s[n][x][i] * a.scale2;
              if constexpr (TL::k8) v *= ks[x][i];
              if (masked) {
                const int key = key0 + 16 * x + 4 * g + i;
                const bool there = key >= lo[n] && key < hi[n] && (x ? ok1 : ok0);
                v = there ? v : -INFINITY;
                seen[n] &= ~((uint32_t)!there << (4 * x + i));
              }
              s[n][x][i] = v;
              mx = fmaxf(mx, v);
            }
          some[n] |= seen[n];
          mx = fmaxf(m[n], groups_max(mx));
          const float f = __builtin_amdgcn_exp2f(m[n] - mx);
          m[n] = mx;
          float e[8], sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            e[j] = __builtin_amdgcn_exp2f(s[n][j / 4][j % 4] - mx);
            sum += e[j];
            if constexpr (TL::k8) {
              e[j] *= vs[j / 4][j % 4];
              e[j] = masked && !(seen[n] >> j & 1) ? 0.0f : e[j];
            }
          }
          l[n] = l[n] * f + sum;
          // two bf16 terms for the second product, whose matrix instructions are few here: the
          // rest of what the first one rounds, 2^-17 of the probability at most left out. (With one
          // term a key that has all the weight moves its row by up to 2^-9: 32 sequences of 8192,
          // INT8, 108 us instead of 110, with 8 tokens each 180 instead of 191, but the result's
          // error half again that of its rounding.)
          v4i w, r;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] = (int)bf16x2(e[2 * j], e[2 * j + 1]);
            float lo[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t u = (uint32_t)w[j];
              const float hi = __uint_as_float(i ? u & 0xffff0000u : u << 16);
              lo[i] = e[2 * j + i] - hi;
              if constexpr (TL::k8) lo[i] = fabsf(hi) < INFINITY ? lo[i] : 0.0f;  // (such a scale)
            }
            r[j] = (int)bf16x2(lo[0], lo[1]);
          }
          p[n] = __builtin_bit_cast(v8bf, w);
          rest[n] = __builtin_bit_cast(v8bf, r);
#pragma unroll
          for (int d = 0; d < kOut; ++d) o[n][d] *= f;
        }
        // values that are not finite, in a tile of which some rows do not see all: an
        // unseen one must not reach a row through 0 times infinity, nor one that is seen
        // through the rest of its probability, which may be 0 or negative. They are taken
        // out, and put back as indicators times the keys that a row sees.
        bool odd = false;
        if (masked || careful) {
#pragma unroll
          for (int d = 0; d < kOut; ++d) odd |= any_odd(TL::value(vt, 0, d, lane));
          odd = __any(odd);
        }
        if (!odd) {
#pragma unroll
          for (int d = 0; d < kOut; ++d) {
            const v8bf f = TL::value(vt, 0, d, lane);
#pragma unroll
            for (int n = 0; n < NQ; ++n) o[n][d] = mfma16bf(f, rest[n], mfma16bf(f, p[n], o[n][d]));
          }
        } else {
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            v4i one = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (seen[n] >> j & 1) one[j / 2] |= 0x3f80 << 16 * (j & 1);
            const v8bf sees = __builtin_bit_cast(v8bf, one);
#pragma unroll
            for (int d = 0; d < kOut; ++d) {
              const v8bf f = TL::value(vt, 0, d, lane);
              const v4f marks = mfma16bf(odd_part<true>(f), sees, v4f{0, 0, 0, 0});
              o[n][d] = mfma16bf(odd_part<false>(f), p[n], o[n][d]);
              o[n][d] = mfma16bf(odd_part<false>(f), rest[n], o[n][d]);
#pragma unroll
              for (int i = 0; i < 4; ++i) o[n][d][i] = add_odd(o[n][d][i], marks[i]);
              __builtin_amdgcn_sched_barrier(0);  // (this path need not be fast: few registers)
            }
          }
        }
      }
      if (TL::k8 || careful) break;
      v4f odd = {0, 0, 0, 0};
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int d = 0; d < kOut; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) odd[i] = __builtin_fmaf(o[n][d][i], 0.0f, odd[i]);
      if (!__any(odd[0] + odd[1] + (odd[2] + odd[3]) != 0.0f)) break;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (the stages are free again)
      begin();
    }

    // join the wavefronts: o / l with the weights exp2(m - largest m)
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] = groups_sum(l[n]);
      const float seen = groups_max(some[n] ? kSeenMax : kNoMax);
      if (g == 0) {
        ml[wave][n * 16 + col][0] = l[n] != 0.0f ? m[n] : seen;
        ml[wave][n * 16 + col][1] = l[n];
      }
    }
    __syncthreads();
    const bool whole = un.pieces == 1;
    float *const jo = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float big = ml[0][n * 16 + col][0];
#pragma unroll
      for (int w = 1; w < W; ++w) big = fmaxf(big, ml[w][n * 16 + col][0]);
      const float f = __builtin_amdgcn_exp2f(m[n] - big);
#pragma unroll
      for (int d = 0; d < kOut; ++d)
        *reinterpret_cast<v4f *>(jo + (wave * 16 + col) * C::kPad + d * 16 + 4 * g) = o[n][d] * f;
      __syncthreads();
      for (int i = tid; i < 16 * D / 4; i += 64 * W) {
        const int r = i / (D / 4), d = i % (D / 4) * 4, row = n * 16 + r;
        if (row >= rows) continue;
        float mm = ml[0][row][0], ll = 0.0f;
        for (int w = 1; w < W; ++w) mm = fmaxf(mm, ml[w][row][0]);
        v4f v = {0, 0, 0, 0};
        for (int w = 0; w < W; ++w) {
          ll += ml[w][row][1] * __builtin_amdgcn_exp2f(ml[w][row][0] - mm);
          v += *reinterpret_cast<const v4f *>(jo + (w * 16 + r) * C::kPad + d);
        }
        if (whole) {
          v *= inverse_sum(ll, mm);
          uint16_t *dst = a.out + (int64_t)(un.w.s.start + row / a.group) * a.ld_out +
                          (h * a.group + row % a.group) * D + d;
          *reinterpret_cast<v2i_e2 *>(dst) = v2i{(int)bf16x2(v[0], v[1]), (int)bf16x2(v[2], v[3])};
        } else {
          const int64_t at = ((int64_t)h * part.slots + un.slot) * C::kRows + row;
          *reinterpret_cast<v4f *>(part.o + at * D + d) = v;
          if (d == 0) {
            part.ml[2 * at] = mm;
            part.ml[2 * at + 1] = ll;
          }
        }
      }
      __syncthreads();
    }
  }
}

template <int D, int kFormat, int NQ>
hipError_t launch(const AttnArgs &a, const CacheView &c, const BatchView &b, const AttnPlan &p,
                  float *partial, hipStream_t st) {
  typedef Rows<D, kFormat, NQ> C;
  return launch_kernel(rows_kernel<D, kFormat, NQ>, dim3(p.row_grid * c.kv_heads),
                       dim3(64 * C::kWaves), st, {}, a, c, b, p.row_target,
                       partial_few(p, c.kv_heads, D, partial));
}
template <int D, int kFormat>
hipError_t launch(const AttnArgs &a, const CacheView &c, const BatchView &b, const AttnPlan &p,
                  float *partial, hipStream_t st) {
  if constexpr (D < 256)
    if (p.row_tiles == 2) return launch<D, kFormat, 2>(a, c, b, p, partial, st);
  return launch<D, kFormat, 1>(a, c, b, p, partial, st);
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

hipError_t launch_attention_rows(const AttnArgs &a, const CacheView &c, int D, int format,
                                 const BatchView &b, const AttnPlan &p, float *partial,
                                 hipStream_t st) {
  if (D == 64) return launch<64>(a, c, format, b, p, partial, st);
  if (D == 128) return launch<128>(a, c, format, b, p, partial, st);
  return launch<256>(a, c, format, b, p, partial, st);
}

}  // namespace moe
