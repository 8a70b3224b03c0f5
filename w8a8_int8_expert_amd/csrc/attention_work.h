// attention_work.h -- how attention's work is cut into units, on the device (lengths
// are known only there). Each kernel takes the sequences of its kind: of few rows (one
// block of rows), or of many (blocks of kTileRows). The keys of a row block are cut
// into pieces of `chunk` key tiles, a chunk such that all pieces of a kv head are about
// `target`; a unit is one piece of one row block. Every wavefront finds its units by
// itself, its lanes reading 64 sequences at a time. Included by the HIP sources only.
#pragma once

#include "attention_internal.h"

namespace moe {

struct Work {
  Seq s;
  int rows, blocks;  // query rows of a kv head, and blocks of them; 0: not of this kind
  int t0, keys;      // first key tile (few rows), and key tiles of the row block that has most
};
// Of a sequence's row blocks the last one sees the most keys; without the causal limit the
// first one: a token then sees the window before it and all that follows. (Written as later
// steps, not as a choice: 8192 tokens, 16 heads of 256, bf16, 902 us, 937 otherwise.)
template <bool kFew, int kKeys>
__device__ __forceinline__ Work work_of(const AttnArgs &a, const BatchView &bt, int b) {
  Work w{};
  if (b >= bt.num_seqs) return w;
  w.s = seq_of(bt, b);
  const int n = w.s.n < bt.max_tokens ? w.s.n : bt.max_tokens;
  if (n > 0 && (n <= a.few_rows / a.group) == kFew) {
    w.rows = n * a.group;
    w.blocks = kFew ? 1 : (w.rows + kTileRows - 1) / kTileRows;
    const int first = w.s.len - w.s.n;
    int lo = seen_lo(first + (w.blocks - 1) * kTileRows / a.group, a.window);
    if (!a.causal) lo = seen_lo(first, a.window);
    const int hi = seen_hi(first + n - 1, w.s.len, a.causal);
    w.t0 = lo / kKeys;
    w.keys = hi > lo ? (hi + kKeys - 1) / kKeys - w.t0 : 0;
  }
  return w;
}

// Pieces of many rows: about 1024 in all, of 512 keys at least. 12 sequences of up to 512 tokens
// over 16384 keys take 387 us, 379 with 1536 pieces and 388 with 2048; 9 of up to 613 tokens with
// a window of 1000 take 43.5, 44.9 and 47.3, and 48.5 with pieces of 256 keys. A lone chunk of 64
// tokens, 32 heads over 8 of 128, bf16, with pieces of 512, 256 and 128 keys at least: over 1024
// keys 28, 24 and 22 us, over 4096 31, 30 and 40, over 16384 50, 87 and 88 (the join takes a
// row's pieces one after the other). Of few rows one round of blocks (rows_per_unit), of 128 keys
// at least, a tile for each wavefront.
struct Unit {
  int b;  // the sequence; -1: there are no more units
  int block, piece, pieces;
  int slot;  // of the partial result, where there is more than one piece
  Work w;
};
template <bool kFew, int kKeys>
struct Schedule {
  Work first;  // this lane's of sequences 0 .. 63
  int chunk, lane;

  __device__ __forceinline__ Schedule(const AttnArgs &a, const BatchView &bt, int target, int least,
                                      int step) {
    lane = threadIdx.x & 63;
    first = work_of<kFew, kKeys>(a, bt, lane);
    uint64_t sum = (uint64_t)first.blocks * (uint64_t)first.keys;
    for (int b0 = 64; b0 < bt.num_seqs; b0 += 64) {
      const Work w = work_of<kFew, kKeys>(a, bt, b0 + lane);
      sum += (uint64_t)w.blocks * (uint64_t)w.keys;
    }
    uint64_t c = (wave_sum_u64(sum) + target - 1) / target;
    if (c > 1u << 30) c = 1u << 30;  // (past any sequence's tiles)
    const int n = (int)((c + step - 1) / step) * step;
    chunk = n > least ? n : least;
  }
  __device__ __forceinline__ int pieces_of(const Work &w) const {
    const int n = (w.keys + chunk - 1) / chunk;
    return n > 1 ? n : 1;
  }
  // Unit u: of each sequence its row blocks from the one that sees the most keys (the long
  // ones come first), each piece by piece. Only row blocks of two pieces or more have slots;
  // those are counted with more tiles than a chunk, so that their pieces are at most 2 target
  // of a kv head.
  // kSlots: u is a slot, not a unit.
  template <bool kSlots = false>
  __device__ __forceinline__ Unit find(const AttnArgs &a, const BatchView &bt, int64_t u) const {
    int64_t before = 0;
    int slots = 0;
    for (int b0 = 0; b0 < bt.num_seqs; b0 += 64) {
      const Work w = b0 ? work_of<kFew, kKeys>(a, bt, b0 + lane) : first;
      const int p = pieces_of(w), ns = p > 1 ? w.blocks * p : 0, n = kSlots ? ns : w.blocks * p;
      const int upto = wave_incl_scan(n), supto = slots + wave_incl_scan(ns);
      const uint64_t hit = __ballot(before + upto > u);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        auto rd = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
        Unit r;
        r.b = b0 + l;
        r.pieces = rd(p);
        const int at = (int)(u - before) - (rd(upto) - rd(n));
        r.block = rd(w.blocks) - 1 - at / r.pieces;
        if (!a.causal) r.block = at / r.pieces;
        r.piece = at % r.pieces;
        r.slot = rd(supto) - rd(ns) + at;
        r.w.s = Seq{rd(w.s.start), rd(w.s.n), rd(w.s.len)};
        r.w.rows = rd(w.rows);
        r.w.blocks = rd(w.blocks);
        r.w.t0 = rd(w.t0);
        r.w.keys = rd(w.keys);
        return r;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
      slots = __builtin_amdgcn_readlane(supto, 63);
    }
    Unit r{};
    r.b = -1;
    return r;
  }
};

}  // namespace moe
