// How latent attention's work is cut on the device, where the lengths are: blocks of kBM query rows (tokens x heads) of one
// sequence, and where there are fewer of them than workgroups fit the card, parts of a block along its keys.
#pragma once

#include "device_latent.h"
#include "latent.h"

namespace bfp8 {

namespace {

struct Desc {  // a block that was cut: its first query row (token * H + head) and rows, partial states slot .. slot + parts - 1
  int first, rows, slot, parts;
};

// Sequence b's chunk of new tokens.
struct Seq {
  int q0, n, len;  // first query token, query tokens, keys
};
__device__ __forceinline__ Seq sequence(const LatentAttnArgs& a, int b) {
  Seq s;
  if (a.cu_q != nullptr) {
    const int lo = min(max(a.cu_q[b], 0), a.T), hi = min(max(a.cu_q[b + 1], 0), a.T);
    s.q0 = lo;
    s.n = max(hi - lo, 0);
  } else {
    s.q0 = b;
    s.n = 1;
  }
  // A length far past the table is as good as one of which every new token sees a key past it (its row is NaN).
  const unsigned reach = (unsigned)a.cache.table_width * (unsigned)a.cache.page_size;  // below 2^31
  s.len = min(max(a.lens[b], 0), (int)min(reach + (unsigned)s.n + 1u, (unsigned)INT32_MAX - 64u));
  return s;
}

// What a workgroup computes: part `part` of `parts` of a block, and where its state goes (-1: nowhere).
struct Work {
  Seq seq;
  int index, block, part, parts, slot;
  int id;  // of all parts (a block's are neighbours)
};

// Every wave cuts the work in the same way and picks its workgroup's part. False: there is none. kHeld: sequences of a lane that are read once.
template <int kBM, int kTile, int kHeld = 4>
__device__ __forceinline__ bool find_work(const LatentAttnArgs& a, Work& work) {
  constexpr int kMany = 1 << 16;  // more parts than ever run at once: sums of 64 such stay in range
  const int lane = threadIdx.x & 63;
  const int per = (a.B + 63) / 64;
  const int b0 = min(lane * per, a.B), count = min(per, a.B - b0);
  auto blocks_of = [&](const Seq& q) { return (int)(((int64_t)q.n * a.H + kBM - 1) / kBM); };
  auto tiles_of = [&](const Seq& q) { return min((q.len + kTile - 1) / kTile, a.max_tiles); };
  Seq held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    held[k] = {0, 0, 0};
    if (k < per && k < count) held[k] = sequence(a, b0 + k);
  }
  // (up to 64 sequences are one a lane: nothing else is stepped through)
  auto each = [&](auto f) {
    if (count > 0) f(b0, held[0], blocks_of(held[0]), tiles_of(held[0]));
    if (per > 1) {
#pragma unroll
      for (int k = 1; k < kHeld; ++k)
        if (k < count) f(b0 + k, held[k], blocks_of(held[k]), tiles_of(held[k]));
      for (int k = kHeld; k < count; ++k) {
        const Seq q = sequence(a, b0 + k);
        f(b0 + k, q, blocks_of(q), tiles_of(q));
      }
    }
  };
  auto cut = [](int tiles, int quantum) {  // max(ceil(tiles / quantum), 1)
    int c = (int)((float)(tiles + quantum - 1) * __builtin_amdgcn_rcpf((float)quantum));
    c += c * quantum < tiles;             // (the quotient by reciprocal is off by one at most)
    c -= c > 0 && (c - 1) * quantum >= tiles;
    return max(c, 1);
  };
  auto total = [](int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); };
  // The quantum: the least number of tiles a part with which the parts do not pass the
  // workgroups that run at once. With as many blocks as that, none is cut.
  int quantum = max(a.max_tiles, 1);
  int64_t blocks = 0;
  each([&](int, const Seq&, int n, int) { blocks += n; });
  const int all_blocks = total((int)min(blocks, (int64_t)kMany));
  const bool rounds = all_blocks > a.target_parts;  // workgroups run one after the other
  if (a.max_slots > 0) {
    if (all_blocks < a.target_parts) {
      int lo = a.min_tiles, hi = max(quantum, lo);
      // All blocks' tiles S bound it: S / q <= parts <= S / q + blocks. (Tables that reach far further than 2^27 tokens are searched through.)
      if (quantum < INT32_MAX / a.target_parts) {
        int tiles_in_all = 0;
        each([&](int, const Seq&, int n, int tiles) { tiles_in_all += n * tiles; });
        tiles_in_all = total(tiles_in_all);
        auto up = [&](int by) { return (int)(((unsigned)tiles_in_all + (unsigned)by - 1u) / (unsigned)by); };
        lo = min(max(up(a.target_parts), lo), hi);
        hi = min(max(up(a.target_parts - all_blocks), lo), hi);
      }
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        int64_t parts = 0;
        each([&](int, const Seq&, int n, int tiles) { parts += (int64_t)n * cut(tiles, mid); });
        if (total((int)min(parts, (int64_t)kMany)) <= a.target_parts) hi = mid;
        else lo = mid + 1;
      }
      quantum = lo;
    }
  }
  int parts = 0, slots = 0, cuts = 0;  // of this lane's sequences
  each([&](int, const Seq&, int n, int tiles) {
    const int c = cut(tiles, quantum);
    parts += n * c;
    if (c > 1) slots += n * c, cuts += n;
  });
  int p0 = wave_scan(parts), s0 = wave_scan(slots), c0 = wave_scan(cuts);
  const int cut_blocks = __builtin_amdgcn_readlane(c0, 63);
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.counts != nullptr) a.counts[0] = cut_blocks;
  p0 -= parts, s0 -= slots, c0 -= cuts;
  if (rounds && a.B <= 64) {
    // the longest sequences' blocks first: the last ones to start are short (6 chunks of 40 tokens behind 700 to
    // 3500 keys, 480 blocks: 190 us in the given order, 148 us so)
    const int t = count > 0 ? tiles_of(held[0]) : 0;
    p0 = 0;
    for (int j = 0; j < a.B; ++j) {
      const int other = __builtin_amdgcn_readlane(t, j), n = __builtin_amdgcn_readlane(parts, j);
      p0 += other > t || (other == t && j < lane) ? n : 0;
    }
  }
  // pairs of parts (the two blocks of a token's 128 heads, most often) go to one XCD (blockIdx % 8), and
  // share its L2
  const int my = (int)(((blockIdx.x >> 4) * 8 + (blockIdx.x & 7)) * 2 + ((blockIdx.x >> 3) & 1));
  const bool mine = my >= p0 && my < p0 + parts;
  const uint64_t who = __ballot(mine);
  if (who == 0) return false;
  Work w{};
  if (mine) {
    bool found = false;
    each([&](int b, const Seq& q, int n, int tiles) {
      const int c = cut(tiles, quantum);
      if (!found && my < p0 + n * c) {
        const int blk = (my - p0) / c, part = (my - p0) - blk * c;
        w = {q, b, blk, part, c, c > 1 ? s0 + blk * c + part : -1, my};
        if (c > 1 && part == 0 && c0 + blk < a.max_cuts && threadIdx.x < 64)
          reinterpret_cast<Desc*>(a.counts + 4)[c0 + blk] = {
              (int)((int64_t)q.q0 * a.H + (int64_t)blk * kBM), (int)min((int64_t)q.n * a.H - (int64_t)blk * kBM, (int64_t)kBM),
              s0 + blk * c, c};
        found = true;
      }
      p0 += n * c;
      if (c > 1) s0 += n * c, c0 += n;
    });
  }
  const int src = __builtin_ctzll(who);
  auto from = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
  work = {{from(w.seq.q0), from(w.seq.n), from(w.seq.len)}, from(w.index), from(w.block), from(w.part), from(w.parts),
          from(w.slot), my};
  // starts that are not rising could ask for more (nothing is promised for them)
  return work.slot < 0 || work.slot - work.part + work.parts <= a.max_slots;
}

}  // namespace

}  // namespace bfp8
