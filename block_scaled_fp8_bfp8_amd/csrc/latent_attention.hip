// Latent attention over the paged FP8 latent cache, in the absorbed form: every head of a query
// token reads the same cached row, as key (512 latents and the rotary key) and as value (latents).
//
//   o[t, h] = sum_j softmax_j(scale * q[t, h] . [c_j, r_j]) c_j,   c_j = 2^(e_j) * codes_j
//
// over the keys j that token t sees (its own sequence up to itself).
//
// Both products run on the FP8 matrix cores, on the cached codes as they are:
//   * scores: a bf16 query has 8 significant bits, so it is the sum of two e4m3 values
//     (hi: its top 4 bits; lo: the rest, scaled 2^4), both under one power-of-two scale a row.
//     Two scaled FP8 products cost as many matrix-core clocks as one bf16 product, and the
//     codes need no conversion. The key's scale code is the instruction's row scale. The rotary
//     part is a bf16 product into the same accumulator.
//   * values: the weight p_j and the key's scale are one number, p_j 2^(e_j) = 2^(x_j) with
//     x_j = scale log2(e) s_j + e_j, kept relative to the row's running maximum of x (not of
//     s), split into hi + lo e4m3 in the same way (at least 8 significant bits, as bf16 would
//     have). The softmax denominator sums 2^(x_j) 2^(-e_j) in float32.
// The products are formed transposed (S^T = K Q^T, O^T = V^T P^T) with 32x32x64 instructions: a
// lane holds 16 scores of one query row, r = lane % 32, for keys 8 q + 4 g + i (g = lane / 32),
// which are at once its operand of the second product. hi and lo fill the two halves of that
// product's 64 slots (the lo half under a scale of 2^-4), against the same 16 value bytes twice.
// Values are read from the key tile with transposing LDS reads.
//
// A workgroup holds 32 query rows a pair of waves; the two waves of a pair take 32 keys each of a
// 64-key tile with maxima and sums of their own, and join when the block's keys are done. So a
// wave's 32 rows x 512 columns of float32 accumulator fill its 256 accumulation registers, the
// queries' two terms 144 of the others, and a key byte read from LDS serves 32 rows: the LDS
// reads of a tile (36 KB a wave) take about half the clocks of its matrix products (16 rows a wave
// and 64 keys each, without the pairs, would read 72 KB for half the products).
//
// Work is cut on the device, where the lengths are: a block is the query rows (tokens x heads)
// of one sequence that a workgroup holds, and where there are fewer blocks than workgroups fit
// the card, they are cut along their keys into parts whose float32 states (accumulator, maximum,
// sum) a second launch joins in order.
#include "device_common.h"
#include "latent.h"
#include "launch.h"

#include <type_traits>

namespace bfp8 {

namespace {

constexpr int kTile = 64;                  // keys of a tile
constexpr int kTileBytes = kTile * kLatentRow;
constexpr int kSlack = 4;                  // the running maximum may lag by a factor of 2^kSlack ...
constexpr float kTop = 8 - kSlack;         // ... so that 2^(x - m + kTop) stays within 2^8 <= 448
constexpr float kNegInf = -__builtin_inff();

struct Desc {  // a block that was cut: rows of block `block`, partial states slot .. slot + parts - 1
  int seq, block, slot, parts;
};

// XOR of the 16-byte columns of a key's 512-byte row in LDS. Conflict-free both for the score
// reads (16 lanes: one column of 16 keys that differ in bits 0 .. 3) and for the transposing value
// reads (32 lanes: two neighbouring columns of 8 keys that differ in bits 0, 1 and 3).
__device__ __forceinline__ int swz(int key) { return ((key & 3) << 1) | (key & 8) | ((key >> 2) & 1); }

__device__ __forceinline__ v16f mfma_scaled(const v8i& a, const v8i& b, const v16f& c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, ea, 0, eb);
}

// The same product added to an accumulator in the accumulation registers. Written in assembly so that it
// stays there: the compiler otherwise moves accumulators between the two register files in bulk. The
// wait in front covers operands that vector instructions have just written.
__device__ __forceinline__ void mfma_scaled_acc(const v8i& a, const v8i& b, v16f& c, int ea, int eb) {
  asm("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
      : "+a"(c)
      : "v"(a), "v"(b), "v"(ea), "v"(eb));
}
// A value that the compiler takes as new here: what is computed from it is formed where it is used, not
// kept in registers across a loop.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
// Keeps an accumulator in the accumulation registers at this point.
__device__ __forceinline__ void keep_acc(v16f& c) { asm volatile("" : "+a"(c)); }

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
  s.len = max(a.lens[b], 0);
  return s;
}

// What a workgroup computes: part `part` of `parts` of a block, and where its state goes (-1: nowhere).
struct Work {
  int seq, block, part, parts, slot;
};

// Every workgroup of kThreads threads cuts the work in the same way and picks its own part. False:
// it has none. `sh`: 64 ints of LDS.
template <int kThreads, int kBM>
__device__ __forceinline__ bool find_work(const LatentAttnArgs& a, int* sh, Work& work) {
  constexpr int kWaves = kThreads / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  // blocks and tiles of this thread's sequences; the first one's are kept
  auto shape = [&](int b, int& n, int& tiles) {
    const Seq s = sequence(a, b);
    n = (int)(((int64_t)s.n * a.H + kBM - 1) / kBM);
    tiles = min((s.len + kTile - 1) / kTile, a.max_tiles);
  };
  int n0 = 0, tiles0 = 0;
  if (b0 < b1) shape(b0, n0, tiles0);
  auto each = [&](auto f) {
    if (b0 < b1) f(b0, n0, tiles0);
    for (int b = b0 + 1; b < b1; ++b) {
      int n, tiles;
      shape(b, n, tiles);
      f(b, n, tiles);
    }
  };
  auto cut = [](int tiles, int quantum) { return max((tiles + quantum - 1) / quantum, 1); };
  int turn = 0;
  auto sum = [&](int64_t v) {  // over the workgroup
#pragma unroll
    for (int mask = 1; mask < 64; mask <<= 1) v += __shfl_xor(v, mask);
    int64_t* s = reinterpret_cast<int64_t*>(sh) + 8 * (turn++ & 1);
    if (lane == 0) s[wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s[w];
    return v;
  };
  int64_t blocks = 0, units = 0;
  each([&](int, int n, int tiles) {
    blocks += n;
    units += (int64_t)n * tiles;
  });
  blocks = sum(blocks);
  // The quantum: the least number of tiles a part with which the parts do not pass the
  // workgroups that run at once. With as many blocks as that, none is cut.
  int quantum = max(a.max_tiles, 1);
  if (a.max_slots > 0 && blocks < a.target_parts) {
    units = sum(units);
    int lo = (int)max((units + a.target_parts - 1) / a.target_parts, (int64_t)a.min_tiles), hi = max(quantum, lo);
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      int64_t parts = 0;
      each([&](int, int n, int tiles) { parts += (int64_t)n * cut(tiles, mid); });
      if (sum(parts) <= a.target_parts) hi = mid;
      else lo = mid + 1;
    }
    quantum = lo;
  }
  int parts = 0, slots = 0, cuts = 0;  // of this thread's sequences
  each([&](int, int n, int tiles) {
    const int c = cut(tiles, quantum);
    parts += n * c;
    if (c > 1) slots += n * c, cuts += n;
  });
  // exclusive sums over the threads
  int p0 = parts, s0 = slots, c0 = cuts;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(p0, d), y = __shfl_up(s0, d), z = __shfl_up(c0, d);
    if (lane >= d) p0 += x, s0 += y, c0 += z;
  }
  __syncthreads();
  if (lane == 63) sh[wave * 3] = p0, sh[wave * 3 + 1] = s0, sh[wave * 3 + 2] = c0;
  __syncthreads();
  int pt = 0, ct = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int x = sh[w * 3], y = sh[w * 3 + 1], z = sh[w * 3 + 2];
    if (w < wave) p0 += x, s0 += y, c0 += z;
    pt += x;
    ct += z;
  }
  p0 -= parts, s0 -= slots, c0 -= cuts;
  if (blockIdx.x == 0 && tid == 0 && a.counts != nullptr) a.counts[0] = ct;
  __syncthreads();
  // pairs of parts (the two blocks of a token's 128 heads, most often) go to one XCD (blockIdx % 8), and
  // share its L2
  const int my = (int)(((blockIdx.x >> 4) * 8 + (blockIdx.x & 7)) * 2 + ((blockIdx.x >> 3) & 1));
  if (my >= pt) return false;
  if (my >= p0 && my < p0 + parts) {
    bool found = false;
    each([&](int b, int n, int tiles) {
      if (found) return;
      const int c = cut(tiles, quantum);
      if (my < p0 + n * c) {
        const int blk = (my - p0) / c, part = (my - p0) - blk * c;
        sh[16] = b;
        sh[17] = blk;
        sh[18] = part;
        sh[19] = c;
        sh[20] = c > 1 ? s0 + blk * c + part : -1;
        if (c > 1 && part == 0 && c0 + blk < a.max_cuts)
          reinterpret_cast<Desc*>(a.counts + 4)[c0 + blk] = {b, blk, s0 + blk * c, c};
        found = true;
        return;
      }
      p0 += n * c;
      if (c > 1) s0 += n * c, c0 += n;
    });
  }
  __syncthreads();
  work = {__builtin_amdgcn_readfirstlane(sh[16]), __builtin_amdgcn_readfirstlane(sh[17]),
          __builtin_amdgcn_readfirstlane(sh[18]), __builtin_amdgcn_readfirstlane(sh[19]),
          __builtin_amdgcn_readfirstlane(sh[20])};
  __syncthreads();
  // starts that are not rising could ask for more (nothing is promised for them)
  return work.slot < 0 || work.slot - work.part + work.parts <= a.max_slots;
}

// The query row of a lane as operands: e4m3 terms hi + lo 2^-4 under the scale code `code`, and the
// rotary part in bf16. Step ks holds latents 64 ks + 16 g .. + 15 and 64 ks + 32 + 16 g .. + 15.
struct Query {
  v8i hi[8], lo[8];
  v8bf rope[4];
  int code;
};
__device__ __forceinline__ void load_query(const uint16_t* src, bool row_ok, int g, Query& q) {
  auto raw = [&](int ks, int j) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row_ok) v = *reinterpret_cast<const uint4*>(src + 64 * ks + 32 * (j >> 1) + 16 * g + 8 * (j & 1));
    return v;
  };
  float amax = 0.f;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
      bf16x8_values(raw(ks, j), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(f[i]));
    }
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row_ok) v = *reinterpret_cast<const uint4*>(src + kLatentDim + 16 * ks + 8 * g);
    q.rope[ks] = __builtin_bit_cast(v8bf, v);
  }
  amax = max_nan(amax, __shfl_xor(amax, 32));
  // the least power of two that holds the row in e4m3 range (kept away from the ends of float32)
  uint32_t code = (__float_as_uint(max_nan(amax, 0x1p-80f) / 448.0f) + 0x7fffffu) >> 23;
  const bool finite = amax < __builtin_inff();
  if (!finite) code = 127;
  const float inv = finite ? __uint_as_float((254u - code) << 23) : __builtin_nanf("");  // a NaN row scores NaN
  q.code = (int)code;
  asm volatile("" ::: "memory");  // the row is read a second time (from L2) rather than held in 128 registers
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8], back[8], lo[8];
      bf16x8_values(raw(ks, j), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= inv;
      const uint2 hi = make_uint2(pack_e4m3(f), pack_e4m3(f + 4));
      e4m3x8_values(hi, back);
#pragma unroll
      for (int i = 0; i < 8; ++i) lo[i] = (f[i] - back[i]) * 16.f;
      q.hi[ks][2 * j] = (int)hi.x;
      q.hi[ks][2 * j + 1] = (int)hi.y;
      q.lo[ks][2 * j] = (int)pack_e4m3(lo);
      q.lo[ks][2 * j + 1] = (int)pack_e4m3(lo + 4);
    }
}

// kPairs pairs of waves, 32 query rows each. kAhead: a tile's scores and softmax run while the products of the
// tile before with its values do, which takes a third tile of LDS.
template <int kPairs, bool kAhead>
__global__ __launch_bounds__(kPairs * 128, 1) void latent_attn_kernel(LatentAttnArgs a) {
  constexpr int kThreads = kPairs * 128, kBM = kPairs * 32, kWaves = kPairs * 2;
  constexpr int kBuffers = kAhead ? 3 : 2;
  __shared__ __align__(1024) uint8_t lds_tiles[kBuffers * kTileBytes];
  Work work;
  if (!find_work<kThreads, kBM>(a, reinterpret_cast<int*>(lds_tiles), work)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int pair = wave >> 1, half = wave & 1;
  Seq seq = sequence(a, work.seq);
  seq = {__builtin_amdgcn_readfirstlane(seq.q0), __builtin_amdgcn_readfirstlane(seq.n),
         __builtin_amdgcn_readfirstlane(seq.len)};
  const int rows = (int)min((int64_t)seq.n * a.H - (int64_t)work.block * kBM, (int64_t)kBM);

  // ---- this lane's query row
  const int row = pair * 32 + r;
  const bool row_ok = row < rows;
  const int flat = work.block * kBM + row;
  const int tok = row_ok ? flat / a.H : 0, head = row_ok ? flat - tok * a.H : 0;
  const int64_t qtok = seq.q0 + tok;
  // keys the row sees: its sequence up to itself
  const int limit = row_ok ? min(max(seq.len - seq.n + tok + 1, 0), seq.len) : 0;
  // keys the block sees (its last row's), cut into parts of whole tiles
  const int last_tok = (work.block * kBM + rows - 1) / a.H;
  const int keys = min(max(seq.len - seq.n + last_tok + 1, 0), seq.len);
  const int tiles = (keys + kTile - 1) / kTile;
  const int t_begin = (int)((int64_t)tiles * work.part / work.parts);
  const int t_end = (int)((int64_t)tiles * (work.part + 1) / work.parts);
  // keys that every row of the block sees: tiles before need no mask
  const int all = rows == kBM ? min(max(seq.len - seq.n + work.block * kBM / a.H + 1, 0), seq.len) : 0;

  v16f acc[16];
#pragma unroll
  for (int d = 0; d < 16; ++d) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
    keep_acc(acc[d]);
  }
  float m = kNegInf, l = 0.f;

  if (t_begin < t_end) {
    // ---- the page table and the scale codes are read ahead: lane L for key L of a tile
    // (no branches: a column past the table reads its last entry, or where it has none a length, and counts as none)
    const int width = a.cache.table_width;
    const int32_t* table = width > 0 ? a.cache.table + (int64_t)work.seq * a.cache.table_stride : a.lens;
    const int page_size = a.cache.page_size;
    const int step_col = kTile / page_size, step_off = kTile - step_col * page_size;
    const int end_col = (keys - 1) / page_size, end_off = (keys - 1) - end_col * page_size;
    int col = (t_begin * kTile + lane) / page_size, off = (t_begin * kTile + lane) - col * page_size;
    // of a tile: the table's entry and the row in its page; keys past the end repeat the last (masked)
    auto look_up = [&](int& page, int& row_in_page) {
      const bool past = col > end_col || (col == end_col && off > end_off);
      const int at = past ? end_col : col;
      row_in_page = past ? end_off : off;
      const int entry = table[min(at, max(width - 1, 0))];
      page = at < width ? entry : -1;
      col += step_col;
      off += step_off;
      if (off >= page_size) off -= page_size, ++col;
    };
    auto bad = [&](int page) { return page < 0 || page >= a.cache.pages; };
    const uint32_t page_units = (uint32_t)(a.cache.page_stride / 128);
    // the row's place in 128-byte units; a page that does not exist reads page 0 ...
    auto unit_of = [&](int page, int o) {
      const bool none = bad(page);
      return (uint32_t)(none ? 0 : page) * page_units + (uint32_t)(none ? 0 : o) * (kLatentRow / 128);
    };
    auto code_of = [&](int page, int o) {  // ... under the code of NaN
      const bool none = bad(page);
      const int byte = a.cache.scales[(int64_t)(none ? 0 : page) * a.cache.scale_stride + (none ? 0 : o)];
      return none ? 255 : byte;
    };
    // ---- copies of a tile: 64 x 512 bytes of codes, then 64 x 128 bytes of rotary keys
    const uint32_t lds = lds_addr(lds_tiles);
    constexpr int kCodeCopies = 32 / kWaves, kCopies = 40 / kWaves;
    // Two rows of codes a copy, lanes 32 .. 63 the second; eight rows of rotary keys. The XORs' lane parts
    // are the same for every copy, its own part a constant.
    auto copy_piece = [&](uint32_t unit, uint32_t at, int j) {
      const int ln = fresh(lane);
      if (j < kCodeCopies) {
        const int kk = wave * (2 * kCodeCopies) + 2 * j + (ln >> 5);
        const uint64_t u = (uint32_t)__builtin_amdgcn_ds_bpermute(kk << 2, (int)unit);
        copy16_from(a.cache.rows + u * 128 + (((ln & 31) ^ ((ln >> 5) << 1) ^ swz(2 * j)) << 4), at + (wave * kCodeCopies + j) * 1024);
      } else {
        const int jr = j - kCodeCopies, kk = wave * (64 / kWaves) + 8 * jr + (ln >> 3);
        const uint64_t u = (uint32_t)__builtin_amdgcn_ds_bpermute(kk << 2, (int)unit);
        copy16_from(a.cache.rows + u * 128 + kLatentDim + (((ln & 7) ^ (ln >> 3) ^ (jr & 1)) << 4),
                    at + kTile * kLatentDim + (wave * (8 / kWaves) + jr) * 1024);
      }
    };

    int page, o, page_next, o_next, page_far, o_far;
    look_up(page, o);
    look_up(page_next, o_next);
    look_up(page_far, o_far);
    int code = code_of(page, o);  // of tile t
    {
      const uint32_t unit = unit_of(page, o);
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy_piece(unit, lds, j);
    }
    int code_next = code_of(page_next, o_next);  // of tile t + 1
    uint32_t unit_next = unit_of(page_next, o_next);
    Query q;
    load_query(a.q + qtok * a.q_tok + (int64_t)head * a.q_head, row_ok, g, q);

    const float c = a.scale * 1.44269504088896341f;
    const int p_code = g == 0 ? 127 : 123, one = 127;  // slots of hi at 1, of lo at 2^-4

    // ---- scores of this wave's 32 keys of a tile; `between(step)` is called at each of 8 steps
    auto scores = [&](uint32_t tile, int tile_code, auto between) {
      const int kc = __shfl(tile_code, half * 32 + r);
      const int kk = fresh(half * 32 + r);
      typedef __attribute__((address_space(3))) const v4i lds_v4i;
      const uint32_t kb = tile + kk * kLatentDim;
      const int sw = g ^ swz(kk);
      auto key = [&](int ks) {
        const v4i x = *reinterpret_cast<lds_v4i*>(kb + ((sw ^ (ks * 4)) << 4));
        const v4i y = *reinterpret_cast<lds_v4i*>(kb + ((sw ^ (ks * 4 + 2)) << 4));
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
      };
      const uint32_t rb = tile + kTile * kLatentDim + kk * 128;
      const int rsw = g ^ lds_swizzle(kk);
      auto rope = [&](int ks) {
        return __builtin_bit_cast(v8bf, *reinterpret_cast<lds_v4i*>(rb + ((rsw ^ (ks * 2)) << 4)));
      };
      v8i k[3];
      v8bf kr[4];
      k[0] = key(0);
      k[1] = key(1);
      v16f s;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        if (ks + 2 < 8) {
          k[(ks + 2) % 3] = key(ks + 2);
        } else {
          kr[2 * (ks - 6)] = rope(2 * (ks - 6));
          kr[2 * (ks - 6) + 1] = rope(2 * (ks - 6) + 1);
        }
        s = mfma_scaled(k[ks % 3], q.hi[ks], s, kc, q.code);
        s = mfma_scaled(k[ks % 3], q.lo[ks], s, kc, q.code - 4);
        asm volatile("" : "+v"(s));  // the products stay here
        between(ks);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kr[ks], q.rope[ks], s, 0, 0, 0);
      return s;
    };
    // ---- x = score in log2 + scale code of the key, its maximum, and the codes of keys 8 q + 4 g .. + 3
    struct Soft {
      v16f x;
      uint32_t codes[4];
      float ref;
    };
    // Returns the factor of a new running maximum (1: none).
    auto soft_begin = [&](const v16f& s, int tile_code, int t, Soft& w) {
      const int up = __builtin_amdgcn_mov_dpp(tile_code, 0xB1, 0xF, 0xF, true);          // the neighbour's: lanes 1 0 3 2
      const int two = (lane & 1) ? (up | tile_code << 8) : (tile_code | up << 8);        // both lanes: even, odd
      const int over = __builtin_amdgcn_mov_dpp(two, 0x4E, 0xF, 0xF, true);              // lanes 2 3 0 1
      const int four = (lane & 2) ? (over | two << 16) : (two | over << 16);             // the quad's four codes
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) w.codes[q4] = (uint32_t)__shfl(four, half * 32 + 8 * q4 + 4 * g);
#pragma unroll
      for (int i = 0; i < 16; ++i) w.x[i] = fmaf(s[i], c, (float)((w.codes[i >> 2] >> (8 * (i & 3))) & 0xffu));
      const int k0 = t * kTile + half * 32;
      if (k0 + 32 > all) {
        const int left = limit - k0 - 4 * g;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (8 * (i >> 2) + (i & 3) >= left) w.x[i] = kNegInf;
      }
      float top = w.x[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, w.x[i]);
      top = fmaxf(top, __shfl_xor(top, 32));
      float f = 1.f;
      if (__any(top > m + kSlack)) {
        const float next = fmaxf(m, top);
        f = m == next ? 1.f : __builtin_amdgcn_exp2f(m - next);  // (m = next = -inf: nothing yet)
        m = next;
        l *= f;
      }
      w.ref = m == kNegInf ? 0.f : m - kTop;
      return f;
    };
    // Weights of four keys (quad q4), into the operand.
    auto soft_quad = [&](const Soft& w, int q4, v8i& pw) {
      float p[4], rest[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = __builtin_amdgcn_exp2f(w.x[4 * q4 + i] - w.ref);
        // times 2^-e (a masked key's p is 0, whatever its code)
        l += __builtin_amdgcn_ldexpf(p[i], 127 - (int)((w.codes[q4] >> (8 * i)) & 0xffu));
      }
      const int h = (int)pack_e4m3(p);
      rest[0] = (p[0] - __builtin_amdgcn_cvt_f32_fp8(h, 0)) * 16.f;
      rest[1] = (p[1] - __builtin_amdgcn_cvt_f32_fp8(h, 1)) * 16.f;
      rest[2] = (p[2] - __builtin_amdgcn_cvt_f32_fp8(h, 2)) * 16.f;
      rest[3] = (p[3] - __builtin_amdgcn_cvt_f32_fp8(h, 3)) * 16.f;
      pw[q4] = h;
      pw[4 + q4] = (int)pack_e4m3(rest);
    };
    auto rescale = [&](float f) {
      if (__any(f != 1.f)) {
        asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");  // products in flight
#pragma unroll
        for (int d = 0; d < 16; ++d) {
          keep_acc(acc[d]);
          acc[d] *= f;
          keep_acc(acc[d]);
        }
      }
    };
    // ---- O^T += V^T P^T, 32 value columns at a time; `between(d)` is called at each of 16 steps
    auto values = [&](uint32_t tile, const v8i& pw, auto between) {
      typedef __attribute__((address_space(3))) v2i lds_v2i;
      const int ln = fresh(lane);
      const int vk = half * 32 + 8 * ((ln >> 3) & 1) + 4 * g + ((ln >> 1) & 3);  // the row this lane addresses (and vk + 16)
      const uint32_t vb = tile + vk * kLatentDim + 8 * (ln & 1);
      const int sw = ((ln >> 4) & 1) ^ swz(vk);
      v2i x[3], y[3];
      auto value = [&](int d) {
        const uint32_t at = vb + ((sw ^ (2 * d)) << 4);
        x[d % 3] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_v2i*>(at));
        y[d % 3] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_v2i*>(at + 16 * kLatentDim));
      };
      value(0);
      value(1);
#pragma unroll
      for (int d = 0; d < 16; ++d) {
        if (d + 2 < 16) value(d + 2);
        const v2i u = x[d % 3], w = y[d % 3];
        const v8i v = {u[0], u[1], w[0], w[1], u[0], u[1], w[0], w[1]};
        mfma_scaled_acc(v, pw, acc[d], one, p_code);
        between(d);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    v8i pw;
    uint32_t tile = lds, tile_before = lds;
    int place = 0;
    // Tile t: everything up to the weights; kFirst: there is no tile before it in this part.
    auto step = [&](int t, auto first) {
      constexpr bool kFirst = decltype(first)::value;
      // tile t and what was read ahead have landed; every wave is done with the tile whose place is next
      wait_copies();
      asm volatile("" : "+v"(page_far), "+v"(code_next));
      lds_barrier();
      const int next_place = place + 1 == kBuffers ? 0 : place + 1;
      const uint32_t next_tile = lds + next_place * kTileBytes;
      const uint32_t unit = unit_next;
      const int tile_code = code;
      code = code_next;
      // (after the last tile the copies bring one that is not used: there always is a key to look up)
      constexpr int kSteps = 4, kEach = (kCopies + kSteps - 1) / kSteps;
      const v16f s = scores(tile, tile_code, [&](int ks) {
        if (ks < kSteps) {
#pragma unroll
          for (int j = 0; j < kEach; ++j)
            if (ks * kEach + j < kCopies) copy_piece(unit, next_tile, ks * kEach + j);
        }
        if (ks == kSteps) {
          unit_next = unit_of(page_far, o_far);
          code_next = code_of(page_far, o_far);
          look_up(page_far, o_far);
        }
      });
      Soft w;
      const float f = soft_begin(s, tile_code, t, w);
      if constexpr (kAhead) {
        v8i next;
        if constexpr (kFirst) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) soft_quad(w, q4, next);
        } else {
          values(tile_before, pw, [&](int d) {
            if ((d & 3) == 3) soft_quad(w, d >> 2, next);
          });
          rescale(f);
        }
        pw = next;
      } else {
        rescale(f);
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) soft_quad(w, q4, pw);
        values(tile, pw, [](int) {});
      }
      tile_before = tile;
      tile = next_tile;
      place = next_place;
    };
    if constexpr (kAhead) {
      step(t_begin, std::true_type{});
      for (int t = t_begin + 1; t < t_end; ++t) step(t, std::false_type{});
      values(tile_before, pw, [](int) {});
    } else {
      for (int t = t_begin; t < t_end; ++t) step(t, std::false_type{});
    }
    wait_copies();
  }

  // the last products' results arrive (the compiler does not know what the assembly above was)
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int d = 0; d < 16; ++d) keep_acc(acc[d]);
  // ---- the two waves of a pair join: each sends the other half its columns
  l += __shfl_xor(l, 32);
  __syncthreads();
  float* sh = reinterpret_cast<float*>(lds_tiles);
  if (g == 0) sh[(wave * 32 + r) * 2] = m, sh[(wave * 32 + r) * 2 + 1] = l;
  __syncthreads();
  const float m0 = sh[(pair * 64 + r) * 2], l0 = sh[(pair * 64 + r) * 2 + 1];
  const float m1 = sh[(pair * 64 + 32 + r) * 2], l1 = sh[(pair * 64 + 32 + r) * 2 + 1];
  const float m_all = fmaxf(m0, m1);
  const float f0 = m0 == m_all ? 1.f : __builtin_amdgcn_exp2f(m0 - m_all);
  const float f1 = m1 == m_all ? 1.f : __builtin_amdgcn_exp2f(m1 - m_all);
  const float l_all = fmaf(f1, l1, f0 * l0);
  const float inv = l_all == 0.f ? 0.f : 1.0f / l_all;  // a row that sees no key is zero
  const float f_own = half ? f1 : f0, f_other = half ? f0 : f1;
  const bool whole = work.slot < 0;
  const int64_t state_row = (int64_t)work.slot * kBM + row;
  uint16_t* dst = a.out + qtok * a.o_tok + (int64_t)head * a.o_head + 4 * g;
  float* state = a.states + state_row * kLatentDim + 4 * g;
  if (!whole && half == 0 && g == 0 && row_ok) {
    a.stats[state_row * 2] = m_all;
    a.stats[state_row * 2 + 1] = l_all;
  }
  v4f* box = reinterpret_cast<v4f*>(lds_tiles);  // 16 KB a wave
  auto send = [&](const v16f& x, int d) {
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4)
      box[(wave * 16 + d * 4 + q4) * 64 + lane] = v4f{x[4 * q4], x[4 * q4 + 1], x[4 * q4 + 2], x[4 * q4 + 3]};
  };
  auto join = [&](const v16f& x, int d, int column) {
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      const v4f y = box[((wave ^ 1) * 16 + d * 4 + q4) * 64 + lane];
      v4f o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(f_other, y[i], f_own * x[4 * q4 + i]);
      if (!row_ok) continue;
      const int at = column + 8 * q4;
      if (whole)
        *reinterpret_cast<uint2*>(dst + at) =
            make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
      else
        *reinterpret_cast<v4f*>(state + at) = o;
    }
  };
#pragma unroll
  for (int step = 0; step < 2; ++step) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (half == 0) send(acc[8 + 4 * step + d], d);
      else send(acc[4 * step + d], d);
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (half == 0) join(acc[4 * step + d], d, 32 * (4 * step + d));
      else join(acc[8 + 4 * step + d], d, 32 * (8 + 4 * step + d));
    }
  }
}

// Joins the parts of a cut block, in order: one wave a row.
template <int kBM>
__global__ __launch_bounds__(256) void latent_join_kernel(LatentAttnArgs a) {
  if ((int)blockIdx.x >= a.counts[0]) return;
  const Desc desc = reinterpret_cast<const Desc*>(a.counts + 4)[blockIdx.x];
  const int lane = threadIdx.x & 63;
  const int row = blockIdx.y * 4 + (threadIdx.x >> 6);
  if (desc.slot + desc.parts > a.max_slots) return;
  const Seq seq = sequence(a, desc.seq);
  const int flat = desc.block * kBM + row;
  if (flat >= seq.n * a.H) return;
  const int tok = flat / a.H, head = flat - tok * a.H;
  float m = kNegInf;
  for (int p = 0; p < desc.parts; ++p) m = fmaxf(m, a.stats[((int64_t)(desc.slot + p) * kBM + row) * 2]);
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
#pragma unroll 4
  for (int p = 0; p < desc.parts; ++p) {
    const int64_t at = (int64_t)(desc.slot + p) * kBM + row;
    const float mp = a.stats[at * 2];
    const float f = mp == m ? 1.f : __builtin_amdgcn_exp2f(mp - m);
    l = fmaf(f, a.stats[at * 2 + 1], l);
    const v4f* src = reinterpret_cast<const v4f*>(a.states + at * kLatentDim + lane * 8);
    const v4f x = src[0], y = src[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(f, x[i], o[i]), o[4 + i] = fmaf(f, y[i], o[4 + i]);
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  uint16_t* dst = a.out + (seq.q0 + (int64_t)tok) * a.o_tok + (int64_t)head * a.o_head + lane * 8;
  *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                                              pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
}

constexpr int kCUs = 256;
constexpr int kMinTiles = 2;  // fewer tiles a part cost more in states than they save

// Pairs of waves a workgroup: one where a sequence has 32 query rows or fewer on average (then two
// workgroups share a CU), otherwise two.
int pairs_for(int64_t T, int64_t B, int64_t H) { return T * H <= 32 * B ? 1 : 2; }

template <int kPairs>
hipError_t launch(const LatentAttnArgs& args, const LatentAttnPlan& plan, hipStream_t stream) {
  const int64_t grid = (plan.parts + 15) / 16 * 16;
  hipLaunchKernelGGL((latent_attn_kernel<kPairs, (kPairs > 1)>), dim3((unsigned)grid), dim3(kPairs * 128), 0, stream, args);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.slots == 0) return e;
  hipLaunchKernelGGL((latent_join_kernel<kPairs * 32>), dim3((unsigned)plan.cuts, kPairs * 8), dim3(256), 0, stream, args);
  return hipGetLastError();
}

}  // namespace

LatentAttnPlan plan_latent_attn(int64_t T, int64_t B, int64_t H, int64_t max_keys) {
  LatentAttnPlan p;
  p.pairs = pairs_for(T, B, H);
  const int64_t bm = 32 * p.pairs;
  // Blocks: a sequence's last may be partly filled.
  p.blocks = T * H / bm + (T < B ? T : B);
  const int64_t max_tiles = (max_keys + kTile - 1) / kTile;
  p.max_tiles = (int)max_tiles;
  p.target_parts = kCUs * 2 / p.pairs;
  p.min_tiles = kMinTiles;
  // Blocks are cut only into as many parts as run at once in all.
  const int64_t per_block = (max_tiles + kMinTiles - 1) / kMinTiles;
  if (per_block <= 1) {
    p.slots = p.cuts = 0;
  } else {
    p.slots = p.target_parts;
    if (p.blocks * per_block < p.slots) p.slots = p.blocks * per_block;
    p.cuts = p.slots / 2;
  }
  p.parts = p.blocks;
  if (p.slots > 0 && p.parts < p.target_parts) p.parts = p.target_parts;
  p.counts_bytes = p.slots ? ((16 + p.cuts * sizeof(Desc) + 255) / 256) * 256 : 0;
  p.stats_bytes = ((p.slots * bm * 2 * sizeof(float) + 255) / 256) * 256;
  p.states_bytes = p.slots * bm * kLatentDim * sizeof(float);
  return p;
}

hipError_t launch_latent_attn(const LatentAttnArgs& args, const LatentAttnPlan& plan, hipStream_t stream) {
  return plan.pairs == 1 ? launch<1>(args, plan, stream) : launch<2>(args, plan, stream);
}

}  // namespace bfp8
