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
//     x_j = scale log2(e) s_j + e_j, split into hi + lo e4m3 in the same way (at least 8
//     significant bits, as bf16 would have). A row's weights of 32 keys share a power of two, the
//     least that holds their largest, which the instruction applies: weights far below the largest
//     of a long sequence keep their bits. The accumulator is kept relative to 2^m, m a whole number
//     that only moves when a score passes it by 2^kSlack, so it is hardly ever rescaled. The softmax
//     denominator sums 2^(x_j) 2^(-e_j) in float32.
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
constexpr float kSlack = 32.f;             // weights may pass the accumulator's reference by a factor of 2^kSlack
constexpr float kTop = 8.f;                // the largest of 32 weights is held at 2^(kTop - 1) .. 2^kTop <= 448
constexpr float kFar = 100.f;              // weights 2^-kFar below the reference are held relative to that
constexpr float kNegInf = -__builtin_inff();

struct Desc {  // a block that was cut: rows of block `block`, partial states slot .. slot + parts - 1
  int seq, block, slot, parts;
};

// XOR of the 16-byte columns of a key's 512-byte row in LDS. Conflict-free both for the score
// reads (16 lanes: one column of 16 keys that differ in bits 0 .. 3) and for the transposing value
// reads (32 lanes: two neighbouring columns of 8 keys that differ in bits 0, 1 and 3).
__device__ __forceinline__ int swz(int key) { return ((key & 3) << 1) | (key & 8) | ((key >> 2) & 1); }

// Scale codes: ea's low byte and byte kByte of eb.
template <int kByte>
__device__ __forceinline__ v16f mfma_scaled(const v8i& a, const v8i& b, const v16f& c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, ea, kByte, eb);
}

// The same product added to an accumulator in the accumulation registers. Written in assembly so that it
// stays there: the compiler otherwise moves accumulators between the two register files in bulk. The
// wait in front covers operands that vector instructions have just written.
// Scale codes: byte 0 of `codes` for a, byte 1 for b.
__device__ __forceinline__ void mfma_scaled_acc(const v8i& a, const v8i& b, v16f& c, int codes) {
  asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %3 op_sel:[0,1,0] op_sel_hi:[0,0,0]"
      : "+a"(c)
      : "v"(a), "v"(b), "v"(codes));
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

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // 1, 2, 4, 8 lanes up within 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 to the next 16, of the odd rows
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to the upper half
  return v;
}

// What a workgroup computes: part `part` of `parts` of a block, and where its state goes (-1: nowhere).
struct Work {
  Seq seq;
  int index, block, part, parts, slot;
};

// Every wave cuts the work in the same way and picks its workgroup's part. False: there is none.
template <int kBM>
__device__ __forceinline__ bool find_work(const LatentAttnArgs& a, Work& work) {
  constexpr int kHeld = 4;   // sequences of a lane that are read once
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
    if (k < count) held[k] = sequence(a, b0 + k);
  }
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (k < count) f(b0 + k, held[k], blocks_of(held[k]), tiles_of(held[k]));
    for (int k = kHeld; k < count; ++k) {
      const Seq q = sequence(a, b0 + k);
      f(b0 + k, q, blocks_of(q), tiles_of(q));
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
  if (a.max_slots > 0) {
    int64_t blocks = 0;
    each([&](int, const Seq&, int n, int) { blocks += n; });
    if (total((int)min(blocks, (int64_t)kMany)) < a.target_parts) {
      int lo = a.min_tiles, hi = max(quantum, lo);
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
        w = {q, b, blk, part, c, c > 1 ? s0 + blk * c + part : -1};
        if (c > 1 && part == 0 && c0 + blk < a.max_cuts && threadIdx.x < 64)
          reinterpret_cast<Desc*>(a.counts + 4)[c0 + blk] = {b, blk, s0 + blk * c, c};
        found = true;
      }
      p0 += n * c;
      if (c > 1) s0 += n * c, c0 += n;
    });
  }
  const int src = __builtin_ctzll(who);
  auto from = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
  work = {{from(w.seq.q0), from(w.seq.n), from(w.seq.len)}, from(w.index), from(w.block), from(w.part), from(w.parts),
          from(w.slot)};
  // starts that are not rising could ask for more (nothing is promised for them)
  return work.slot < 0 || work.slot - work.part + work.parts <= a.max_slots;
}

// The query row of a lane as operands: e4m3 terms hi + lo 2^-4 under the scale code `code`, and the
// rotary part in bf16. Step ks holds latents 64 ks + 16 g .. + 15 and 64 ks + 32 + 16 g .. + 15.
struct Query {
  v8i hi[8], lo[8];
  v8bf rope[4];
  int code;  // of hi in byte 0, of lo in byte 1
};
// What a wave reads of its 32 rows: the latents of 4 of the 8 steps (the other wave of its pair reads
// the rest).
struct RawQuery {
  uint4 lat[4][4];
};
__device__ __forceinline__ void read_query(const uint16_t* src, bool row_ok, int g, int half, RawQuery& x) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x.lat[ks][j] = make_uint4(0, 0, 0, 0);
      if (row_ok)
        x.lat[ks][j] = *reinterpret_cast<const uint4*>(src + 256 * half + 64 * ks + 32 * (j >> 1) + 16 * g + 8 * (j & 1));
    }
}
// `box`: 16 KB of LDS a wave, and one int a row and wave behind them.
template <int kWaves>
__device__ __forceinline__ void split_query(const RawQuery& x, int lane, int wave, uint8_t* box, Query& q) {
  typedef unsigned short v2us __attribute__((ext_vector_type(2)));
  typedef short v2s __attribute__((ext_vector_type(2)));
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  typedef float v2f __attribute__((ext_vector_type(2)));
  const int r = lane & 31;
  // the largest magnitude: without its sign a bf16 pattern grows with its value, NaN last
  v2us top = {0, 0};
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {x.lat[ks][j].x, x.lat[ks][j].y, x.lat[ks][j].z, x.lat[ks][j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(v2us, w[i] & 0x7fff7fffu));
    }
  int bits = max((int)top[0], (int)top[1]);
  const auto swapped = __builtin_amdgcn_permlane32_swap((unsigned)bits, (unsigned)bits, false, false);
  bits = max((int)swapped[0], (int)swapped[1]);
  int* tops = reinterpret_cast<int*>(box + kWaves * 16384);
  if (lane < 32) tops[wave * 32 + r] = bits;
  __syncthreads();
  bits = max(bits, tops[(wave ^ 1) * 32 + r]);
  // the least power of two that holds the row in e4m3 range (kept away from the ends of float32)
  const float amax = __uint_as_float((uint32_t)bits << 16);
  const bool finite = bits < 0x7f80;
  const uint32_t code = finite ? (__float_as_uint(fmaxf(amax, 0x1p-80f) / 448.0f) + 0x7fffffu) >> 23 : 127;
  const float scale = __uint_as_float(code << 23);
  q.code = finite ? (int)(code | (code - 4) << 8) : 0xffff;  // a NaN row scores NaN
  v4i* out = reinterpret_cast<v4i*>(box) + wave * 1024 + lane;
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    v8i hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[4] = {x.lat[ks][j].x, x.lat[ks][j].y, x.lat[ks][j].z, x.lat[ks][j].w};
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        v2s h = {0, 0}, l = {0, 0};
        // (values over the scale, to nearest even; then what is left of them, exactly, over a sixteenth)
        h = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(h, __builtin_bit_cast(v2bf, w[i]), scale, false);
        h = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(h, __builtin_bit_cast(v2bf, w[i + 1]), scale, true);
        const unsigned hb = __builtin_bit_cast(unsigned, h);
        const v2f b0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hb, scale, false);
        const v2f b1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hb, scale, true);
        const float tiny = scale * 0.0625f;
        l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, __uint_as_float(w[i] << 16) - b0[0],
                                                     __uint_as_float(w[i] & 0xffff0000u) - b0[1], tiny, false);
        l = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(l, __uint_as_float(w[i + 1] << 16) - b1[0],
                                                     __uint_as_float(w[i + 1] & 0xffff0000u) - b1[1], tiny, true);
        hi[2 * j + (i >> 1)] = (int)hb;
        lo[2 * j + (i >> 1)] = __builtin_bit_cast(int, l);
      }
    }
    out[(4 * ks) * 64] = __builtin_shufflevector(hi, hi, 0, 1, 2, 3);
    out[(4 * ks + 1) * 64] = __builtin_shufflevector(hi, hi, 4, 5, 6, 7);
    out[(4 * ks + 2) * 64] = __builtin_shufflevector(lo, lo, 0, 1, 2, 3);
    out[(4 * ks + 3) * 64] = __builtin_shufflevector(lo, lo, 4, 5, 6, 7);
  }
  __syncthreads();
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const v4i* in = reinterpret_cast<const v4i*>(box) + ((wave & ~1) + (ks >> 2)) * 1024 + (ks & 3) * 256 + lane;
    q.hi[ks] = __builtin_shufflevector(in[0], in[64], 0, 1, 2, 3, 4, 5, 6, 7);
    q.lo[ks] = __builtin_shufflevector(in[128], in[192], 0, 1, 2, 3, 4, 5, 6, 7);
  }
}

// kPairs pairs of waves, 32 query rows each. kAhead: a tile's scores and softmax run while the products of the
// tile before with its values do, which takes a third tile of LDS.
template <int kPairs, bool kAhead>
__global__ __launch_bounds__(kPairs * 128, 1) void latent_attn_kernel(LatentAttnArgs a) {
  constexpr int kBM = kPairs * 32, kWaves = kPairs * 2;
  constexpr int kBuffers = kAhead ? 3 : 2;
  // with room for it, the rotary part of the queries stays in LDS (4 KB a pair)
  __shared__ __align__(1024) uint8_t lds_tiles[kBuffers * kTileBytes + (kAhead ? kPairs * 4096 : 0)];
  Work work;
  if (!find_work<kBM>(a, work)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int pair = wave >> 1, half = wave & 1;
  const Seq seq = work.seq;
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
    RawQuery raw;
    const uint16_t* q_row = a.q + qtok * a.q_tok + (int64_t)head * a.q_head;
    read_query(q_row, row_ok, g, half, raw);
    // ---- the page table and the scale codes are read ahead: lane L for key L of a tile
    // (no branches: a column past the table reads its last entry, or where it has none a length, and counts as none)
    const int width = a.cache.table_width;
    const int32_t* table = width > 0 ? a.cache.table + (int64_t)work.index * a.cache.table_stride : a.lens;
    const int page_size = a.cache.page_size;
    auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    const int step_col = uniform(kTile / page_size), step_off = kTile - step_col * page_size;
    const int end_col = uniform((keys - 1) / page_size), end_off = (keys - 1) - end_col * page_size;
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
    struct Lanes {  // formed once a tile
      int code_from, rope_from, code_at, rope_at;
    };
    auto lanes = [&] {
      const int ln = fresh(lane);
      Lanes x;
      x.code_from = fresh((wave * (2 * kCodeCopies) + (ln >> 5)) << 2);
      x.rope_from = fresh((wave * (64 / kWaves) + (ln >> 3)) << 2);
      x.code_at = ((ln & 31) ^ ((ln >> 5) << 1)) << 4;
      x.rope_at = ((ln & 7) ^ (ln >> 3)) << 4;
      return x;
    };
    auto place_of = [&](const Lanes& x, uint32_t unit, int j) {  // the row's place, from the lane that looked it up
      return (uint32_t)__builtin_amdgcn_ds_bpermute(
          j < kCodeCopies ? x.code_from + 8 * j : x.rope_from + 32 * (j - kCodeCopies), (int)unit);
    };
    auto copy_piece = [&](const Lanes& x, uint32_t u, uint32_t at, int j) {
      const int jr = j - kCodeCopies;
      if (j < kCodeCopies)
        copy16_from(a.cache.rows + (uint64_t)u * 128 + (x.code_at ^ (swz(2 * j) << 4)), at + (wave * kCodeCopies + j) * 1024);
      else
        copy16_from(a.cache.rows + (uint64_t)u * 128 + kLatentDim + (x.rope_at ^ ((jr & 1) << 4)),
                    at + kTile * kLatentDim + (wave * (8 / kWaves) + jr) * 1024);
    };

    int page, o, page_next, o_next, page_far, o_far;
    look_up(page, o);
    look_up(page_next, o_next);
    look_up(page_far, o_far);
    int code = code_of(page, o);  // of tile t
    {
      const uint32_t unit = unit_of(page, o);
      const Lanes x = lanes();
#pragma unroll
      for (int j = 0; j < kCopies; ++j) copy_piece(x, place_of(x, unit, j), lds, j);
    }
    int code_next = code_of(page_next, o_next);  // of tile t + 1
    uint32_t unit_next = unit_of(page_next, o_next);
    Query q;
    split_query<kWaves>(raw, lane, wave, lds_tiles + kTileBytes, q);
    v4i* rope_box = reinterpret_cast<v4i*>(lds_tiles + kBuffers * kTileBytes) + pair * 256 + lane;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row_ok) v = *reinterpret_cast<const uint4*>(q_row + kLatentDim + 16 * ks + 8 * g);
      if constexpr (kAhead) rope_box[ks * 64] = __builtin_bit_cast(v4i, v);  // (both waves of a pair write the same)
      else q.rope[ks] = __builtin_bit_cast(v8bf, v);
    }
    const float c = __uint_as_float((uint32_t)uniform((int)__float_as_uint(a.scale * 1.44269504088896341f)));
    const int p_base = 127 | (g == 0 ? 127 : 123) << 8;  // values at 1; slots of hi at 1, of lo at 2^-4

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
      const uint32_t qr = lds + kBuffers * kTileBytes + pair * 4096 + fresh(lane) * 16;
      auto q_rope = [&](int ks) {
        if constexpr (kAhead) return __builtin_bit_cast(v8bf, *reinterpret_cast<lds_v4i*>(qr + ks * 1024));
        else return q.rope[ks];
      };
      constexpr int kRing = kAhead ? 3 : 2;
      v8i k[kRing];
      v8bf kr[2], qk[2];
#pragma unroll
      for (int ks = 0; ks + 1 < kRing; ++ks) k[ks] = key(ks);
      v16f s;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        if (ks + kRing - 1 < 8) k[(ks + kRing - 1) % kRing] = key(ks + kRing - 1);
        if (ks >= 6) kr[ks - 6] = rope(ks - 6), qk[ks - 6] = q_rope(ks - 6);
        s = mfma_scaled<0>(k[ks % kRing], q.hi[ks], s, kc, q.code);
        s = mfma_scaled<1>(k[ks % kRing], q.lo[ks], s, kc, q.code);
        asm volatile("" : "+v"(s));  // the products stay here
        between(ks);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const v8bf x = kr[ks & 1], y = qk[ks & 1];
        if (ks < 2) kr[ks] = rope(ks + 2), qk[ks] = q_rope(ks + 2);
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, s, 0, 0, 0);
      }
      return s;
    };
    // ---- softmax of this lane's 16 scores, in pieces that fit between matrix products
    struct Soft {
      v16f x;             // score in log2 + scale code of the key
      uint32_t codes[4];  // of keys 8 q + 4 g .. + 3
      float ref, sum;
      int up;  // weights are 2^(x - ref); the accumulator's are 2^up times those
    };
    auto soft_codes = [&](int tile_code, Soft& w) {
      const int up = __builtin_amdgcn_mov_dpp(tile_code, 0xB1, 0xF, 0xF, true);    // the neighbour's: lanes 1 0 3 2
      const int two = (lane & 1) ? (up | tile_code << 8) : (tile_code | up << 8);  // both lanes: even, odd
      const int over = __builtin_amdgcn_mov_dpp(two, 0x4E, 0xF, 0xF, true);        // lanes 2 3 0 1
      const int four = (lane & 2) ? (over | two << 16) : (two | over << 16);       // the quad's four codes
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
        w.codes[q4] = (uint32_t)__builtin_amdgcn_ds_bpermute(((half * 32 + 4 * g) << 2) + 32 * q4, four);
    };
    auto soft_x = [&](const v16f& s, Soft& w) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w.x[i] = fmaf(s[i], c, (float)((w.codes[i >> 2] >> (8 * (i & 3))) & 0xffu));
    };
    auto soft_mask = [&](int t, Soft& w) {
      const int k0 = t * kTile + half * 32;
      if (k0 + 32 > all) {
        const int left = limit - k0 - 4 * g;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (8 * (i >> 2) + (i & 3) >= left) w.x[i] = kNegInf;
      }
    };
    // Returns the factor of a new reference (1: none).
    auto soft_top = [&](Soft& w) {
      float top = w.x[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, w.x[i]);
      const unsigned bits = __float_as_uint(top);
      const auto both = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
      top = ceilf(fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])));
      const bool higher = top > m + kSlack;  // also at the first key that the row sees (m = -inf)
      const float f = higher && m > kNegInf ? __builtin_amdgcn_exp2f(m - top) : 1.f;
      m = higher ? top : m;
      l *= f;
      const float base = m == kNegInf ? 0.f : m;
      w.ref = fmaxf(top, base - kFar) - kTop;
      w.up = (int)(w.ref - base);
      w.sum = 0.f;
      return f;
    };
    // Weights of keys 2 k and 2 k + 1, into the operand.
    auto soft_pair = [&](Soft& w, int k, v8i& pw) {
      typedef float v2f __attribute__((ext_vector_type(2)));
      const int q4 = k >> 1;
      const float p0 = __builtin_amdgcn_exp2f(w.x[2 * k] - w.ref), p1 = __builtin_amdgcn_exp2f(w.x[2 * k + 1] - w.ref);
      // times 2^-e (a masked key's p is 0, whatever its code)
      w.sum += __builtin_amdgcn_ldexpf(p0, 127 - (int)((w.codes[q4] >> (16 * (k & 1))) & 0xffu));
      w.sum += __builtin_amdgcn_ldexpf(p1, 127 - (int)((w.codes[q4] >> (16 * (k & 1) + 8)) & 0xffu));
      if (k & 1) {
        pw[q4] = __builtin_amdgcn_cvt_pk_fp8_f32(p0, p1, pw[q4], true);
        const v2f back = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((unsigned)pw[q4], 16.f, true);  // 16 times
        pw[4 + q4] = __builtin_amdgcn_cvt_pk_fp8_f32(fmaf(p0, 16.f, -back[0]), fmaf(p1, 16.f, -back[1]), pw[4 + q4], true);
      } else {
        pw[q4] = __builtin_amdgcn_cvt_pk_fp8_f32(p0, p1, 0, false);
        const v2f back = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((unsigned)pw[q4], 16.f, false);
        pw[4 + q4] = __builtin_amdgcn_cvt_pk_fp8_f32(fmaf(p0, 16.f, -back[0]), fmaf(p1, 16.f, -back[1]), 0, false);
      }
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
    // ---- O^T += V^T P^T, 32 value columns at a time: accumulator d is columns 32 (d ^ 8 half) .. + 31, so
    // that the first 8 are those that the wave joins at the end; `between(d)` is called at each of 16 steps
    auto values = [&](uint32_t tile, const v8i& pw, int p_code, auto between) {
      typedef __attribute__((address_space(3))) v2i lds_v2i;
      const int ln = fresh(lane);
      const int vk = half * 32 + 8 * ((ln >> 3) & 1) + 4 * g + ((ln >> 1) & 3);  // the row this lane addresses (and vk + 16)
      const uint32_t vb = tile + vk * kLatentDim + 8 * (ln & 1);
      const int sw = ((ln >> 4) & 1) ^ swz(vk) ^ (16 * half);
      v2i x[2], y[2];
      auto value = [&](int d) {
        const uint32_t at = vb + ((sw ^ (2 * d)) << 4);
        x[d % 2] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_v2i*>(at));
        y[d % 2] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_v2i*>(at + 16 * kLatentDim));
      };
      value(0);
#pragma unroll
      for (int d = 0; d < 16; ++d) {
        if (d + 1 < 16) value(d + 1);
        const v2i u = x[d % 2], w = y[d % 2];
        const v8i v = {u[0], u[1], w[0], w[1], u[0], u[1], w[0], w[1]};
        mfma_scaled_acc(v, pw, acc[d], p_code);
        between(d);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    v8i pw;
    int p_code = 127;
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
      constexpr int kSteps = 4, kEach = kCopies / kSteps + (kCopies % kSteps != 0), kFirstPlaces = kEach;
      uint32_t places[kCopies];
      const Lanes at = lanes();
#pragma unroll
      for (int j = 0; j < kFirstPlaces && j < kCopies; ++j) places[j] = place_of(at, unit, j);
      Soft w;
      soft_codes(tile_code, w);
      const v16f s = scores(tile, tile_code, [&](int ks) {
        if (ks < kSteps) {
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            if (ks * kEach + j < kCopies) copy_piece(at, places[ks * kEach + j], next_tile, ks * kEach + j);
            const int far = ks * kEach + j + kFirstPlaces;
            if (far < kCopies) places[far] = place_of(at, unit, far);
          }
        }
        if (ks == kSteps) {
          unit_next = unit_of(page_far, o_far);
          code_next = code_of(page_far, o_far);
          look_up(page_far, o_far);
        }
      });
      if constexpr (kAhead && !kFirst) {
        v8i next;
        float f;
        values(tile_before, pw, p_code, [&](int d) {
          if (d == 0) soft_x(s, w);
          if (d == 1) soft_mask(t, w);
          if (d == 2) f = soft_top(w);
          if (d >= 3 && d < 11) soft_pair(w, d - 3, next);
        });
        rescale(f);
        pw = next;
      } else {
        soft_x(s, w);
        soft_mask(t, w);
        const float f = soft_top(w);
        if constexpr (!kAhead) rescale(f);  // (the first tile's factor is 1)
#pragma unroll
        for (int k = 0; k < 8; ++k) soft_pair(w, k, pw);
      }
      p_code = p_base + (w.up << 8);
      if constexpr (!kAhead) values(tile, pw, p_code, [](int) {});
      l += __builtin_amdgcn_ldexpf(w.sum, w.up);
      tile_before = tile;
      tile = next_tile;
      place = next_place;
    };
    if constexpr (kAhead) {
      step(t_begin, std::true_type{});
      for (int t = t_begin + 1; t < t_end; ++t) step(t, std::false_type{});
      values(tile_before, pw, p_code, [](int) {});
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
  const bool whole = work.slot < 0;
  const float inv = !whole ? 1.f : l_all == 0.f ? 0.f : 1.0f / l_all;  // a row that sees no key is zero
  const float f_own = (half ? f1 : f0), f_other = (half ? f0 : f1);
  const int64_t state_row = (int64_t)work.slot * kBM + row;
  if (!whole && half == 0 && g == 0 && row_ok) {
    a.stats[state_row * 2] = m_all;
    a.stats[state_row * 2 + 1] = l_all;
  }
  uint16_t* dst = a.out + qtok * a.o_tok + (int64_t)head * a.o_head + 256 * half;
  float* state = a.states + state_row * kLatentDim + 256 * half;
  v4f* box = reinterpret_cast<v4f*>(lds_tiles);  // 16 KB a wave
#pragma unroll
  for (int step = 0; step < 2; ++step) {
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const v16f x = acc[8 + 4 * step + d];
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
        box[(wave * 16 + d * 4 + q4) * 64 + lane] = v4f{x[4 * q4], x[4 * q4 + 1], x[4 * q4 + 2], x[4 * q4 + 3]};
    }
    __syncthreads();
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const v16f x = acc[4 * step + d];
      v4f o[4];  // columns 8 q + 4 g .. + 3 of 32
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        const v4f y = box[((wave ^ 1) * 16 + d * 4 + q4) * 64 + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[q4][i] = fmaf(f_other, y[i], f_own * x[4 * q4 + i]) * inv;
      }
      const int column = 32 * (4 * step + d);
      if (whole) {
        // lanes g = 0 and 1 of a row swap quads, so that each stores 16 neighbouring columns
        uint32_t u[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const auto v = __builtin_amdgcn_permlane32_swap(pack_bf16(o[h][2 * i], o[h][2 * i + 1]),
                                                            pack_bf16(o[2 + h][2 * i], o[2 + h][2 * i + 1]), false, false);
            u[h][i] = v[0];
            u[h][2 + i] = v[1];
          }
        if (row_ok) {
          uint4* p = reinterpret_cast<uint4*>(dst + column + 16 * g);
          p[0] = make_uint4(u[0][0], u[0][1], u[0][2], u[0][3]);
          p[1] = make_uint4(u[1][0], u[1][1], u[1][2], u[1][3]);
        }
      } else if (row_ok) {
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) *reinterpret_cast<v4f*>(state + column + 8 * q4 + 4 * g) = o[q4];
      }
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
