// Latent attention over the paged FP8 latent cache, in the absorbed form: every head of a query
// token reads the same cached row, as key (512 latents and the rotary key) and as value (latents).
//
//   o[t, h] = sum_j softmax_j(scale * q[t, h] . [c_j, r_j]) c_j,   c_j = 2^(e_j) * codes_j
//
// over the keys j that token t sees (its own sequence up to itself).
//
// Both products run on the FP8 matrix cores, on the cached codes as they are:
//   * scores: a bf16 query has 8 significant bits, so it is the sum of two e4m3 values
//     (hi: its top 4 bits; lo: the rest, scaled 2^4), both under one power-of-two scale a row:
//     exactly, down to 2^-13 of the row's largest element; below, to 2^-21 of that.
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
// which are at once its operand of the second product. Values are read from the key tile with
// transposing LDS reads.
//
// A workgroup holds 32 query rows a pair of waves and walks tiles of 64 keys. Of each tile a wave
// scores 32 keys; the two waves of a pair then exchange their weights through LDS, and each
// multiplies all 64 with 256 of the 512 value columns. So the accumulator takes 128 accumulation
// registers, the queries' two terms 128 others, and both products read a key byte from LDS for 32
// rows. There is one wave a SIMD, which issues an instruction every 4 clocks at best, so the kernel
// is bound by its instruction count as much as by the matrix cores: tile t's softmax runs between
// the value products of tile t - 1 (whose weights crossed at t's only barrier), copies between its
// score products, and the LDS layout (below) leaves all but a few addresses to constant offsets.
//
// Measured: 128 sequences of 2500 to 4096 keys x 128 heads 128 us (matrix cores busy 39 % of the clocks), 64 of 500
// to 8000 x 16 heads 54 us (5.4 TB/s in its middle), one of 1111 x 128 heads 18.6 us.
//
// Work is cut on the device, where the lengths are: a block is the query rows (tokens x heads)
// of one sequence that a workgroup holds, and where there are fewer blocks than workgroups fit
// the card, they are cut along their keys into parts whose float32 states (accumulator, maximum,
// sum) a second launch joins in order.
#include "device_latent.h"
#include "latent.h"
#include "latent_work.h"
#include "launch.h"

namespace bfp8 {

namespace {

constexpr int kTile = 64;                  // keys of a tile
// A tile in LDS: groups of 8 rows, each in 5 blocks of 128 bytes of every row (4 of codes, 1 of the rotary key) and
// 64 bytes of padding; of each 64 bytes the 16-byte columns are XORed with bits 2 and 1 of the row. No bank conflicts
// for the score reads (16 lanes: one column of 16 rows) and the transposing value reads (32 lanes: two columns of 8
// rows that differ in bits 0, 1 and 3). A copy brings one block, whole lines of 8 rows, so that a lane keeps to one
// row of a group, and a column of a later step lies a constant further on.
constexpr int kBlockBytes = 8 * 128, kGroupBytes = 5 * kBlockBytes + 64;
constexpr int kTileBytes = 8 * kGroupBytes;
constexpr int kBuffers = 3;                // tile t - 1 (values), t, and t + 1 on its way
constexpr int kWeightBytes = 2 * 2048;     // a wave's weights of 32 keys (two terms), for two tiles in turn
constexpr int kRefBytes = 2 * 128;         // their exponents
constexpr int kKeyBytes = 2 * 256;         // a wave's scale codes of a tile as floats, and 2^-e
constexpr float kSlack = 32.f;             // weights may pass the accumulator's reference by a factor of 2^kSlack
constexpr float kTop = 8.f;                // the largest of 32 weights is held at 2^(kTop - 1) .. 2^kTop <= 448
constexpr float kNone = -__FLT_MAX__;      // exponent of no weight at all: no finite score is below it
constexpr float kNegInf = -__builtin_inff();

// The row that a key without a page stands on: finite codes, so that rows that do not see it (weight zero) stay finite.
__device__ const uint4 kZeroRow[kLatentRow / 16] = {};

// Scale codes: ea's low byte and byte kByte of eb.
template <int kByte>
__device__ __forceinline__ v16f mfma_scaled(const v8i& a, const v8i& b, const v16f& c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, ea, kByte, eb);
}

// The same product added to an accumulator in the accumulation registers, written in assembly so that it
// stays there (the compiler otherwise moves accumulators between the two register files in bulk). The
// wait in front of the first term's covers operands that vector instructions have just written; the second
// term's product follows it with the same values. Scale codes: byte 0 of `codes` for a, byte 1 (kLow: 2) for b.
template <bool kLow>
__device__ __forceinline__ void mfma_scaled_acc(const v8i& a, const v8i& b, v16f& c, int codes) {
  if constexpr (kLow)
    asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %3 op_sel_hi:[0,1,0]"
                 : "+a"(c)
                 : "v"(a), "v"(b), "v"(codes));
  else
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %3 op_sel:[0,1,0] op_sel_hi:[0,0,0]"
                 : "+a"(c)
                 : "v"(a), "v"(b), "v"(codes));
}
// Keeps an accumulator in the accumulation registers at this point.
__device__ __forceinline__ void keep_acc(v16f& c) { asm volatile("" : "+a"(c)); }

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

// kPairs pairs of waves, 32 query rows each.
template <int kPairs>
__global__ __launch_bounds__(kPairs * 128, 1) void latent_attn_kernel(LatentAttnArgs a) {
  constexpr int kBM = kPairs * 32, kWaves = kPairs * 2;
  constexpr int kWeightsAt = kBuffers * kTileBytes, kRefsAt = kWeightsAt + kWaves * kWeightBytes;
  constexpr int kKeysAt = kRefsAt + kWaves * kRefBytes;
  __shared__ __align__(1024) uint8_t lds_tiles[kKeysAt + kWaves * kKeyBytes];
  Work work;
  if (!find_work<kBM, kTile>(a, work)) return;
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
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const int last_tok = uniform((work.block * kBM + rows - 1) / a.H);
  const int keys = min(max(seq.len - seq.n + last_tok + 1, 0), seq.len);
  const int tiles = (keys + kTile - 1) / kTile;
  const int t_begin = uniform((int)((int64_t)tiles * work.part / work.parts));
  const int t_end = uniform((int)((int64_t)tiles * (work.part + 1) / work.parts));
  // keys that every row of the block sees: tiles before need no mask
  const int first_tok = uniform(work.block * kBM / a.H);
  const int all = rows == kBM ? min(max(seq.len - seq.n + first_tok + 1, 0), seq.len) : 0;

  v16f acc[8];  // columns 256 half + 32 d .. + 31
#pragma unroll
  for (int d = 0; d < 8; ++d) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
    keep_acc(acc[d]);
  }
  // The accumulator's weights are relative to 2^m (the same in both waves of a pair); l sums this wave's keys.
  float m = kNone, l = 0.f;
  const uint32_t lds = lds_addr(lds_tiles);

  if (t_begin < t_end) {
    const uint16_t* q_row = a.q + qtok * a.q_tok + (int64_t)head * a.q_head;
    RawQuery raw;
    read_query(q_row, row_ok, g, half, raw);
    // ---- the page table and the scale codes are read ahead: lane L for key L of a tile
    // (no branches: a column past the table reads its last entry, or where it has none a length, and counts as none)
    const int width = a.cache.table_width;
    const int32_t* table = width > 0 ? a.cache.table + (int64_t)work.index * a.cache.table_stride : a.lens;
    const int page_size = a.cache.page_size;
    const int step_col = uniform(kTile / page_size), step_off = kTile - step_col * page_size;
    const int end_col = uniform((keys - 1) / page_size), end_off = (keys - 1) - end_col * page_size;
    int key = t_begin * kTile + lane, col = key / page_size, off = key - col * page_size;
    // Of a tile: the table's entry (valid: whether the table has one) and the row in its page; keys past the end
    // repeat the last (masked). What is loaded is not touched before the next tile's wait.
    struct Entry {
      int page, row, valid;
    };
    auto look_up = [&](Entry& x) {
      const bool past = key >= keys;
      const int at = past ? end_col : col;
      x.row = past ? end_off : off;
      x.page = table[min(at, max(width - 1, 0))];
      x.valid = at < width;
      key += kTile;
      col += step_col;
      off += step_off;
      const bool wrap = off >= page_size;
      off -= wrap ? page_size : 0;
      col += wrap ? 1 : 0;
    };
    const uint32_t page_units = (uint32_t)(a.cache.page_stride / 128);
    // A row's place in 128-byte units, and its scale code as loaded; a key without a page has the code of NaN
    // (and reads page 0's first).
    struct Row {
      uint32_t unit;
      int byte, none;
    };
    auto row_of = [&](const Entry& x) {
      const bool none = !x.valid || (unsigned)x.page >= (unsigned)a.cache.pages;
      const int p = none ? 0 : x.page, o = none ? 0 : x.row;
      return Row{(uint32_t)p * page_units + (uint32_t)o * (kLatentRow / 128),
                 a.cache.scales[(int64_t)p * a.cache.scale_stride + o], none ? 255 : 0};
    };
    // ---- copies of a tile: a wave's groups of 8 rows, lanes 8 r .. 8 r + 7 at row r, five blocks of 128 bytes each
    constexpr int kGroups = 8 / kWaves, kCopies = 5 * kGroups;
    auto swizzle = [](int row) { return ((row >> 2) & 1) | (row & 2); };
    const uint8_t* lane_src = a.cache.rows + (((lane & 7) ^ swizzle(lane >> 3)) << 4);
    const int row_from = (wave * kGroups * 8 + (lane >> 3)) << 2;
    auto places_of = [&](const Row& x, const uint8_t** places) {  // of the rows, from the lanes that looked them up
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const uint32_t u = (uint32_t)__builtin_amdgcn_ds_bpermute(row_from + 32 * j, (int)x.unit);
        places[j] = lane_src + (uint64_t)u * 128;
      }
    };
    auto put_missing = [&](const Row& x, const uint8_t** places) {  // keys without a page on the row of zeros
      if (__builtin_expect(__any(x.none), 0)) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j)
          if (__builtin_amdgcn_ds_bpermute(row_from + 32 * j, x.none))
            places[j] = reinterpret_cast<const uint8_t*>(kZeroRow) + (lane_src - a.cache.rows);
      }
    };
    auto copy_piece = [&](const uint8_t* const* places, uint32_t tile, auto piece) {
      constexpr int j = decltype(piece)::v, group = j / 5, block = j % 5;
      copy16_block<128 * block>(places[group], tile + (wave * kGroups + group) * kGroupBytes + (kBlockBytes - 128) * block);
    };
    auto copy_pieces = [&](const uint8_t* const* places, uint32_t tile, auto first, auto count) {
      static_for<decltype(count)::v>([&](auto i) {
        constexpr int j = decltype(first)::v + decltype(i)::v;
        if constexpr (j < kCopies) copy_piece(places, tile, Const<j>{});
      });
    };

    Entry here, next, far;
    look_up(here);
    look_up(next);
    look_up(far);  // of tile t + 2
    int code;      // of tile t
    {
      const Row x = row_of(here);
      const uint8_t* from[kGroups];
      places_of(x, from);
      put_missing(x, from);
      copy_pieces(from, lds, Const<0>{}, Const<kCopies>{});
      code = x.byte | x.none;
    }
    Row ahead = row_of(next);  // of tile t + 1
    Query q;
    split_query<kWaves>(raw, lane, wave, lds_tiles + kTileBytes, q);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row_ok) v = *reinterpret_cast<const uint4*>(q_row + kLatentDim + 16 * ks + 8 * g);
      q.rope[ks] = __builtin_bit_cast(v8bf, v);
    }
    const float c = __uint_as_float((uint32_t)uniform((int)__float_as_uint(a.scale * 1.44269504088896341f)));

    // ---- LDS addresses within a tile
    typedef __attribute__((address_space(3))) const v4i lds_v4i;
    typedef __attribute__((address_space(3))) v4i lds_w4i;
    typedef __attribute__((address_space(3))) const v4f lds_v4f;
    typedef __attribute__((address_space(3))) float lds_f;
    typedef __attribute__((address_space(3))) v2i lds_v2i;
    const uint32_t key_base = (half * 4 + (r >> 3)) * kGroupBytes + (r & 7) * 128;
    const uint32_t key_first = key_base + ((g ^ swizzle(r)) << 4), key_second = key_base + (((2 + g) ^ swizzle(r)) << 4);
    const int vk = 4 * g + ((lane >> 1) & 3);  // the row this lane addresses, of every other group
    const uint32_t value_base = ((lane >> 3) & 1) * kGroupBytes + vk * 128 + 8 * (lane & 1) + 2 * half * kBlockBytes;
    const int value_column = ((lane >> 4) & 1) ^ swizzle(vk);
    const uint32_t value_even = value_base + (value_column << 4), value_odd = value_base + ((2 ^ value_column) << 4);  // d
    const uint32_t weights = lds + kWeightsAt + pair * (2 * kWeightBytes) + lane * 16;  // half, tile in turn, term
    const uint32_t refs = lds + kRefsAt + pair * (2 * kRefBytes) + r * 4;
    const uint32_t floats = lds + kKeysAt + wave * kKeyBytes;

    // ---- softmax of this lane's 16 scores, in pieces that fit between matrix products
    struct Soft {
      v16f x;          // score in log2 + scale code of the key
      v4f inv[4];      // 2^-e of keys 8 q + 4 g .. + 3
      float ref, sum[2];  // weights are 2^(x - ref); two sums, so that no addition waits for the one before
    };
    auto soft_x = [&](const v16f& s, const v4f* e, Soft& w) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w.x[i] = fmaf(s[i], c, e[i >> 2][i & 3]);
    };
    auto soft_mask = [&](int t, Soft& w) {
      const int k0 = t * kTile + half * 32;
      if (__builtin_expect(k0 + 32 > all, 0)) {  // (out of the loop's line: a taken branch costs it dear)
        const int left = limit - k0 - 4 * g;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (8 * (i >> 2) + (i & 3) >= left) w.x[i] = kNegInf;
      }
    };
    auto soft_top = [&](Soft& w) {
      float top = w.x[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, w.x[i]);
      const unsigned bits = __float_as_uint(top);
      const auto both = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
      top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1]));
      // (where whole numbers are 16 apart, 2^27 on, top - kTop may be rounded to top - 16: the weights would pass 448)
      const float low = ceilf(top) - kTop;
      w.ref = top == kNegInf ? kNone : low + kTop < top ? top : low;
      w.sum[0] = w.sum[1] = 0.f;
    };
    // Weights of keys 2 k and 2 k + 1; the same into the two terms.
    auto soft_weight = [&](Soft& w, float ref, int k) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = 2 * k + j;
        w.x[i] = __builtin_amdgcn_exp2f(w.x[i] - ref);
        w.sum[j] = fmaf(w.x[i], w.inv[i >> 2][i & 3], w.sum[j]);  // (a masked key's weight is 0, whatever its scale)
      }
    };
    auto soft_terms = [&](const Soft& w, int k, v4i& hi, v4i& lo) {
      typedef float v2f __attribute__((ext_vector_type(2)));
      const int q4 = k >> 1;
      const float p0 = w.x[2 * k], p1 = w.x[2 * k + 1];
      // what the first term leaves, 16 times: exact
      if (k & 1) {
        hi[q4] = __builtin_amdgcn_cvt_pk_fp8_f32(p0, p1, hi[q4], true);
        const v2f back = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((unsigned)hi[q4], 16.f, true);
        lo[q4] = __builtin_amdgcn_cvt_pk_fp8_f32(fmaf(p0, 16.f, -back[0]), fmaf(p1, 16.f, -back[1]), lo[q4], true);
      } else {
        hi[q4] = __builtin_amdgcn_cvt_pk_fp8_f32(p0, p1, 0, false);
        const v2f back = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((unsigned)hi[q4], 16.f, false);
        lo[q4] = __builtin_amdgcn_cvt_pk_fp8_f32(fmaf(p0, 16.f, -back[0]), fmaf(p1, 16.f, -back[1]), 0, false);
      }
    };
    // Piece 0 .. 9: the weights of pair `piece` and the terms of the pair two before, so that results are not
    // waited for.
    auto soft_piece = [&](Soft& w, float ref, int piece, v4i& hi, v4i& lo) {
      if (piece < 8) soft_weight(w, ref, piece);
      if (piece >= 2) soft_terms(w, piece - 2, hi, lo);
      // (here, not after the products)
      if (piece < 8) asm volatile("" : "+v"(w.x[2 * piece]), "+v"(w.x[2 * piece + 1]), "+v"(w.sum[0]), "+v"(w.sum[1]));
      if (piece >= 2) asm volatile("" : "+v"(hi[(piece - 2) >> 1]), "+v"(lo[(piece - 2) >> 1]));
    };
    // ---- the weights of a tile, as both waves of the pair wrote them: slots 0 .. 31 of a product are the first
    // wave's keys, 32 .. 63 the second's, each under its own scale code (lanes g = 0 and 1 hold the two)
    struct Weights {
      v8i hi, lo;
      float r0, r1;
      int codes;
    };
    auto read_weights = [&](int turn, Weights& w) {
      const uint32_t at = weights + turn * 2048;
      w.r0 = *reinterpret_cast<lds_f*>(refs + turn * 128), w.r1 = *reinterpret_cast<lds_f*>(refs + turn * 128 + kRefBytes);
      const v4i h0 = *reinterpret_cast<lds_v4i*>(at), h1 = *reinterpret_cast<lds_v4i*>(at + kWeightBytes);
      const v4i l0 = *reinterpret_cast<lds_v4i*>(at + 1024), l1 = *reinterpret_cast<lds_v4i*>(at + kWeightBytes + 1024);
      w.hi = __builtin_shufflevector(h0, h1, 0, 1, 2, 3, 4, 5, 6, 7);
      w.lo = __builtin_shufflevector(l0, l1, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    // Their scale codes, and a new reference where they pass the old one (no branches but for the accumulator).
    // Returns its factor.
    auto refer = [&](Weights& w, float ref_own, float sum_own) {
      const float top = fmaxf(w.r0, w.r1);
      const bool higher = top > m + kSlack;  // also at the first key that a row sees (m = kNone; the accumulator is zero)
      const float f = higher && m > kNone ? __builtin_amdgcn_exp2f(m - top) : 1.f;
      m = higher ? top : m;
      // (exponents far below the reference stop at 2^-120 of it)
      const int up = (int)fmaxf((g ? w.r1 : w.r0) - m, -120.f);
      w.codes = 127 | (127 + up) << 8 | (123 + up) << 16;
      l = fmaf(l, f, __builtin_amdgcn_ldexpf(sum_own, (int)(ref_own - m)));
      return f;
    };
    auto rescale = [&](float f) {
      if (__builtin_expect(__any(f != 1.f), 0)) {
        asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");  // products in flight
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          keep_acc(acc[d]);
          acc[d] *= f;
          keep_acc(acc[d]);
        }
      }
    };
    // ---- O^T += V^T P^T, 32 value columns at a time; `between(i)` is called after each of 14 products. The first
    // columns are read by the caller, and the last ones are left to finish(): after the next barrier, while
    // the first keys are read.
    auto value_at = [&](uint32_t tile, int d) {
      const uint32_t at = tile + ((d & 1) ? value_odd : value_even) + (d >> 2) * kBlockBytes + (d & 2) * 32;
      v2i x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<lds_v2i*>(at + i * 2 * kGroupBytes));
      return v8i{x[0][0], x[0][1], x[1][0], x[1][1], x[2][0], x[2][1], x[3][0], x[3][1]};
    };
    Weights late{};  // (nothing is late at the first tile: its products are with zeros)
    v8i late_v{};
    late.codes = 127 | 127 << 8 | 127 << 16;
    auto values = [&](uint32_t tile, const Weights& w, const v8i& v0, auto between) {
      v8i v[2];
      v[0] = v0;
#pragma unroll
      for (int d = 0; d < 7; ++d) {
        v[(d + 1) & 1] = value_at(tile, d + 1);
        mfma_scaled_acc<false>(v[d & 1], w.hi, acc[d], w.codes);
        between(2 * d);
        __builtin_amdgcn_sched_barrier(0);
        mfma_scaled_acc<true>(v[d & 1], w.lo, acc[d], w.codes);
        between(2 * d + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      late = w;
      late_v = v[1];
    };
    auto finish = [&] {
      mfma_scaled_acc<false>(late_v, late.hi, acc[7], late.codes);
      mfma_scaled_acc<true>(late_v, late.lo, acc[7], late.codes);
    };

    // ---- scores of this wave's 32 keys of a tile; `between(step)` is called at each of 8 steps
    auto scores = [&](uint32_t tile, int kc, auto between) {
      auto key_at = [&](int ks) {
        const v4i x = *reinterpret_cast<lds_v4i*>(tile + key_first + (ks >> 1) * kBlockBytes + (ks & 1) * 64);
        const v4i y = *reinterpret_cast<lds_v4i*>(tile + key_second + (ks >> 1) * kBlockBytes + (ks & 1) * 64);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
      };
      auto rope_at = [&](int ks) {
        return __builtin_bit_cast(v8bf, *reinterpret_cast<lds_v4i*>(tile + ((ks & 1) ? key_second : key_first) + 4 * kBlockBytes + (ks >> 1) * 64));
      };
      v8i k[3];
      v8bf kr[4];
      k[0] = key_at(0);
      k[1] = key_at(1);
      finish();
      v16f s;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0.f;
      static_for<8>([&](auto step) {
        constexpr int ks = decltype(step)::v;
        if constexpr (ks + 2 < 8) k[(ks + 2) % 3] = key_at(ks + 2);
        else kr[2 * ks - 12] = rope_at(2 * ks - 12), kr[2 * ks - 11] = rope_at(2 * ks - 11);
        s = mfma_scaled<0>(k[ks % 3], q.hi[ks], s, kc, q.code);
        s = mfma_scaled<1>(k[ks % 3], q.lo[ks], s, kc, q.code);
        asm volatile("" : "+v"(s));  // the products stay here
        between(step);
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kr[ks], q.rope[ks], s, 0, 0, 0);
      return s;
    };
    constexpr int kSteps = 5, kEach = kCopies / kSteps;
    const uint8_t* places[kGroups];  // where the rows of the next copies lie
    int kc;                    // scale code of this lane's key of the tile at hand
    auto prepare = [&](int tile_code, const Row& x) {
      kc = __builtin_amdgcn_ds_bpermute((half * 32 + r) << 2, tile_code);
      places_of(x, places);
      *reinterpret_cast<lds_f*>(floats + lane * 4) = (float)tile_code;
      *reinterpret_cast<lds_f*>(floats + 256 + lane * 4) = __builtin_amdgcn_ldexpf(1.f, 127 - tile_code);
    };
    prepare(code, ahead);
    uint32_t tile = lds, tile_before = lds;
    int place = 0, turn = 0;
    float ref_before = kNone, sum_before = 0.f;
    // Before the first tile there are no weights: its value products are with zeros (one copy of the code, which
    // every workgroup has to fetch, costs less than a step without them would save).
    {
      const uint32_t at = weights + half * kWeightBytes + 2048;
      *reinterpret_cast<lds_w4i*>(at) = v4i{0, 0, 0, 0};
      *reinterpret_cast<lds_w4i*>(at + 1024) = v4i{0, 0, 0, 0};
      *reinterpret_cast<lds_f*>(refs + half * kRefBytes + 128) = kNone;
    }
    for (int t = t_begin; t < t_end; ++t) {
      // tile t and what was read ahead have landed, the weights of tile t - 1 are written, and every wave is
      // done with the tile whose place is next
      wait_copies();
      asm volatile("" : "+v"(far.page), "+v"(ahead.byte));
      lds_barrier();
      const int next_place = place + 1 == kBuffers ? 0 : place + 1;
      const uint32_t next_tile = lds + next_place * kTileBytes;
      code = ahead.byte | ahead.none;
      // (after the last tile the copies bring one that is not used: there always is a key to look up)
      Weights before;
      v8i v0;
      float f = 1.f;
      const v16f s = scores(tile, kc, [&](auto ks) {
        constexpr int step = decltype(ks)::v;
        if (step == 0) put_missing(ahead, places);  // (beside the first products; before the barrier it costs 1 to 2 %)
        if constexpr (step < kSteps) copy_pieces(places, next_tile, Const<step * kEach>{}, Const<kEach>{});
        if (step == kSteps) {
          ahead = row_of(far);
          look_up(far);
        }
        if (step == 5) read_weights(turn ^ 1, before);
        if (step == 7) {
          f = refer(before, ref_before, sum_before);
          asm volatile("" : "+v"(f), "+v"(before.codes));
          v0 = value_at(tile_before, 0);
        }
      });
      Soft w;
      v4f e[4];
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
        e[q4] = *reinterpret_cast<lds_v4f*>(floats + (half * 32 + 8 * q4 + 4 * g) * 4);
        w.inv[q4] = *reinterpret_cast<lds_v4f*>(floats + 256 + (half * 32 + 8 * q4 + 4 * g) * 4);
      }
      v4i hi, lo;
      float ref;  // (a row that sees none of the keys: its x are -inf, its weights 0)
      rescale(f);
      values(tile_before, before, v0, [&](int d) {
        if (d == 0) soft_x(s, e, w);
        if (d == 1) soft_mask(t, w);
        if (d == 2) soft_top(w), ref = w.ref == kNone ? 0.f : w.ref;
        if (d >= 3 && d < 13) soft_piece(w, ref, d - 3, hi, lo);
      });
      const uint32_t at = weights + half * kWeightBytes + turn * 2048;
      *reinterpret_cast<lds_w4i*>(at) = hi;
      *reinterpret_cast<lds_w4i*>(at + 1024) = lo;
      *reinterpret_cast<lds_f*>(refs + half * kRefBytes + turn * 128) = w.ref;  // (lanes r and r + 32 write the same)
      prepare(code, ahead);
      ref_before = w.ref;
      sum_before = w.sum[0] + w.sum[1];
      turn ^= 1;
      tile_before = tile;
      tile = next_tile;
      place = next_place;
    }
    wait_copies();
    lds_barrier();
    Weights before;
    read_weights(turn ^ 1, before);
    finish();
    rescale(refer(before, ref_before, sum_before));
    values(tile_before, before, value_at(tile_before, 0), [](int) {});
    finish();
  }

  // the last products' results arrive (the compiler does not know what the assembly above was)
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int d = 0; d < 8; ++d) keep_acc(acc[d]);
  // ---- the row's sum over its keys, then the wave's columns
  l += __shfl_xor(l, 32);
  __syncthreads();
  float* sums = reinterpret_cast<float*>(lds_tiles);
  if (g == 0) sums[wave * 32 + r] = l;
  __syncthreads();
  const float l_all = sums[pair * 64 + r] + sums[pair * 64 + 32 + r];
  if (!row_ok) return;
  if (work.slot < 0) {
    const float inv = l_all == 0.f ? 0.f : 1.0f / l_all;  // a row that sees no key is zero
    uint16_t* dst = a.out + qtok * a.o_tok + (int64_t)head * a.o_head + 256 * half + 16 * g;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      // lanes g = 0 and 1 of a row swap quads of columns, so that each stores 16 neighbouring ones
      uint32_t u[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const auto v = __builtin_amdgcn_permlane32_swap(
              pack_bf16(acc[d][4 * h + 2 * i] * inv, acc[d][4 * h + 2 * i + 1] * inv),
              pack_bf16(acc[d][8 + 4 * h + 2 * i] * inv, acc[d][8 + 4 * h + 2 * i + 1] * inv), false, false);
          u[h][i] = v[0];
          u[h][2 + i] = v[1];
        }
      uint4* p = reinterpret_cast<uint4*>(dst + 32 * d);
      p[0] = make_uint4(u[0][0], u[0][1], u[0][2], u[0][3]);
      p[1] = make_uint4(u[1][0], u[1][1], u[1][2], u[1][3]);
    }
  } else {
    const int64_t state_row = (int64_t)work.slot * kBM + row;
    if (half == 0 && g == 0) {
      a.stats[state_row * 2] = m;
      a.stats[state_row * 2 + 1] = l_all;
    }
    float* state = a.states + state_row * kLatentDim + 256 * half + 4 * g;
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
        *reinterpret_cast<v4f*>(state + 32 * d + 8 * q4) = v4f{acc[d][4 * q4], acc[d][4 * q4 + 1], acc[d][4 * q4 + 2], acc[d][4 * q4 + 3]};
  }
}

constexpr int kMaxParts = 256;  // of a block: no more parts run at once

// Joins the parts of a cut block, in a fixed order: one wave a row or, where blocks are cut into many parts, eight, which take every 64 parts 8 a wave and add their sums through LDS. The lanes hold the parts'
// references and sums, then take 8 columns each. Bound by latency (a chain of three loads) where there are few
// rows, and by HBM and the L2s where every workgroup left a state.
template <int kBM, int kSplit>
__global__ __launch_bounds__(kSplit == 1 ? 256 : kSplit * 64) void latent_join_kernel(LatentAttnArgs a) {
  const int cuts = a.counts[0];
  const Desc desc = reinterpret_cast<const Desc*>(a.counts + 4)[blockIdx.x];
  if ((int)blockIdx.x >= cuts) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = kSplit == 1 ? blockIdx.y * 4 + wave : blockIdx.y;
  constexpr int kSpan = 64 / kSplit;  // of every 64 parts, this wave's
  const int first = kSplit == 1 ? 0 : wave * kSpan;
  if (row >= desc.rows || desc.parts > kMaxParts || desc.slot + desc.parts > a.max_slots) return;
  // the first parts' states are on their way while the statistics are joined
  constexpr int kTogether = 8;
  const float* src = a.states + ((int64_t)desc.slot * kBM + row) * kLatentDim + lane * 8;
  v4f x[kTogether], y[kTogether];
  auto read_states = [&](int p0, int last) {
#pragma unroll
    for (int k = 0; k < kTogether; ++k) {
      const v4f* at = reinterpret_cast<const v4f*>(src + (int64_t)min(p0 + k, last) * kBM * kLatentDim);
      x[k] = at[0], y[k] = at[1];
    }
  };
  read_states(first, desc.parts - 1);
  constexpr int kEach = kMaxParts / 64;
  float f[kEach], sums[kEach];
  float m = kNegInf;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int p = 64 * i + lane;
    f[i] = kNegInf;
    sums[i] = 0.f;
    if (p < desc.parts) {
      const float2 x = reinterpret_cast<const float2*>(a.stats)[(int64_t)(desc.slot + p) * kBM + row];
      f[i] = x.x;
      sums[i] = x.y;
    }
    m = fmaxf(m, f[i]);
  }
#pragma unroll
  for (int mask = 1; mask < 64; mask <<= 1) m = fmaxf(m, __shfl_xor(m, mask));
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    f[i] = f[i] == m ? 1.f : __builtin_amdgcn_exp2f(f[i] - m);
    l = fmaf(f[i], sums[i], l);
  }
#pragma unroll
  for (int mask = 1; mask < 64; mask <<= 1) l += __shfl_xor(l, mask);
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int n = min(desc.parts - 64 * i, first + kSpan);
    for (int p0 = first; p0 < n; p0 += kTogether) {
      if (i > 0 || p0 > first) read_states(64 * i + p0, desc.parts - 1);
#pragma unroll
      for (int k = 0; k < kTogether; ++k) {
        // (past the last part: its state again, times zero)
        const float at = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(f[i]), min(p0 + k, 63)));
        const float fp = p0 + k < n ? at : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = fmaf(fp, x[k][j], o[j]), o[4 + j] = fmaf(fp, y[k][j], o[4 + j]);
      }
    }
  }
  if constexpr (kSplit > 1) {
    __shared__ float sums_of[kSplit][kLatentDim];
#pragma unroll
    for (int j = 0; j < 8; ++j) sums_of[wave][j * 64 + lane] = o[j];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < kSplit; ++w)
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += sums_of[w][j * 64 + lane];
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const int flat = desc.first + row, tok = flat / a.H, head = flat - tok * a.H;
  uint16_t* dst = a.out + (int64_t)tok * a.o_tok + (int64_t)head * a.o_head + lane * 8;
  *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                                              pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv));
}

constexpr int kCUs = 256;
static_assert(kCUs <= kMaxParts, "a block's parts fit the join's lanes");
// Where no sequence has more tiles, no block is cut and there is no second launch (1 sequence x 128 heads, 200 keys:
// 17.6 us in two parts, 15.5 whole).
constexpr int kWhole = 4;

// Pairs of waves a workgroup: one where a sequence has 32 query rows or fewer on average (64 sequences x 32 heads:
// 53 us, 59 with two pairs; x 48 heads: 102 and 65), or where blocks of 32 rows leave at most 8 tiles for each
// compute unit, so that half as large states weigh more than the idle SIMDs (128 heads: 8 sequences of 4000 keys 34.5
// us, 37.1 with two pairs; 16 of 2000 34.9 and 35.7; 16 of 4000 48.2 and 43.5).
int pairs_for(int64_t T, int64_t B, int64_t H, int64_t max_tiles) {
  const int64_t rows = T * H, most = 32 * 8 * kCUs;
  return rows <= 32 * B || (rows <= most && rows * max_tiles <= most) ? 1 : 2;
}

// Tiles a part at least: 2, or 3 of long sequences, where more states cost more than they save (1 sequence x 128
// heads, at least 2 or 3: 1000 keys 19.7 and 19.9 us, 4000 26.7 and 23.6).
int min_tiles_for(int64_t max_tiles) { return max_tiles > 32 ? 3 : 2; }

// Eight waves a row join more parts than this (1 sequence x 128 heads, one wave and eight: 32 parts 26.6 and 27.3 us,
// 63 parts 45.6 and 32.9).
constexpr int kManyParts = 32;

template <int kPairs>
hipError_t launch(const LatentAttnArgs& args, const LatentAttnPlan& plan, hipStream_t stream) {
  const int64_t grid = (plan.parts + 15) / 16 * 16;
  hipLaunchKernelGGL((latent_attn_kernel<kPairs>), dim3((unsigned)grid), dim3(kPairs * 128), 0, stream, args);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !plan.join) return e;
  if (plan.split_join)
    hipLaunchKernelGGL((latent_join_kernel<kPairs * 32, 8>), dim3((unsigned)plan.cuts, kPairs * 32), dim3(512), 0, stream, args);
  else
    hipLaunchKernelGGL((latent_join_kernel<kPairs * 32, 1>), dim3((unsigned)plan.cuts, kPairs * 8), dim3(256), 0, stream, args);
  return hipGetLastError();
}

}  // namespace

LatentAttnPlan plan_latent_attn(int64_t T, int64_t B, int64_t H, int64_t max_keys) {
  LatentAttnPlan p;
  const int64_t max_tiles = (max_keys + kTile - 1) / kTile;
  p.pairs = pairs_for(T, B, H, max_tiles);
  const int64_t bm = 32 * p.pairs;
  // Blocks: a sequence's last may be partly filled.
  p.blocks = T * H / bm + (T < B ? T : B);
  p.max_tiles = (int)max_tiles;
  p.target_parts = kCUs;
  p.min_tiles = min_tiles_for(max_tiles);
  // Blocks are cut only into as many parts as run at once in all.
  const int64_t per_block = (max_tiles + p.min_tiles - 1) / p.min_tiles;
  p.split_join = false;
  const int64_t fewest = (T * H + bm - 1) / bm;  // blocks, if the sequences' rows fill theirs
  // As many blocks as run at once are not cut, and the second launch, of which every workgroup would find nothing to
  // do, is left out (128 sequences x 128 heads: 4.6 us of GPU time beside 131.2, of which calls in a row show 0.4).
  // The workspace does not shrink for it.
  p.join = max_tiles > kWhole && fewest < kCUs;
  if (max_tiles <= kWhole) {
    p.slots = p.cuts = 0;
  } else {
    p.slots = p.target_parts;
    if (p.blocks * per_block < p.slots) p.slots = p.blocks * per_block;
    p.cuts = p.slots / 2;
    p.split_join = per_block > kManyParts && p.slots / fewest > kManyParts;  // the fewest are cut into most parts
  }
  p.parts = p.blocks > p.slots ? p.blocks : p.slots;
  p.counts_bytes = p.slots ? ((16 + p.cuts * sizeof(Desc) + 255) / 256) * 256 : 0;
  p.stats_bytes = ((p.slots * bm * 2 * sizeof(float) + 255) / 256) * 256;
  p.states_bytes = p.slots * bm * kLatentDim * sizeof(float);
  return p;
}

hipError_t launch_latent_attn(const LatentAttnArgs& args, const LatentAttnPlan& plan, hipStream_t stream) {
  return plan.pairs == 1 ? launch<1>(args, plan, stream) : launch<2>(args, plan, stream);
}

}  // namespace bfp8
