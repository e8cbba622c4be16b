// Accumulated attention weights of the tokens in the paged FP8 latent cache:
//   mass[b, j] += sum over new tokens t and heads h of softmax_j(scale q[t, h] . [c_j, r_j])
//
// A weight needs its row's maximum and sum over all keys first. A first launch scores the keys and leaves each row's
// maximum and sum over a part of the keys. A second forms the weights and adds them up over the rows: from the scores,
// where the first launch had room to leave them too, else by scoring the keys again, whose sums over blocks of 128 rows a
// third launch then adds up. Nothing is added by atomics: results do not depend on the order of the workgroups.
//
// Scores are bf16 products on the cached codes, which bf16 holds exactly (32x32x16 instructions, latents and
// rotary part in accumulators of their own, as the key's scale belongs to the first alone), so a weight is off by float32
// roundings only: the sums of thousands of weights stay good to 1e-5 or better.
//
// A workgroup holds 128 query rows of one sequence, 32 a wave, in registers and walks tiles of 32 keys, of which two are on
// their way to LDS while a third is multiplied (the layout is that of the attention kernel, without bank conflicts). Where
// the keys of its part lie is looked up before, 2048 at a time, so that the loop holds no dependent load. One
// instruction serves both directions: with the keys first a lane holds one row and 16 keys, whose maximum and sum are near;
// with the rows first it holds one key and 16 rows, whose weights add up in registers. Two workgroups run on a compute unit,
// so that one's softmax and conversions (128 instructions a tile) run beside the other's products.
//
// Measured, beside the attention: 1 sequence of 1111 x 128 heads 11.5 us for the scores (a chain of look-ups, rows and two tiles) and 7.7 for
// their sum; 64 of 500 to 8000 x 16 heads 38 us (186 MB of rows, 4.9 TB/s) and 12; 6 chunks of 40 x 128 heads 92 us for each of two passes (matrix
// cores busy 36 % of the clocks: parts of 43 tiles at most where an even share is 33, and a softmax that only another workgroup's products
// run beside) and 6.
//
// A row's weights are formed with its maximum and its sum apart, from scores that both passes round alike, so they add up to one wherever the scores
// lie in float32's range.
#include <algorithm>

#include "device_latent.h"
#include "latent.h"
#include "latent_work.h"
#include "launch.h"

namespace bfp8 {

namespace {

constexpr int kRows = 128;  // of a block
constexpr int kTile = 32;   // keys
// A tile in LDS: groups of 8 rows, each in 5 blocks of 128 bytes of every row and 64 bytes of padding; of each 64 bytes the
// 16-byte columns are XORed with bits 2 and 1 of the row.
constexpr int kBlockBytes = 8 * 128, kGroupBytes = 5 * kBlockBytes + 64;
constexpr int kTileBytes = 4 * kGroupBytes;
constexpr int kBuffers = 3;
constexpr int kMap = 2048;  // keys that are looked up at a time
constexpr float kNone = -__FLT_MAX__;  // a maximum over no keys: no finite score is below it
constexpr float kNegInf = -__builtin_inff();
constexpr uint32_t kNowhere = 0xffffffffu;

// The row that a key without a page stands on.
__device__ const uint4 kNoRow[kLatentRow / 16] = {};

// The keys that token `tok` of a sequence's new ones sees, and how many the page table reaches (a row that sees one past that is NaN).
__device__ __forceinline__ int sees(const Seq& s, int tok) { return min(max(s.len - s.n + tok + 1, 0), s.len); }
__device__ __forceinline__ int reach_of(const LatentAttnArgs& a) { return a.cache.table_width * a.cache.page_size; }  // (below 2^31)

// 8 codes as bf16, exactly.
__device__ __forceinline__ v8bf codes_bf16(int lo, int hi) {
  auto two = [](auto v) { return __builtin_bit_cast(int, v); };
  return __builtin_bit_cast(v8bf, v4i{two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false)),
                                      two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true)),
                                      two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false)),
                                      two(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true))});
}

// A row's maximum and sum over more keys.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  l = l * __builtin_amdgcn_exp2f(m - top) + l2 * __builtin_amdgcn_exp2f(m2 - top);
  m = top;
}
// What a row's weights are formed with, 2^(x - top) * share: the maximum over all keys that it sees and one over its sum. (They are not one
// number, top + log2(sum): for scores far from zero that rounds the sum away.) A row whose softmax is none (a key past the table, a sum that is
// NaN, or zero, as all its scores are minus infinity) has a NaN maximum and a finite share, so that a weight masked to zero stays zero.
__device__ __forceinline__ float2 row_sum(float m, float l, int limit, int reach) {
  if (limit == 0) return make_float2(0.f, 0.f);
  if (limit > reach || !(l > 0.f)) return make_float2(__builtin_nanf(""), 1.f);
  return make_float2(m, 1.f / l);
}

enum class Pass { kSums, kScores, kWeights };  // maxima and sums; the scores too; sums of weights by key

template <Pass kPass>
__global__ __launch_bounds__(256, 2) void latent_mass_kernel(LatentMassArgs args) {
  constexpr bool kWeights = kPass == Pass::kWeights;
  const LatentAttnArgs& a = args.work;
  __shared__ __attribute__((aligned(1024))) uint8_t tiles_lds[kBuffers * kTileBytes];
  __shared__ __attribute__((aligned(16))) uint32_t map_unit[kMap];  // where a key lies, in 128 bytes
  __shared__ __attribute__((aligned(16))) float map_scale[kMap];    // its scale times scale log2(e)
  __shared__ __attribute__((aligned(16))) float row_top[kRows];
  __shared__ __attribute__((aligned(16))) float row_share[kRows];
  __shared__ __attribute__((aligned(16))) int row_limit[kRows];
  __shared__ float sums[2][4][kTile];
  Work work;
  if (!find_work<kRows, kTile, 8>(a, work)) return;  // (more than 512 sequences are not cut, so none is looked at often)
  if (work.id - work.part + work.parts > args.ids) return;  // (starts that are not rising)
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, g = lane >> 5;
  const Seq seq = work.seq;
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const int rows = uniform((int)min((int64_t)seq.n * a.H - (int64_t)work.block * kRows, (int64_t)kRows));
  const int reach = reach_of(a);
  const int row = wave * 32 + r;
  const bool row_ok = row < rows;
  const bool active = uniform(wave * 32) < rows;
  const int flat = work.block * kRows + row;
  const int tok = row_ok ? flat / a.H : 0, head = row_ok ? flat - tok * a.H : 0;
  const int limit = row_ok ? sees(seq, tok) : 0;
  const int last_tok = uniform((work.block * kRows + rows - 1) / a.H);
  const int keys = min(sees(seq, last_tok), reach);
  const int tiles = (keys + kTile - 1) / kTile;
  const int even = tiles / work.parts, odd = tiles - even * work.parts;  // (the first parts take one tile more)
  const int t_begin = uniform(even * work.part + min(work.part, odd));
  const int t_end = uniform(t_begin + even + (work.part < odd ? 1 : 0));
  // keys that every row of the wave sees: tiles before need no mask
  const int all = uniform(wave * 32 + 32 <= rows ? limit : 0);
  const float c = a.scale * 1.44269504088896341f;
  // (rounded alike in both passes, so that no weight is above one)
  auto score = [&](float lat, float unit, float rot) { return fmaf(lat, unit, rot * c); };
  if (!kWeights && work.block == 0 && work.part == 0 && tid == 0) args.first[work.index] = make_int2(work.id, work.parts);

  if constexpr (kWeights) {
    // the rows' sums, joined over the parts of their block
    if (tid < kRows) {
      const int mine = work.block * kRows + tid;
      const int lim = tid < rows ? sees(seq, mine / a.H) : 0;
      float m = kNone, l = 0.f;
      const float2* p = args.stats + (int64_t)(work.id - work.part) * kRows + tid;
      if (tid < rows)
        for (int i = 0; i < work.parts; ++i) {
          const float2 f = p[(int64_t)i * kRows];
          join(m, l, f.x, f.y);
        }
      const float2 sum = row_sum(m, l, lim, reach);
      row_top[tid] = sum.x;
      row_share[tid] = sum.y;
      row_limit[tid] = lim;
    }
  }
  float tops[kWeights ? 16 : 1], shares[kWeights ? 16 : 1];
  if constexpr (kWeights) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const v4f top = *reinterpret_cast<const v4f*>(&row_top[wave * 32 + 8 * i + 4 * g]);
      const v4f share = *reinterpret_cast<const v4f*>(&row_share[wave * 32 + 8 * i + 4 * g]);
#pragma unroll
      for (int j = 0; j < 4; ++j) tops[4 * i + j] = top[j], shares[4 * i + j] = share[j];
    }
  }

  // ---- copies: the wave's 8 keys of a tile, lanes 8 i .. 8 i + 7 at key i
  auto swizzle = [](int k) { return ((k >> 2) & 1) | (k & 2); };
  const uint32_t lane_off = (uint32_t)(((lane & 7) ^ swizzle(lane >> 3)) << 4);
  const uint32_t lds = lds_addr(tiles_lds);
  auto copy_tile = [&](int i, int buffer) {  // tile i of those looked up
    const uint32_t unit = map_unit[i * kTile + wave * 8 + (lane >> 3)];
    const uint8_t* src = (unit == kNowhere ? reinterpret_cast<const uint8_t*>(kNoRow) : a.cache.rows + (uint64_t)unit * 128) + lane_off;
    const uint32_t dst = __builtin_amdgcn_readfirstlane(lds + buffer * kTileBytes + wave * kGroupBytes);
    static_for<5>([&](auto b) {
      constexpr int block = decltype(b)::v;
      copy16_block<128 * block>(src, dst + (kBlockBytes - 128) * block);
    });
  };
  const uint32_t key_base = (r >> 3) * kGroupBytes + (r & 7) * 128;
  const uint32_t key_first = key_base + ((g ^ swizzle(r)) << 4), key_second = key_base + (((2 + g) ^ swizzle(r)) << 4);

  float m = kNone, l = 0.f;  // of the lane's row, over its 16 keys of every tile
  float x[16];               // scores of a tile (kScores: stored a tile later)
  const int64_t row0 = (int64_t)seq.q0 * a.H;
  float* partial = kWeights ? args.partial + (row0 / kRows + work.index + work.block) * args.pitch : nullptr;
  float* scores = kPass == Pass::kScores ? args.scores + (row0 + flat) * args.pitch + 4 * g : nullptr;
  const int waves_on = (rows + 31) / 32;
  // what the tile before left, to memory
  auto flush = [&](int t, int turn) {
    if constexpr (kPass == Pass::kScores) {
      if (row_ok)
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<v4f*>(scores + t * kTile + 8 * i) = v4f{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
    }
    if constexpr (kWeights) {
      if (wave == (t & 3) && lane < kTile) {
        float v = sums[turn][0][lane];
        for (int w = 1; w < waves_on; ++w) v += sums[turn][w][lane];
        partial[t * kTile + lane] = v;
      }
    }
  };

  // ---- where the keys of tiles t0 .. t0 + n - 1 lie (four a thread at a time: their loads overlap)
  auto look_up = [&](int t0, int n) {
    for (int i0 = tid; i0 < n * kTile; i0 += 4 * 256) {
      int page[4], off[4], code[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = t0 * kTile + i0 + 256 * j, col = key / a.cache.page_size;
        off[j] = key - col * a.cache.page_size;
        page[j] = -1;
        if (i0 + 256 * j < n * kTile && key < keys) page[j] = a.cache.table[(int64_t)work.index * a.cache.table_stride + col];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (page[j] >= a.cache.pages) page[j] = -1;
        code[j] = 255;
        if (page[j] >= 0) code[j] = a.cache.scales[(int64_t)page[j] * a.cache.scale_stride + off[j]];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 256 * j;
        if (i >= n * kTile) break;
        map_unit[i] = page[j] < 0 ? kNowhere : (uint32_t)page[j] * (uint32_t)(a.cache.page_stride / 128) + (uint32_t)off[j] * (kLatentRow / 128);
        map_scale[i] = e8_value(code[j]) * c;
      }
    }
  };
  constexpr int kMapTiles = kMap / kTile;
  if (t_begin < t_end) look_up(t_begin, min(t_end - t_begin, kMapTiles));
  // ---- the wave's rows (asked for behind the look-up's chain of loads): step s holds dimensions 16 (2 (s / 2) + g) + 8 (s % 2) .. + 7,
  // then the rotary part
  v8bf q[36];
  {
    const uint16_t* from = a.q + (int64_t)(seq.q0 + tok) * a.q_tok + (int64_t)head * a.q_head;
#pragma unroll
    for (int s = 0; s < 36; ++s) {
      v4i v = {0, 0, 0, 0};
      if (row_ok) v = *reinterpret_cast<const v4i*>(from + (s < 32 ? 16 * (2 * (s >> 1) + g) + 8 * (s & 1) : kLatentDim + 8 * (2 * (s - 32) + g)));
      q[s] = __builtin_bit_cast(v8bf, v);
    }
  }
  for (int t0 = t_begin; t0 < t_end; t0 += kMapTiles) {
    const int n = min(t_end - t0, kMapTiles);
    if (t0 > t_begin) {
      __syncthreads();
      look_up(t0, n);
    }
    __syncthreads();
    copy_tile(0, 0);
    if (n > 1) copy_tile(1, 1);
    int buffer = 0;
    for (int i = 0; i < n; ++i) {
      const int t = t0 + i;
      // tile t has landed (the five copies of the next may be under way), and every wave is done with the one before
      if (i + 1 < n) wait_copies_upto<5>();
      else wait_copies();
      lds_barrier();
      if (t > t_begin && (kWeights || active)) flush(t - 1, (t - 1) & 1);
      if (i + 2 < n) copy_tile(i + 2, buffer == 0 ? 2 : buffer - 1);
      const uint8_t* tile = tiles_lds + buffer * kTileBytes;
      buffer = buffer == 2 ? 0 : buffer + 1;
      if (!active) continue;
      v16f lat, rot;
#pragma unroll
      for (int j = 0; j < 16; ++j) lat[j] = rot[j] = 0.f;
      // 16 bytes of codes are two products, then of the rotary part one. They are read four steps ahead, in an order that is held to (left
      // to itself the compiler reads them just before their products, which then wait).
      constexpr int kSteps = 20, kAhead = 4;
      v4i ring[kAhead];
      auto read = [&](int s) __attribute__((always_inline)) {
        const int block = s < 16 ? s >> 2 : 4, pair = s < 16 ? (s >> 1) & 1 : (s >> 1) - 8;
        ring[s % kAhead] = *reinterpret_cast<const v4i*>(tile + (s & 1 ? key_second : key_first) + block * kBlockBytes + pair * 64);
      };
      auto product = [&](v16f& sum, const v8bf& key, int step) __attribute__((always_inline)) {
        sum = kWeights ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[step], key, sum, 0, 0, 0)
                       : __builtin_amdgcn_mfma_f32_32x32x16_bf16(key, q[step], sum, 0, 0, 0);
      };
#pragma unroll
      for (int s = 0; s < kAhead; ++s) read(s);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const v4i k = ring[s % kAhead];
        if (s < 16) {
          const v8bf lo = codes_bf16(k[0], k[1]), hi = codes_bf16(k[2], k[3]);
          if (s + kAhead < kSteps) read(s + kAhead);
          product(lat, lo, 2 * s);
          product(lat, hi, 2 * s + 1);
        } else {
          product(rot, __builtin_bit_cast(v8bf, k), 16 + s);
          if (s + kAhead < kSteps) read(s + kAhead);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (kWeights) {
        const float unit = map_scale[i * kTile + r];
        float total = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __builtin_amdgcn_exp2f(score(lat[j], unit, rot[j]) - tops[j]);
        if (t * kTile + kTile > all) {
#pragma unroll
          for (int j4 = 0; j4 < 4; ++j4) {
            const v4i lim = *reinterpret_cast<const v4i*>(&row_limit[wave * 32 + 8 * j4 + 4 * g]);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * j4 + j] = t * kTile + r < lim[j] ? x[4 * j4 + j] : 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) total = fmaf(x[j], shares[j], total);
        total += __shfl_xor(total, 32);
        if (g == 0) sums[t & 1][wave][r] = total;
      } else {
#pragma unroll
        for (int j4 = 0; j4 < 4; ++j4) {
          const v4f unit = *reinterpret_cast<const v4f*>(&map_scale[i * kTile + 8 * j4 + 4 * g]);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[4 * j4 + j] = score(lat[4 * j4 + j], unit[j], rot[4 * j4 + j]);
        }
        if (t * kTile + kTile > all) {
          const int left = limit - t * kTile - 4 * g;
#pragma unroll
          for (int j = 0; j < 16; ++j) x[j] = 8 * (j >> 2) + (j & 3) >= left ? kNegInf : x[j];
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, x[j]);
        float more[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 16; ++j) more[j & 1] += __builtin_amdgcn_exp2f(x[j] - top);
        l = fmaf(l, __builtin_amdgcn_exp2f(m - top), more[0] + more[1]);
        m = top;
      }
    }
  }
  if constexpr (kWeights) lds_barrier();
  if (t_begin < t_end && (kWeights || active)) flush(t_end - 1, (t_end - 1) & 1);
  if constexpr (!kWeights) {
    join(m, l, __shfl_xor(m, 32), __shfl_xor(l, 32));
    if (g == 0 && row_ok) args.stats[(int64_t)work.id * kRows + row] = make_float2(m, l);
  }
}

// The keys of a workgroup of the last launch.
constexpr int kSumKeys = 256;
constexpr int sum_keys(bool more) { return more ? kSumKeys / 2 : kSumKeys; }

// The mass that a token had: none if it is new in this call, and none is past the sequence.
__device__ __forceinline__ float mass_before(const LatentMassArgs& args, const Seq& seq, int b, int key) {
  return args.mass_in != nullptr && key < min(seq.len - seq.n, args.width) ? args.mass_in[(int64_t)b * args.in_stride + key] : 0.f;
}
__device__ __forceinline__ void store_mass(const LatentMassArgs& args, const Seq& seq, int b, int key, int reach, float mass) {
  if (key < args.width) args.mass[(int64_t)b * args.out_stride + key] = key < min(seq.len, reach) ? mass : 0.f;
}

// Weights from the scores: the lanes of a wave hold 4 keys each, and four waves take every fourth row, 4 rows at a time. Of sequences with
// many rows lanes hold 2 keys (kVec) and waves take 8 rows at a time; 16 waves then hold 128 rows all at once and join the sums of 512.
// Bound by latency: what does not depend on anything else is asked for at once, the masses that were there and the first scores before the
// rows' sums are joined and, by 16 waves, the next scores before these rows' weights are formed.
template <int kWaves, int kVec>
__global__ __launch_bounds__(kWaves * 64) void latent_sum_kernel(LatentMassArgs args) {
  constexpr int kTogether = 16 / kVec, kThreads = 64 * kWaves, kAtOnce = kThreads / 2;
  constexpr bool kAhead = kWaves == 16;  // (with more workgroups a compute unit the registers are worth more: 64 x 16 heads 49 us, 52 so)
  static_assert(kAtOnce % kRows == 0, "rows at once are whole blocks");
  typedef float vec __attribute__((ext_vector_type(kVec)));
  const LatentAttnArgs& a = args.work;
  __shared__ float2 row_sums[kAtOnce];
  __shared__ int row_limit[kAtOnce];
  __shared__ float2 joined[kThreads];
  __shared__ __attribute__((aligned(16))) vec sums[kWaves][64];
  const int b = (int)(blockIdx.x / (unsigned)args.each), first = (int)(blockIdx.x - (unsigned)b * args.each);
  const int2 parts = args.first[b];  // (not set where a sequence has no rows)
  const Seq seq = sequence(a, b);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t rows = (int64_t)seq.n * a.H, row0 = (int64_t)seq.q0 * a.H;
  const int reach = reach_of(a), keys = min(seq.len, reach);
  // (unsigned: the step past the last column may pass 2^31, but not 2^32)
  for (unsigned at = (unsigned)first * 64 * kVec; at < (unsigned)args.width; at += (unsigned)args.each * 64 * kVec) {
    const int k0 = (int)at, key = k0 + lane * kVec;
    const float before = tid < 64 * kVec ? mass_before(args, seq, b, k0 + tid) : 0.f;
    vec total = 0.f;
    for (int64_t from_row = 0; from_row < rows && k0 < keys; from_row += kAtOnce) {
      const int count = (int)min(rows - from_row, (int64_t)kAtOnce), blocks = (count + kRows - 1) / kRows;
      const int64_t id = parts.x + from_row / kRows * parts.y;
      if (parts.x < 0 || parts.y < 1 || (int64_t)blocks * parts.y > args.ids - id) break;  // (starts that are not rising)
      const float* from = args.scores + (row0 + from_row) * args.pitch + key;
      auto read = [&](int p, vec* x) __attribute__((always_inline)) {  // (what no key of the row's block filled is not used below)
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
          if (p + kWaves * i < count && key < keys) x[i] = *reinterpret_cast<const vec*>(from + (int64_t)(p + kWaves * i) * args.pitch);
      };
      vec x[kAhead ? 2 : 1][kTogether];
      read(wave, x[0]);
      // ---- the rows' sums: 2 to 64 threads a row take every so many parts, then one joins theirs
      const int held = count <= 16 ? 16 : 1 << (32 - __builtin_clz(count - 1)), ways = kThreads / held;
      const int of = min(tid & (held - 1), count - 1), way = tid / held;
      float m = kNone, l = 0.f;
      const float2* from_stats = args.stats + (id + of / kRows * parts.y) * kRows + of % kRows;
      constexpr int kBatch = kWaves == 4 && kVec == 2 ? 12 : 4;
      for (int i = way; i < parts.y; i += kBatch * ways) {
        float2 f[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) f[j] = from_stats[(int64_t)min(i + j * ways, parts.y - 1) * kRows];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i + j * ways < parts.y) join(m, l, f[j].x, f[j].y);
      }
      joined[tid] = make_float2(m, l);
      lds_barrier();
      if (tid < count) {
        for (int i = 1; i < ways; ++i) {
          const float2 f = joined[i * held + tid];
          join(m, l, f.x, f.y);
        }
        const int limit = sees(seq, (int)((from_row + tid) / a.H));
        row_sums[tid] = row_sum(m, l, limit, reach);
        row_limit[tid] = min(limit, reach);
      }
      lds_barrier();
      auto add = [&](int p, const vec* x) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          const int at = min(p + kWaves * i, count - 1);
          const float2 sum = row_sums[at];
          const int limit = p + kWaves * i < count ? row_limit[at] : 0;
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            const float w = __builtin_amdgcn_exp2f(x[i][j] - sum.x);
            total[j] = fmaf(key + j < limit ? w : 0.f, sum.y, total[j]);
          }
        }
      };
      constexpr int kStep = kWaves * kTogether;
      if constexpr (kAhead) {
        for (int p = wave; p < count; p += 2 * kStep) {
          if (p + kStep < count) read(p + kStep, x[1]);
          add(p, x[0]);
          if (p + kStep >= count) break;
          if (p + 2 * kStep < count) read(p + 2 * kStep, x[0]);
          add(p + kStep, x[1]);
        }
      } else {
        for (int p = wave; p < count; p += kStep) {
          if (p > wave) read(p, x[0]);
          add(p, x[0]);
        }
      }
      lds_barrier();
    }
    sums[wave][lane] = total;
    lds_barrier();
    if (tid < 64 * kVec) {
      const float* flat = reinterpret_cast<const float*>(sums) + tid;
      float of_waves[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) of_waves[w & 3] += flat[w * 64 * kVec];
      store_mass(args, seq, b, k0 + tid, reach, before + ((of_waves[0] + of_waves[1]) + (of_waves[2] + of_waves[3])));
    }
    lds_barrier();
  }
}

// The sums of a sequence's blocks of rows.
__global__ __launch_bounds__(kSumKeys) void latent_blocks_kernel(LatentMassArgs args) {
  const LatentAttnArgs& a = args.work;
  const int b = (int)(blockIdx.x / (unsigned)args.each), first = (int)(blockIdx.x - (unsigned)b * args.each);
  const Seq seq = sequence(a, b);
  const int64_t rows = (int64_t)seq.n * a.H, row0 = (int64_t)seq.q0 * a.H;
  const int reach = reach_of(a), blocks = (int)((rows + kRows - 1) / kRows);
  // (unsigned: the step past the last column may pass 2^31, but not 2^32)
  for (unsigned at = (unsigned)first * kSumKeys + threadIdx.x; at < (unsigned)args.width; at += (unsigned)args.each * kSumKeys) {
    const int key = (int)at;
    float total = 0.f;
    if (blocks > 0 && key < min(seq.len, reach)) {
      // the first block whose last row sees the key: later ones all do
      const int64_t from = (int64_t)max(key - (seq.len - seq.n), 0) * a.H / kRows;
      const float* p = args.partial + (row0 / kRows + b) * args.pitch + key;
#pragma unroll 4
      for (int64_t i = from; i < blocks; ++i) total += p[i * args.pitch];
    }
    store_mass(args, seq, b, key, reach, mass_before(args, seq, b, key) + total);
  }
}

template <Pass kPass>
hipError_t launch_pass(const LatentMassArgs& args, int64_t grid, hipStream_t stream) {
  hipLaunchKernelGGL((latent_mass_kernel<kPass>), dim3((unsigned)grid), dim3(256), 0, stream, args);
  return hipGetLastError();
}

}  // namespace

// Scores are kept where this has both sides of it: a score costs 8 bytes of traffic, scoring a key again its 641 bytes and the products of
// its sequence's blocks. Batches of 32 rows a sequence or fewer (256 x 16 heads, 1000 to 8000 keys: 235 us kept, 366 scored again) keep up to 512 MB,
// those of up to 1024 what the MALL holds (us beside the attention, kept and scored again: 8 sequences x 3 tokens x 128 heads 60 and
// 70, 32 x 3 x 128 heads, 147 MB, 79 and 90, 8 x 8 x 128 heads, 131 MB, 68 and 83; above it 50 x 20 x 16 heads, 256 MB, 142 and 136, and 205 MB
// come out either way). With more rows the products of all blocks cost less than a last launch that takes a sequence's rows in turn
// (1 sequence of 2000 tokens, 1024 rows 34 and 32, 2048 rows 50 and 32). Rows are counted on average, as the host does not know the sequences' own; a
// long chunk among decoding sequences so has all its rows taken in turn: 63 sequences of 1024 tokens x 16 heads 47 us with the attention, 234 with a
// chunk of 256 tokens beside them and 738 with one of 1024, which by themselves take 68 and 106.
constexpr int64_t kMostScores = (int64_t)512 << 20, kMostOfMany = (int64_t)192 << 20;

LatentMassPlan plan_latent_mass(int64_t T, int64_t B, int64_t H, int64_t max_keys) {
  auto up = [](int64_t v) { return (size_t)((v + 255) / 256 * 256); };
  LatentMassPlan p{};
  const int64_t blocks = T * H / kRows + std::min(T, B), tiles = (max_keys + kTile - 1) / kTile;
  p.max_tiles = (int)tiles;
  // Tiles a part at least: 2, or 4 where sequences have more than 64 rows and the parts of 2 would fill the card (us beside the attention
  // with 2 and 4: 8 sequences of 4000 x 128 heads 29.0 and 26.2, 16 of 1000 to 4000 x 64 heads 25.0 and 27.5, 1 of 1111 x 128 heads 17.4
  // and 20.5).
  p.min_tiles = T * H <= 64 * B || blocks * tiles <= 512 ? 2 : 4;
  p.target_parts = 512;  // two workgroups on every compute unit (1024: 64 x 128 heads 94 us, 85 so, 6 chunks of 40 x 128 heads 185 and 181)
  const int64_t cut = std::min<int64_t>(blocks * std::max<int64_t>((tiles + p.min_tiles - 1) / p.min_tiles, 1), p.target_parts);
  p.ids = (std::max(blocks, cut) + 15) / 16 * 16;
  p.pitch = tiles * kTile;
  p.keeps_scores = T * H <= 8 * kRows * B && T * H <= (T * H <= 32 * B ? kMostScores : kMostOfMany) / 4 / std::max<int64_t>(p.pitch, 1);
  p.first_bytes = up(B * (int64_t)sizeof(int2));
  p.stats_bytes = up(p.ids * kRows * (int64_t)sizeof(float2));
  p.rest_bytes = up((p.keeps_scores ? T * H : T * H / kRows + B + 1) * p.pitch * (int64_t)sizeof(float));
  return p;
}

hipError_t launch_latent_mass(LatentMassArgs args, const LatentMassPlan& plan, hipStream_t stream) {
  LatentAttnArgs& a = args.work;
  hipError_t e = hipSuccess;
  if (a.T > 0) {
    e = plan.keeps_scores ? launch_pass<Pass::kScores>(args, plan.ids, stream) : launch_pass<Pass::kSums>(args, plan.ids, stream);
    if (e == hipSuccess && !plan.keeps_scores) e = launch_pass<Pass::kWeights>(args, plan.ids, stream);
  }
  if (e != hipSuccess || args.width < 1) return e;
  // Workgroups a sequence: one for its columns' every 128 or 256, but a page table may reach much further than its sequences do.
  const bool sum = a.T > 0 && plan.keeps_scores, more = sum && (int64_t)a.T * a.H > 32 * (int64_t)a.B;
  const int64_t columns = (args.width + sum_keys(more) - 1) / sum_keys(more);
  args.each = (int)std::min<int64_t>(columns, 8192 / a.B + 1);
  const dim3 grid((unsigned)(args.each * a.B));
  // (16 waves while every workgroup has a compute unit to itself: 8 sequences of 4000 tokens x 128 heads 2.6 us less than with 4, 16 x 64
  // heads in 512 workgroups 3.7 us more, 64 x 128 heads 28 us more)
  if (more && (int64_t)args.each * a.B <= 256) hipLaunchKernelGGL((latent_sum_kernel<16, 2>), grid, dim3(1024), 0, stream, args);
  else if (more) hipLaunchKernelGGL((latent_sum_kernel<4, 2>), grid, dim3(256), 0, stream, args);
  else if (sum) hipLaunchKernelGGL((latent_sum_kernel<4, 4>), grid, dim3(256), 0, stream, args);
  else hipLaunchKernelGGL(latent_blocks_kernel, grid, dim3(kSumKeys), 0, stream, args);
  return hipGetLastError();
}

}  // namespace bfp8
