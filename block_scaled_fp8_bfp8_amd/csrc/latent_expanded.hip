// Latent attention in the expanded form: ragged causal attention whose keys and values were expanded
// from the latents by a GEMM (kv [Tk][H][256]: 128 key dimensions, then 128 value dimensions of a head)
// and whose keys end in a rotary part that all heads share (rope [Tk][64]).
//
//   o[t, h] = sum_j softmax_j(scale * (q[t, h, :128] . kv[j, h, :128] + q[t, h, 128:] . rope[j])) kv[j, h, 128:]
//
// over the keys j of t's sequence up to t (the last query token sees the last key).
//
// One pass with the running maximum and sum of the softmax. A workgroup takes 32 query rows of one head
// a wave and walks the keys in tiles of 64, copied straight to LDS a tile ahead. Both products are
// 32x32x16 matrix-core products, formed transposed (S^T = K Q^T, O^T = V^T P^T): a lane then holds
// scores of one query row, r = lane % 32, which are its operand of the second product without any
// exchange, and the running maximum and sum are plain per-lane numbers. V is read from the tile with
// transposing LDS reads.
//
// Bound by the matrix cores and by how well their time is shared: with 8 waves a workgroup (256 rows) two
// waves a SIMD, of which the second multiplies a tile's values one tile later, so that one wave's softmax
// runs beside the other's products. The LDS layout leaves the copies one lane offset for all of a tile's rows,
// and the reads two addresses each, with constant offsets for everything else. 4 prompts of 2100 to 4090 x 32 heads:
// 510 us, 1.0 PFLOP/s (matrix cores busy 46 % of the clocks).
#include "device_latent.h"
#include "latent.h"
#include "launch.h"

namespace bfp8 {

namespace {

constexpr int kTile = 64;    // keys of a tile
constexpr float kNegInf = -__builtin_inff();
// The running maximum may lag by a factor of 2^kSlack: weights stay within 2^8, far inside fp16 and
// bf16, and the accumulator is rescaled only when a tile exceeds that.
constexpr float kSlack = 8.f;

// A tile in LDS. Rows of kv are 512 bytes; a copy brings two, 2 keys apart, as a pair of 1024 + 16 bytes with the
// 16-byte columns of the second XORed with 8. Pair p holds keys 16 (p / 8) + 4 (p % 4) + p / 4 % 2 and that + 2:
// 16 consecutive keys then lie 16 different columns apart modulo 256 bytes (score reads: one column of 16 keys), and
// 4 consecutive ones 4 columns apart (transposing value reads: 64 bytes of 4 keys). The XOR changes bit 3 of a
// column alone. Rotary keys: groups of 8 rows of 128 bytes, 1024 + 64 bytes apart, columns XORed with (row / 2) % 4.
constexpr int kPairStride = 1024 + 16, kRopeStride = 1024 + 64;
constexpr int kRopeAt = kTile / 2 * kPairStride;
constexpr int kTileBytes = kRopeAt + kTile / 8 * kRopeStride;
constexpr int kBuffers = 3;
constexpr int kRing = 5;  // operands in registers

template <bool kF16>
__device__ __forceinline__ v16f mfma(const v4i& a, const v4i& b, const v16f& c) {
  if constexpr (kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kF16) return f32_to_f16_rne(lo) | (f32_to_f16_rne(hi) << 16);
  else return pack_bf16(lo, hi);
}

// Of two 16-bit values, those that are infinite or NaN: all ones in their place.
template <bool kF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t pair) {
  constexpr uint32_t kInf = kF16 ? 0x7c00u : 0x7f80u;
  return ((pair & 0x7fffu) >= kInf ? 0xffffu : 0u) | ((pair >> 16 & 0x7fffu) >= kInf ? 0xffff0000u : 0u);
}

// A wave's 32 rows again, for values that may be infinite or NaN, of which a weight of zero does not make nothing: the
// products leave them out, and each is added in the end to the rows that see it (any weight makes the same of it).
// Everything else has the bits of the first time, so the steps are the kernel's (which has them in place: calling one
// function for both cost it 6 % on 5 short prompts x 8 heads). Operands come from memory as they are needed: this is
// rare (4 prompts of 4000 x 32 heads: 0.7 ms; with a NaN at the first key of one 2.1, of all four 6.0).
template <bool kF16>
__device__ __forceinline__ void attend_not_finite(const uint16_t* q_row, bool row_ok, const uint8_t* kv, int64_t kv_step,
                                                  const uint8_t* rope, int64_t rope_step, int limit, int any, int flip,
                                                  float c, v16f* acc, float& l) {
  const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = kNegInf;
  l = 0.f;
#pragma unroll 1
  for (int t0 = 0; t0 < any; t0 += kTile) {
    v16f s[2];
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[kt][i] = 0.f;
#pragma unroll
    for (int n = 0; n < 24; ++n) {
      const int kt = n & 1, ks = n >> 1, key = min(t0 + 32 * kt + r, any - 1);
      const uint8_t* at = ks < 8 ? kv + key * kv_step + 32 * ks : rope + key * rope_step + 32 * (ks - 8);
      v4i q = {0, 0, 0, 0};
      if (row_ok) q = *reinterpret_cast<const v4i*>(q_row + 16 * ks + 8 * g) ^ v4i{flip, flip, flip, flip};
      s[kt] = mfma<kF16>(*reinterpret_cast<const v4i*>(at + 16 * g), q, s[kt]);
      __builtin_amdgcn_sched_barrier(0);
    }
    v4i p[4];
    const int left = limit - t0 - 4 * g;
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (kt * 32 + 8 * (i >> 2) + (i & 3) >= left) s[kt][i] = kNegInf;
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) top = fmaxf(top, s[i >> 4][i & 15]);
    const unsigned bits = __float_as_uint(top);
    const auto both = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
    top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * c;
    if (__any(top > m + kSlack)) {
      const float next = fmaxf(m, top);
      const float f = m == next ? 1.f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[d] *= f;
    }
    const float ref = m == kNegInf ? 0.f : m;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float x = __builtin_amdgcn_exp2f(fmaf(s[i >> 4][i & 15], c, -ref));
      s[i >> 4][i & 15] = x;
      sum[i & 1] += x;
    }
    l += sum[0] + sum[1];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      p[i >> 2][i & 3] = (int)pack16<kF16>(s[i >> 3][2 * (i & 7)], s[i >> 3][2 * (i & 7) + 1]);
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      const int u = n >> 2, d = n & 3;
      v4i v;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t pair = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = min(t0 + 16 * u + 8 * (w >> 1) + 4 * g + 2 * (w & 1) + e, any - 1);
          pair |= (uint32_t)*reinterpret_cast<const uint16_t*>(kv + key * kv_step + 256 + 2 * (32 * d + r)) << (16 * e);
        }
        v[w] = (int)(pair & ~not_finite<kF16>(pair));
      }
      acc[d] = mfma<kF16>(v, p[u], acc[d]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll 1
  for (int t0 = 0; t0 < any; t0 += 64) {
    // lane k: whether key t0 + k has such values
    const uint4* row = reinterpret_cast<const uint4*>(kv + min(t0 + lane, any - 1) * kv_step + 256);
    uint32_t bad = 0;
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
      const uint4 x = row[j];
      bad |= not_finite<kF16>(x.x) | not_finite<kF16>(x.y) | not_finite<kF16>(x.z) | not_finite<kF16>(x.w);
    }
#pragma unroll 1
    for (uint64_t which = __ballot(bad != 0 && t0 + lane < any); which != 0; which &= which - 1) {
      const int key = t0 + __builtin_ctzll(which);
      const bool seen = key < limit;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        v16f add;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {  // columns 32 d + 2 i + 4 g .. + 3
          const uint2 x = *reinterpret_cast<const uint2*>(kv + key * kv_step + 256 + 8 * g + 64 * d + 4 * i);
          const uint32_t y[2] = {x.x & not_finite<kF16>(x.x), x.y & not_finite<kF16>(x.y)};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t half = y[k >> 1] >> (16 * (k & 1)) & 0xffffu;
            add[i + k] = !seen ? 0.f : kF16 ? f16_value(half) : __uint_as_float(half << 16);
          }
        }
        acc[d] += add;
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

__device__ __forceinline__ int clip(int v, int top) { return min(max(v, 0), top); }

// The workgroup's block of kBM query rows: the sequences' blocks one after the other, of each the last, which has
// most keys, first; or all blocks with most keys first (counted in blocks; of equal ones the first sequence's), so
// that the last to start are short. False: there is none. Every wave looks for itself.
template <int kBM>
__device__ __forceinline__ bool find_block(const LatentExpandedArgs& a, int index, int& seq, int& block) {
  const int lane = threadIdx.x & 63;
  const int per = (a.B + 63) / 64;
  const int b0 = min(lane * per, a.B), b1 = min(b0 + per, a.B);
  auto blocks = [&](int b) { return (max(clip(a.cu_q[b + 1], a.Tq) - clip(a.cu_q[b], a.Tq), 0) + kBM - 1) / kBM; };
  if (a.longest_first) {
    // lane b: sequence b, whose blocks are at the levels top, top - 1, .. top - n + 1 (all at least 1)
    int n = 0, top = 0;
    if (lane < a.B) {
      const int nq = clip(a.cu_q[lane + 1], a.Tq) - clip(a.cu_q[lane], a.Tq);
      const int nk = max(clip(a.cu_k[lane + 1], a.Tk) - clip(a.cu_k[lane], a.Tk), 0);
      n = blocks(lane);
      top = n + max(nk - nq, 0) / kBM;
    }
    auto total = [](int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); };
    auto down_to = [&](int level) { return total(min(max(top - level + 1, 0), n)); };  // blocks at it and above
    if (index >= total(n)) return false;
    int lo = 1, hi = (int)wave_max((float)top) + 4;  // the highest level down to which there are more than `index`
    while (lo < hi) {
      const int mid = lo + ((hi - lo + 1) >> 1);
      if (down_to(mid) > index) lo = mid;
      else hi = mid - 1;
    }
    const int above = down_to(lo + 1);
    const uint64_t at = __ballot(lo <= top && lo > top - n);
    const bool me = (at >> lane & 1) && __popcll(at & ((1ull << lane) - 1)) == index - above;
    seq = __builtin_ctzll(__ballot(me));
    block = __builtin_amdgcn_readlane(n - 1 - (top - lo), seq);
    return true;
  }
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += blocks(b);
  int first = wave_scan(mine) - mine;
  const uint64_t who = __ballot(index >= first && index < first + mine);
  if (who == 0) return false;
  int s = 0, blk = 0;
  if (index >= first && index < first + mine) {
    for (int b = b0; b < b1; ++b) {
      const int n = blocks(b);
      if (index < first + n) {
        s = b;
        blk = n - 1 - (index - first);
        break;
      }
      first += n;
    }
  }
  seq = __builtin_amdgcn_readlane(s, __builtin_ctzll(who));
  block = __builtin_amdgcn_readlane(blk, __builtin_ctzll(who));
  return true;
}

template <bool kF16, int kWaves>
__global__ __launch_bounds__(kWaves * 64, kWaves / 4) void latent_expanded_kernel(LatentExpandedArgs a) {
  constexpr int kBM = kWaves * 32;
  __shared__ __align__(1024) uint8_t lds_tiles[kBuffers * kTileBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int head = blockIdx.x % a.H, index = blockIdx.x / a.H;
  int b, blk;
  if (!find_block<kBM>(a, index, b, blk)) return;
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const int q0 = uniform(clip(a.cu_q[b], a.Tq)), nq = uniform(clip(a.cu_q[b + 1], a.Tq)) - q0;
  const int k0 = uniform(clip(a.cu_k[b], a.Tk)), nk = max(uniform(clip(a.cu_k[b + 1], a.Tk)) - k0, 0);

  // ---- this lane's query row
  const int row = blk * kBM + wave * 32 + r;
  const bool row_ok = row < nq;
  const int limit = row_ok ? clip(nk - nq + row + 1, nk) : 0;  // keys it sees
  const int keys = clip(nk - nq + min(blk * kBM + kBM, nq), nk);  // keys the block sees
  const int tiles = (keys + kTile - 1) / kTile;
  // the wave's rows: keys that all of them see (tiles before need no mask), and that any of them sees
  const int w0 = blk * kBM + wave * 32;
  const int all = w0 + 32 <= nq ? clip(nk - nq + w0 + 1, nk) : 0;
  const int any = w0 < nq ? clip(nk - nq + min(w0 + 32, nq), nk) : 0;

  // ---- copies: this wave's share of a tile. In a full tile all rows of a copy lie one lane offset from a
  // uniform address; in the last tile keys past the block's repeat its last (masked).
  constexpr int kKvCopies = 32 / kWaves, kRopeCopies = 8 / kWaves;
  const uint8_t* kv = reinterpret_cast<const uint8_t*>(a.kv + (int64_t)k0 * a.kv_tok + (int64_t)head * a.kv_head);
  const uint8_t* rope = reinterpret_cast<const uint8_t*>(a.rope + (int64_t)k0 * a.ld_rope);
  const int64_t kv_step = a.kv_tok * 2, rope_step = a.ld_rope * 2;
  const bool near = kv_step < (1 << 28) && rope_step < (1 << 27);  // lane offsets fit 32 bits
  const uint32_t kv_col = ((lane & 31) ^ (g * 8)) << 4, rope_col = ((lane & 7) ^ ((lane >> 4) & 3)) << 4;
  const uint32_t kv_off = (uint32_t)(2 * g * kv_step) + kv_col, rope_off = (uint32_t)((lane >> 3) * rope_step) + rope_col;
  const uint32_t lds = lds_addr(lds_tiles);
  // first key of this wave's pairs and of its rotary groups
  const int kv_key = kWaves == 8 ? 16 * (wave >> 1) + (wave & 1) : 16 * wave, rope_key = wave * (64 / kWaves);
  const uint8_t* kv_next = kv + kv_key * kv_step;        // of the next tile to copy
  const uint8_t* rope_next = rope + rope_key * rope_step;
  auto copy_tile = [&](int t, uint32_t tile) {  // tiles in order
    const uint32_t kv_at = tile + wave * kKvCopies * kPairStride, rope_at = tile + kRopeAt + wave * kRopeCopies * kRopeStride;
    if (near && (t + 1) * kTile <= keys) {
      const uint8_t* src = kv_next;
#pragma unroll
      for (int j = 0; j < kKvCopies; ++j) {  // keys 0, 4, 8, 12 and, of 8 copies, 1, 5, 9, 13
        copy16_m0(src, kv_off, kv_at + j * kPairStride);
        src += j == 3 ? kv_step - 12 * kv_step : 4 * kv_step;
      }
#pragma unroll
      for (int j = 0; j < kRopeCopies; ++j) copy16_m0(rope_next + 8 * j * rope_step, rope_off, rope_at + j * kRopeStride);
    } else {
#pragma unroll
      for (int j = 0; j < kKvCopies; ++j) {
        const int key = t * kTile + kv_key + 4 * (j & 3) + (j >> 2) + 2 * g;
        copy16_m0(kv + min(key, keys - 1) * kv_step + kv_col, kv_at + j * kPairStride);
      }
#pragma unroll
      for (int j = 0; j < kRopeCopies; ++j) {
        const int key = t * kTile + rope_key + 8 * j + (lane >> 3);
        copy16_m0(rope + min(key, keys - 1) * rope_step + rope_col, rope_at + j * kRopeStride);
      }
    }
    kv_next += kTile * kv_step;
    rope_next += kTile * rope_step;
  };

  const uint16_t* qs = a.q + (int64_t)(q0 + (row_ok ? row : 0)) * a.q_tok + (int64_t)head * a.q_head;
  // a negative scale is the queries' sign, so that the largest score in log2 is that of the largest product; a
  // scale of zero is as good as zero (masked products are infinite)
  const int flip = a.scale < 0.f ? (int)0x80008000 : 0;
  const float c = fmaxf(fabsf(a.scale) * 1.44269504088896341f, 0x1p-120f);
  v4i q[12];
  v16f acc[4];
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.f;
  float m = kNegInf, l = 0.f;

  if (tiles > 0) {
#pragma unroll
    for (int ks = 0; ks < 12; ++ks) {
      q[ks] = v4i{0, 0, 0, 0};
      if (row_ok) q[ks] = *reinterpret_cast<const v4i*>(qs + 16 * ks + 8 * g);
    }
#pragma unroll
    for (int ks = 0; ks < 12; ++ks) q[ks] ^= v4i{flip, flip, flip, flip};
#pragma unroll
    for (int ks = 0; ks < 12; ++ks) asm volatile("" : "+v"(q[ks]));  // loaded before the copies are counted

    copy_tile(0, lds);

    // ---- LDS addresses within a tile
    typedef __attribute__((address_space(3))) const v4i lds_v4i;
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    auto row_at = [](int key) {  // of 16
      return (((key & 1) << 2) + ((key >> 2) & 3)) * kPairStride + ((key >> 1) & 1) * 512;
    };
    const int second = (r >> 1) & 1;
    const uint32_t key_base = (r >> 4) * 8 * kPairStride + row_at(r & 15) + (g << 4);
    const uint32_t key_low = key_base + 128 * second, key_high = key_base - 128 * second;  // steps 0 .. 3 and 4 .. 7
    const uint32_t rope_base = kRopeAt + (r >> 3) * kRopeStride + (r & 7) * 128;
    const uint32_t rope_even = rope_base + ((g ^ ((r >> 1) & 3)) << 4), rope_odd = rope_base + (((2 + g) ^ ((r >> 1) & 3)) << 4);
    const int vk = 4 * g + ((lane >> 2) & 3);  // the row this lane addresses (and 8 further on), of 16
    const uint32_t value_base = row_at(vk) + 256 + (((lane >> 4) & 1) << 5) + (((lane >> 1) & 1) << 4) + 8 * (lane & 1);
    const uint32_t value_low = value_base + 128 * ((vk >> 1) & 1), value_high = value_base - 128 * ((vk >> 1) & 1);  // d < 2, d >= 2

    // ---- O^T += V^T P^T: 16 keys a step, of which lane g holds 4 g + {0..3} and 8 + 4 g + {0..3}
    v4i p[4];
    auto values = [&](uint32_t tile) {
      auto value_at = [&](int n) {  // operand of product n
        const int u = n >> 2, d = n & 3;
        const uint32_t at = tile + (d < 2 ? value_low : value_high) + u * 8 * kPairStride + 64 * d;
        const v2i lo = __builtin_bit_cast(v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_v4s*>(at)));
        const v2i hi = __builtin_bit_cast(
            v2i, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_v4s*>(at + 2 * kPairStride)));
        return v4i{lo[0], lo[1], hi[0], hi[1]};
      };
      v4i v[kRing];  // operands are read kRing - 1 products ahead (and kept there: the compiler reads them late)
#pragma unroll
      for (int n = 0; n + 1 < kRing; ++n) v[n] = value_at(n);
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        if (n + kRing - 1 < 16) v[(n + kRing - 1) % kRing] = value_at(n + kRing - 1);
        __builtin_amdgcn_sched_barrier(0);
        acc[n & 3] = mfma<kF16>(v[n % kRing], p[n >> 2], acc[n & 3]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    const bool late = kWaves == 8 && wave >= 4;        // the second wave of its SIMD
    const int mine = (any + kTile - 1) / kTile;        // tiles of which a row of this wave sees a key
    uint32_t tile = lds, tile_before = lds;
    int place = 0;
    for (int t = 0; t < tiles; ++t) {
      wait_copies();
      lds_barrier();  // tile t is there for every wave, and all are done with tile t - 2
      place = place == kBuffers - 1 ? 0 : place + 1;
      const uint32_t next_tile = lds + place * kTileBytes, tile_at_hand = tile;
      if (t + 1 < tiles) copy_tile(t + 1, next_tile);
      if (late && t > 0 && t - 1 < mine) values(tile_before);
      tile_before = tile;
      tile = next_tile;
      if (t >= mine) continue;  // none of the wave's rows sees these keys
      const int t0 = t * kTile;

      // ---- scores of 2 x 32 keys: lane (r, g), register i: key 8 (i / 4) + 4 g + i % 4
      v16f s[2];
      {
        auto key_at = [&](int n) {  // operand of product n
          const int kt = n & 1, ks = n >> 1;
          return ks < 8 ? *reinterpret_cast<lds_v4i*>(tile_at_hand + (ks < 4 ? key_low : key_high) + kt * 16 * kPairStride + 32 * ks)
                        : *reinterpret_cast<lds_v4i*>(tile_at_hand + ((ks & 1) ? rope_odd : rope_even) + kt * 4 * kRopeStride +
                                                      64 * ((ks - 8) >> 1));
        };
        v4i k[kRing];
#pragma unroll
        for (int n = 0; n + 1 < kRing; ++n) k[n] = key_at(n);
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[kt][i] = 0.f;
#pragma unroll
        for (int n = 0; n < 24; ++n) {
          if (n + kRing - 1 < 24) k[(n + kRing - 1) % kRing] = key_at(n + kRing - 1);
          __builtin_amdgcn_sched_barrier(0);
          s[n & 1] = mfma<kF16>(k[n % kRing], q[n >> 1], s[n & 1]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (t0 + kTile > all) {
        const int left = limit - t0 - 4 * g;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (kt * 32 + 8 * (i >> 2) + (i & 3) >= left) s[kt][i] = kNegInf;
      }
      float top = s[0][0];
#pragma unroll
      for (int i = 1; i < 32; ++i) top = fmaxf(top, s[i >> 4][i & 15]);
      const unsigned bits = __float_as_uint(top);
      const auto both = __builtin_amdgcn_permlane32_swap(bits, bits, false, false);
      top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * c;
      if (__any(top > m + kSlack)) {
        const float next = fmaxf(m, top);
        const float f = m == next ? 1.f : __builtin_amdgcn_exp2f(m - next);
        m = next;
        l *= f;
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[d] *= f;
      }
      const float ref = m == kNegInf ? 0.f : m;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = __builtin_amdgcn_exp2f(fmaf(s[i >> 4][i & 15], c, -ref));
        s[i >> 4][i & 15] = x;
        sum[i & 1] += x;
      }
      l += sum[0] + sum[1];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        p[i >> 2][i & 3] = (int)pack16<kF16>(s[i >> 3][2 * (i & 7)], s[i >> 3][2 * (i & 7) + 1]);
      if (!late) values(tile_at_hand);
    }
    if (late && tiles - 1 < mine) values(tile_before);
  }

  // Values that are not finite make an output not finite, that of a row that does not see them included (0.1 us of 12
  // to find out).
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 64; i += 2)
    top[(i >> 1) & 3] = max_nan(max_nan(top[(i >> 1) & 3], fabsf(acc[i >> 4][i & 15])), fabsf(acc[i >> 4][(i & 15) + 1]));
  const float largest = max_nan(max_nan(top[0], top[1]), max_nan(top[2], top[3]));
  if (__builtin_expect(__any(!(largest < __builtin_inff())), 0))
    attend_not_finite<kF16>(qs, row_ok, kv, kv_step, rope, rope_step, limit, any, flip, c, acc, l);

  l += __shfl_xor(l, 32);
  if (!row_ok) return;
  const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row that sees no key is zero
  uint16_t* dst = a.out + (int64_t)(q0 + row) * a.o_tok + (int64_t)head * a.o_head + 16 * g;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    // lanes g = 0 and 1 of a row swap quads of columns, so that each stores 16 neighbouring ones
    uint32_t u[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto v = __builtin_amdgcn_permlane32_swap(
            pack16<kF16>(acc[d][4 * h + 2 * i] * inv, acc[d][4 * h + 2 * i + 1] * inv),
            pack16<kF16>(acc[d][8 + 4 * h + 2 * i] * inv, acc[d][8 + 4 * h + 2 * i + 1] * inv), false, false);
        u[h][i] = v[0];
        u[h][2 + i] = v[1];
      }
    uint4* p = reinterpret_cast<uint4*>(dst + 32 * d);
    p[0] = make_uint4(u[0][0], u[0][1], u[0][2], u[0][3]);
    p[1] = make_uint4(u[1][0], u[1][1], u[1][2], u[1][3]);
  }
}

// The longest blocks first where a compute unit gets no more than about six (4 prompts of 2048 x 16 heads: 132 us in
// the given order, 105 so; 32 of 50 to 1000 x 16, 1552 workgroups: 145 and 130). Beyond, the tail is short, and the
// given order is the faster one (4 of 2100 to 4090 x 32, 1664 workgroups: 602 and 619; 16 of 100 to 4000 x 32: 1145 and
// 1262), it is thought because blocks of one sequence run together and share its keys in the L2s: the limit stands
// between these sizes, the cause was not measured by itself. Where all have a compute unit of their own the search is
// 0.4 us for nothing (5 of 17 to 300 x 8: 11.9 and 12.3). A wave looks among 64 sequences.
constexpr int64_t kLongestFirst = 1600;

template <bool kF16, int kWaves>
void launch(LatentExpandedArgs args, hipStream_t stream) {
  const int64_t grid = (args.Tq / (kWaves * 32) + (args.Tq < args.B ? args.Tq : args.B)) * (int64_t)args.H;
  args.longest_first = grid > 256 && grid <= kLongestFirst && args.B <= 64;
  hipLaunchKernelGGL((latent_expanded_kernel<kF16, kWaves>), dim3((unsigned)grid), dim3(kWaves * 64), 0, stream, args);
}

}  // namespace

int64_t latent_expanded_blocks(int64_t Tq, int64_t B) { return Tq / 128 + (Tq < B ? Tq : B); }

hipError_t launch_latent_expanded(const LatentExpandedArgs& args, bool f16, hipStream_t stream) {
  // 256 rows a workgroup where that more than fills the card and the sequences are long enough on average (128 and
  // 256 rows: 1 prompt of 4096 x 16 heads, 256 workgroups of 256 rows, 117 and 139 us; x 20 heads 157 and 146; 64 of
  // 180 to 200 x 16 74 and 58)
  const bool many = (int64_t)args.Tq * args.H > 256 * 256 && args.Tq > 128 * (int64_t)args.B;
  if (f16) many ? launch<true, 8>(args, stream) : launch<true, 4>(args, stream);
  else many ? launch<false, 8>(args, stream) : launch<false, 4>(args, stream);
  return hipGetLastError();
}

}  // namespace bfp8
