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
// The products are formed transposed (S^T = K Q^T, O^T = V^T P^T): a lane holds the scores of one
// query row, r = lane % 16, for keys 16 t + 4 g + i (g = lane / 16), which is at once its operand
// of the second product; hi and lo fill the two halves of that product's 128 slots (the lo half
// under a scale of 2^-4), against the same 16 value bytes twice. Values are read from the key
// tile with transposing LDS reads.
//
// Work is cut on the device, where the lengths are: a block is up to 64 query rows (tokens x
// heads) of one sequence, and a block of more than `quantum` tiles of 64 keys is cut into parts
// whose float32 states (accumulator, maximum, sum) a second launch joins in order.
#include "device_common.h"
#include "latent.h"
#include "launch.h"

namespace bfp8 {

namespace {

constexpr int kTile = 64;                  // keys of a tile
constexpr int kBM = 64;                    // query rows of a block: 16 for each of 4 waves
constexpr int kSlack = 4;                  // the running maximum may lag by a factor of 2^kSlack ...
constexpr float kTop = 8 - kSlack;         // ... so that 2^(x - m + kTop) stays within 2^8 <= 448
constexpr float kNegInf = -__builtin_inff();

struct Desc {  // a block that was cut: rows row0 .. of the output, partial states slot .. slot + parts - 1
  int seq, block, slot, parts;
};

// XOR of the 16-byte columns of a key's 512-byte row in LDS. Conflict-free both for the score
// reads (16 lanes: one column of 16 consecutive keys) and for the transposing value reads (32
// lanes: one column of 16 keys that differ in bits 0, 1, 2 and 4).
__device__ __forceinline__ int swz(int key) { return (key & 7) | ((((key >> 3) ^ (key >> 4)) & 1) << 3); }

__device__ __forceinline__ v4f mfma_scaled(const v8i& a, const v8i& b, const v4f& c, int ea, int eb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, ea, 0, eb);
}

// Sequence b's chunk: rows (token, head) and how many keys its block `blk` sees.
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

__device__ __forceinline__ int blocks_of(const Seq& s, int H) { return (int)(((int64_t)s.n * H + kBM - 1) / kBM); }

__global__ __launch_bounds__(256, 2) void latent_attn_kernel(LatentAttnArgs a) {
  __shared__ __align__(1024) uint8_t tile[kTile * kLatentRow];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;

  // ---- which part is this workgroup's: every workgroup cuts the work in the same way
  int* sh = reinterpret_cast<int*>(tile);
  const int per = (a.B + 255) / 256;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  // total units (blocks x tiles) give the quantum
  auto tiles_of = [&](const Seq& s) { return min((s.len + kTile - 1) / kTile, a.max_tiles); };
  int64_t units = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(a, b);
    units += (int64_t)blocks_of(s, a.H) * tiles_of(s);
  }
#pragma unroll
  for (int mask = 1; mask < 64; mask <<= 1) units += __shfl_xor(units, mask);
  int64_t* sh64 = reinterpret_cast<int64_t*>(tile);
  if (lane == 0) sh64[wave] = units;
  __syncthreads();
  units = sh64[0] + sh64[1] + sh64[2] + sh64[3];
  const int quantum = (int)max((units + a.target_parts - 1) / a.target_parts, (int64_t)a.min_tiles);
  int parts = 0, slots = 0, cuts = 0;  // of this thread's sequences
  auto cut_of = [&](const Seq& s) { return max((tiles_of(s) + quantum - 1) / quantum, 1); };
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(a, b);
    const int c = cut_of(s), n = blocks_of(s, a.H);
    parts += n * c;
    if (c > 1) slots += n * c, cuts += n;
  }
  __syncthreads();
  // exclusive sums over the threads
  int p0 = parts, s0 = slots, c0 = cuts;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(p0, d), y = __shfl_up(s0, d), z = __shfl_up(c0, d);
    if (lane >= d) p0 += x, s0 += y, c0 += z;
  }
  if (lane == 63) sh[wave * 3] = p0, sh[wave * 3 + 1] = s0, sh[wave * 3 + 2] = c0;
  __syncthreads();
  int pt = 0, ct = 0;
  for (int w = 0; w < 4; ++w) {
    const int x = sh[w * 3], y = sh[w * 3 + 1], z = sh[w * 3 + 2];
    if (w < wave) p0 += x, s0 += y, c0 += z;
    pt += x;
    ct += z;
  }
  p0 -= parts, s0 -= slots, c0 -= cuts;
  if (blockIdx.x == 0 && tid == 0 && a.counts != nullptr) a.counts[0] = ct;
  __syncthreads();
  // workgroups of one XCD (blockIdx % 8) take consecutive parts, so blocks of a sequence share its L2
  const int per_xcd = (pt + 7) / 8;
  const int my = (int)(blockIdx.x & 7) * per_xcd + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || my >= pt) return;
  if (my >= p0 && my < p0 + parts) {
    for (int b = b0; b < b1; ++b) {
      const Seq s = sequence(a, b);
      const int c = cut_of(s), n = blocks_of(s, a.H);
      if (my < p0 + n * c) {
        const int blk = (my - p0) / c, part = (my - p0) - blk * c;
        sh[0] = b;
        sh[1] = blk;
        sh[2] = part;
        sh[3] = c;
        sh[4] = c > 1 ? s0 + blk * c + part : -1;
        if (c > 1 && part == 0 && c0 + blk < a.max_cuts) reinterpret_cast<Desc*>(a.counts + 4)[c0 + blk] = {b, blk, s0 + blk * c, c};
        break;
      }
      p0 += n * c;
      if (c > 1) s0 += n * c, c0 += n;
    }
  }
  __syncthreads();
  const int b = sh[0], blk = sh[1], part = sh[2], nparts = sh[3], slot = sh[4];
  __syncthreads();
  if (slot >= 0 && slot - part + nparts > a.max_slots) return;  // (starts that are not rising; nothing is promised for them)
  const Seq seq = sequence(a, b);
  const int rows = seq.n * a.H - blk * kBM;  // rows left in this block (may exceed kBM)

  // ---- this lane's query row
  const int row = wave * 16 + r;
  const bool row_ok = row < rows;
  const int flat = blk * kBM + row;
  const int tok = row_ok ? flat / a.H : 0, head = row_ok ? flat - tok * a.H : 0;
  const int64_t qtok = seq.q0 + tok;
  // keys the row sees: its sequence up to itself
  const int limit = row_ok ? min(max(seq.len - seq.n + tok + 1, 0), seq.len) : 0;
  // keys the block sees (its last row's), cut into nparts of whole tiles
  const int last_tok = (min(blk * kBM + kBM, seq.n * a.H) - 1) / a.H;
  const int keys = min(max(seq.len - seq.n + last_tok + 1, 0), seq.len);
  const int tiles = (keys + kTile - 1) / kTile;
  const int t_begin = (int)((int64_t)tiles * part / nparts), t_end = (int)((int64_t)tiles * (part + 1) / nparts);

  v8i q_hi[4], q_lo[4];
  v8bf q_rope[2];
  int q_code;
  {
    const uint16_t* src = a.q + qtok * a.q_tok + (int64_t)head * a.q_head;
    uint4 raw[4][4];
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // 8 values: the halves' first and second 16 bytes of codes
        raw[ks][j] = make_uint4(0, 0, 0, 0);
        if (row_ok) raw[ks][j] = *reinterpret_cast<const uint4*>(src + 128 * ks + 64 * (j >> 1) + 16 * g + 8 * (j & 1));
        float f[8];
        bf16x8_values(raw[ks][j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(f[i]));
      }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row_ok) v = *reinterpret_cast<const uint4*>(src + kLatentDim + 32 * ks + 8 * g);
      q_rope[ks] = __builtin_bit_cast(v8bf, v);
    }
    amax = max_nan(amax, __shfl_xor(amax, 16));
    amax = max_nan(amax, __shfl_xor(amax, 32));
    // the least power of two that holds the row in e4m3 range (kept away from the ends of float32)
    uint32_t code = (__float_as_uint(max_nan(amax, 0x1p-80f) / 448.0f) + 0x7fffffu) >> 23;
    const bool finite = amax < __builtin_inff();
    if (!finite) code = 127;
    const float inv = finite ? __uint_as_float((254u - code) << 23) : __builtin_nanf("");  // a NaN row scores NaN
    q_code = (int)code;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[8], back[8], lo[8];
        bf16x8_values(raw[ks][j], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inv;
        const uint2 hi = make_uint2(pack_e4m3(f), pack_e4m3(f + 4));
        e4m3x8_values(hi, back);
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = (f[i] - back[i]) * 16.f;
        q_hi[ks][2 * j] = (int)hi.x;
        q_hi[ks][2 * j + 1] = (int)hi.y;
        q_lo[ks][2 * j] = (int)pack_e4m3(lo);
        q_lo[ks][2 * j + 1] = (int)pack_e4m3(lo + 4);
      }
  }

  v4f acc[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  float m = kNegInf, l = 0.f;
  const float c = a.scale * 1.44269504088896341f;
  const uint32_t lds = lds_addr(tile);
  const int p_code = g < 2 ? 127 : 123;  // hi slots at 1, lo slots at 2^-4

  for (int t = t_begin; t < t_end; ++t) {
    const int k0 = t * kTile;
    // ---- lane L looks up key k0 + L (keys past the block's repeat its last: finite, and masked)
    const int key = min(k0 + lane, keys - 1);
    const int col = key / a.cache.page_size, off = key - col * a.cache.page_size;
    const int page = col < a.cache.table_width ? a.cache.table[(int64_t)b * a.cache.table_stride + col] : -1;
    const bool bad = page < 0 || page >= a.cache.pages;
    const uint32_t unit =
        bad ? 0u : (uint32_t)page * (uint32_t)(a.cache.page_stride / 128) + (uint32_t)off * (kLatentRow / 128);
    const int code = bad ? 255 : a.cache.scales[(int64_t)page * a.cache.scale_stride + off];
    // ---- the tile into LDS: 64 x 512 bytes of codes, then 64 x 128 bytes of rotary keys
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int kk = (wave * 8 + j) * 2 + (lane >> 5);
      const uint64_t u = (uint32_t)__shfl((int)unit, kk);
      copy16_from(a.cache.rows + u * 128 + (((lane & 31) ^ swz(kk)) << 4), lds + (wave * 8 + j) * 1024);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int kk = (wave * 2 + j) * 8 + (lane >> 3);
      const uint64_t u = (uint32_t)__shfl((int)unit, kk);
      copy16_from(a.cache.rows + u * 128 + kLatentDim + (((lane & 7) ^ lds_swizzle(kk)) << 4),
                  lds + kTile * kLatentDim + (wave * 2 + j) * 1024);
    }
    wait_copies();
    __syncthreads();

    // ---- scores of 4 x 16 keys
    v4f s[4];
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      const int kk = kt * 16 + r;
      const int kc = __shfl(code, kk);
      const uint8_t* base = tile + kk * kLatentDim;
      v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const v4i x = *reinterpret_cast<const v4i*>(base + (((ks * 8 + g) ^ swz(kk)) << 4));
        const v4i y = *reinterpret_cast<const v4i*>(base + (((ks * 8 + 4 + g) ^ swz(kk)) << 4));
        const v8i k = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        d = mfma_scaled(k, q_hi[ks], d, kc, q_code);
        d = mfma_scaled(k, q_lo[ks], d, kc, q_code - 4);
      }
      const uint8_t* rb = tile + kTile * kLatentDim + kk * 128;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const v8bf k = *reinterpret_cast<const v8bf*>(rb + (((ks * 4 + g) ^ lds_swizzle(kk)) << 4));
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q_rope[ks], d, 0, 0, 0);
      }
      s[kt] = d;
    }
    // ---- x = score in log2 + key exponent; weights relative to the running maximum
    int kcode[4][4];
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) kcode[kt][i] = __shfl(code, kt * 16 + 4 * g + i);
    float top = kNegInf;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x = fmaf(s[kt][i], c, (float)(kcode[kt][i] - 127));
        if (k0 + kt * 16 + 4 * g + i >= limit) x = kNegInf;
        s[kt][i] = x;
        top = fmaxf(top, x);
      }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > m + kSlack)) {
      const float next = fmaxf(m, top);
      const float f = m == next ? 1.f : __builtin_amdgcn_exp2f(m - next);  // (m = next = -inf: nothing yet)
      m = next;
      l *= f;
#pragma unroll
      for (int d = 0; d < 32; ++d) acc[d] *= f;
    }
    const float ref = m == kNegInf ? 0.f : m - kTop;
    v4i p_hi, p_lo;
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
      float p[4], back[4], rest[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = __builtin_amdgcn_exp2f(s[kt][i] - ref);
        // 2^-e; for the code of NaN a zero, so that a masked key (p = 0) adds nothing
        l += p[i] * __uint_as_float((uint32_t)(254 - min(kcode[kt][i], 254)) << 23);
      }
      const int h = (int)pack_e4m3(p);
      back[0] = __builtin_amdgcn_cvt_f32_fp8(h, 0);
      back[1] = __builtin_amdgcn_cvt_f32_fp8(h, 1);
      back[2] = __builtin_amdgcn_cvt_f32_fp8(h, 2);
      back[3] = __builtin_amdgcn_cvt_f32_fp8(h, 3);
#pragma unroll
      for (int i = 0; i < 4; ++i) rest[i] = (p[i] - back[i]) * 16.f;
      p_hi[kt] = h;
      p_lo[kt] = (int)pack_e4m3(rest);
    }
    const v8i pw = __builtin_shufflevector(p_hi, p_lo, 0, 1, 2, 3, 4, 5, 6, 7);
    // ---- O^T += V^T P^T, 16 value columns at a time
    const int vk = 16 * (r >> 3) + 4 * g + ((r >> 1) & 3);  // the row this lane addresses (and vk + 32)
#pragma unroll
    for (int d = 0; d < 32; ++d) {
      typedef __attribute__((address_space(3))) v2i lds_v2i;
      const uint8_t* at = tile + vk * kLatentDim + ((d ^ swz(vk)) << 4) + 8 * (r & 1);
      const v2i x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)at);
      const v2i y = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(at + 32 * kLatentDim));
      const v8i v = {x[0], x[1], y[0], y[1], x[0], x[1], y[0], y[1]};
      acc[d] = mfma_scaled(v, pw, acc[d], 127, p_code);
    }
    __syncthreads();
  }

  // ---- the row's sum over its four lanes, then the output or this part's state
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (!row_ok) return;
  if (slot < 0) {
    const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row that sees no key is zero
    uint16_t* dst = a.out + qtok * a.o_tok + (int64_t)head * a.o_head + 4 * g;
#pragma unroll
    for (int d = 0; d < 32; ++d)
      *reinterpret_cast<uint2*>(dst + 16 * d) =
          make_uint2(pack_bf16(acc[d][0] * inv, acc[d][1] * inv), pack_bf16(acc[d][2] * inv, acc[d][3] * inv));
  } else {
    float* dst = a.states + ((int64_t)slot * kBM + row) * kLatentDim + 4 * g;
#pragma unroll
    for (int d = 0; d < 32; ++d) *reinterpret_cast<v4f*>(dst + 16 * d) = acc[d];
    if (g == 0) {
      a.stats[((int64_t)slot * kBM + row) * 2] = m;
      a.stats[((int64_t)slot * kBM + row) * 2 + 1] = l;
    }
  }
}

// Joins the parts of a cut block, in order: one wave a row.
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

constexpr int kTargetParts = 512;  // two workgroups on each of 256 CUs
constexpr int kMinTiles = 2;       // fewer tiles a part cost more in states than they save

}  // namespace

LatentAttnPlan plan_latent_attn(int64_t T, int64_t B, int64_t H, int64_t max_keys) {
  LatentAttnPlan p;
  // Blocks: a sequence's last may be partly filled.
  p.blocks = T * H / kBM + (T < B ? T : B);
  const int64_t max_tiles = (max_keys + kTile - 1) / kTile;
  p.max_tiles = (int)max_tiles;
  p.target_parts = kTargetParts;
  p.min_tiles = kMinTiles;
  // A part has more than quantum / 2 tiles where a block is cut, and the quantum is at least
  // units / target: no more than 2 target + 2 blocks cut parts; and no more than a block's tiles allow.
  const int64_t per_block = (max_tiles + kMinTiles - 1) / kMinTiles;
  if (per_block <= 1) {
    p.slots = p.cuts = 0;
  } else {
    p.slots = 2 * kTargetParts;
    if (p.blocks * per_block < p.slots) p.slots = p.blocks * per_block;
    p.cuts = p.slots / 2;
  }
  p.parts = p.blocks + (p.slots > 0 ? kTargetParts : 0);
  p.counts_bytes = p.slots ? ((16 + p.cuts * sizeof(Desc) + 255) / 256) * 256 : 0;
  p.stats_bytes = ((p.slots * kBM * 2 * sizeof(float) + 255) / 256) * 256;
  p.states_bytes = p.slots * kBM * kLatentDim * sizeof(float);
  return p;
}

hipError_t launch_latent_attn(const LatentAttnArgs& args, const LatentAttnPlan& plan, hipStream_t stream) {
  const int64_t grid = (plan.parts + 7) / 8 * 8;
  hipLaunchKernelGGL(latent_attn_kernel, dim3((unsigned)grid), dim3(256), 0, stream, args);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.slots == 0) return e;
  hipLaunchKernelGGL(latent_join_kernel, dim3((unsigned)plan.cuts, kBM / 4), dim3(256), 0, stream, args);
  return hipGetLastError();
}

}  // namespace bfp8
