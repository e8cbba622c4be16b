// Accumulated attention weights of the tokens in the paged FP8 latent cache:
//   mass[b, j] += sum over new tokens t and heads h of softmax_j(scale q[t, h] . [c_j, r_j])
//
// A weight needs its row's maximum and sum over all keys first, so keys are scored twice: a first launch leaves each
// row's maximum and sum over every block of 128 keys, a second joins them, and a third forms the weights and adds them
// up over the rows. Scores are bf16 products on the cached codes, which bf16 holds exactly (32x32x16 instructions,
// latents and rotary part in accumulators of their own, as the key's scale belongs to the first alone), so a weight is
// off by float32 roundings only: the sums of thousands of weights stay good to 1e-5 or better.
//
// A wave holds 32 keys in registers and walks the query rows of their sequence in tiles of 32, which the waves of a
// workgroup share through LDS (9 blocks of 128 bytes a row, columns XORed by the row: no bank conflicts). One
// instruction serves both directions: with the keys as its second operand a lane holds one key and 16 rows, so that
// their weights add up in registers (no atomics: one wave owns a key); with the keys first a lane holds one row and 16
// keys, whose maximum and sum are as near.
#include <algorithm>

#include "device_latent.h"
#include "latent.h"
#include "launch.h"

namespace bfp8 {

namespace {

constexpr int kKeys = 128;                 // of a workgroup: 4 groups of 32
constexpr int kRowsTile = 32;
constexpr int kTileBytes = 9 * kRowsTile * 128;
constexpr float kNegInf = -__builtin_inff();

// The row that a key without a page stands on.
__device__ const uint4 kNoRow[kLatentRow / 16] = {};

// Sequence b: its new tokens, its length, and how many of its keys the page table reaches (a row that sees one past
// that is NaN).
struct Seq {
  int q0, n, len, reach;
};
__device__ __forceinline__ Seq sequence(const LatentMassArgs& a, int b) {
  Seq s{b, 1, 0, 0};
  if (a.cu_q != nullptr) {
    s.q0 = min(max(a.cu_q[b], 0), a.T);
    s.n = max(min(max(a.cu_q[b + 1], 0), a.T) - s.q0, 0);
  }
  s.len = max(a.lens[b], 0);
  s.reach = min(s.len, a.cache.table_width * a.cache.page_size);  // (below 2^31)
  return s;
}
// The keys that token `tok` of its new ones sees.
__device__ __forceinline__ int sees(const Seq& s, int tok) { return min(max(s.len - s.n + tok + 1, 0), s.len); }

// 8 codes as bf16, exactly.
__device__ __forceinline__ v8bf codes_bf16(uint32_t lo, uint32_t hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf x[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true),
                     __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true)};
  return v8bf{x[0][0], x[0][1], x[1][0], x[1][1], x[2][0], x[2][1], x[3][0], x[3][1]};
}

// kHalves groups of 4 waves take the tiles of rows in turn. kMass: weights (the third launch), else maxima and sums.
template <int kHalves, bool kMass>
__global__ __launch_bounds__(kHalves * 256, 2) void latent_mass_kernel(LatentMassArgs a) {
  constexpr int kBuffers = 2;
  __shared__ __attribute__((aligned(1024))) uint8_t tiles_lds[kHalves][kBuffers][kTileBytes];
  __shared__ float2 found[2][kHalves][4][kRowsTile];                  // maxima and sums of a tile, by group of keys
  __shared__ __attribute__((aligned(16))) float row_lse[2][kHalves][kRowsTile];
  __shared__ __attribute__((aligned(16))) int row_limit[2][kHalves][kRowsTile];
  __shared__ float sums[kHalves][kKeys];

  const int b = (int)(blockIdx.x / (unsigned)a.each), first_block = (int)(blockIdx.x - (unsigned)b * a.each);
  const Seq seq = sequence(a, b);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave & 3, half = wave >> 2;
  const int r = lane & 31, g = lane >> 5;
  const int64_t rows = (int64_t)seq.n * a.H;
  const int tiles = (int)((rows + kRowsTile - 1) / kRowsTile), rounds = (tiles + kHalves - 1) / kHalves;
  const float c = a.scale * 1.44269504088896341f;
  const int64_t all_rows = (int64_t)a.T * a.H, row0 = (int64_t)seq.q0 * a.H;

  // copies of a tile: group w brings rows 8 w .. 8 w + 7, lanes 8 i .. 8 i + 7 row i
  const int copy_row = group * 8 + (lane >> 3);
  const int copy_col = ((lane & 7) ^ lds_swizzle(copy_row)) * 16;
  auto copy_tile = [&](int t, int buffer) {
    const int64_t flat = min((int64_t)t * kRowsTile + copy_row, rows - 1);  // (past the last row: it again)
    const int tok = (int)(flat / a.H), head = (int)(flat - (int64_t)tok * a.H);
    const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q + (int64_t)(seq.q0 + tok) * a.q_tok + (int64_t)head * a.q_head) + copy_col;
    const uint32_t dst = lds_addr(&tiles_lds[half][buffer][group * 1024]);
#pragma unroll
    for (int i = 0; i < 9; ++i) copy16_m0(src + i * 128, __builtin_amdgcn_readfirstlane(dst + i * kRowsTile * 128));
  };
  const int sw = lds_swizzle(r);
  auto row_piece = [&](const uint8_t* tile, int column) {  // 16 bytes of row r
    return __builtin_bit_cast(v8bf, *reinterpret_cast<const v4i*>(tile + (column >> 3) * kRowsTile * 128 + r * 128 + (((column & 7) ^ sw) << 4)));
  };

  for (int kb = first_block; kb < (kMass ? (a.width + kKeys - 1) / kKeys : (seq.reach + kKeys - 1) / kKeys); kb += a.each) {
    const int key0 = kb * kKeys, key = key0 + group * 32 + r;
    const bool any = key0 < seq.reach && rows > 0;  // (the same in the whole workgroup)
    float total = 0.f;
    if (any) {
      copy_tile(min(half, tiles - 1), 0);
      // ---- the keys
      const int col = key / a.cache.page_size, off = key - col * a.cache.page_size;
      const int page = key < seq.reach ? a.cache.table[(int64_t)b * a.cache.table_stride + col] : -1;
      const bool none = page < 0 || page >= a.cache.pages;
      const uint8_t* src = none ? reinterpret_cast<const uint8_t*>(kNoRow)
                                : a.cache.rows + (int64_t)page * a.cache.page_stride + (int64_t)off * kLatentRow;
      uint4 codes[16];
      v8bf rope[4];
#pragma unroll
      for (int s = 0; s < 16; ++s) codes[s] = *reinterpret_cast<const uint4*>(src + (2 * s + g) * 16);
#pragma unroll
      for (int s = 0; s < 4; ++s) rope[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4i*>(src + kLatentDim + (2 * s + g) * 16));
      const float unit = (none ? __builtin_nanf("") : e8_value(a.cache.scales[(int64_t)page * a.cache.scale_stride + off])) * c;
      v8bf keys[32];
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        keys[2 * s] = codes_bf16(codes[s].x, codes[s].y);
        keys[2 * s + 1] = codes_bf16(codes[s].z, codes[s].w);
      }
      float units[kMass ? 1 : 16];  // of the lane's key, or of its 16 keys
      if constexpr (kMass) units[0] = unit;
      else
#pragma unroll
        for (int i = 0; i < 16; ++i) units[i] = __shfl(unit, 8 * (i >> 2) + 4 * g + (i & 3));

      for (int round = 0; round < rounds; ++round) {
        const int t = round * kHalves + half, turn = round & 1;
        const bool real = t < tiles;
        // ---- this tile's rows: what they see, and (kMass) the log2 of their sums
        const int64_t flat = (int64_t)t * kRowsTile + r;
        const int tok = (int)(min(flat, rows - 1) / a.H);
        const int limit = flat < rows ? sees(seq, tok) : 0;
        if constexpr (kMass) {
          if (group == 0 && g == 0) {
            row_limit[turn][half][r] = limit;
            row_lse[turn][half][r] = flat < rows ? a.lse[row0 + flat] : __builtin_inff();
          }
        }
        wait_copies();
        lds_barrier();
        if (round + 1 < rounds) copy_tile(min(t + kHalves, tiles - 1), turn ^ 1);
        if constexpr (!kMass) {
          // the tile before: its groups' maxima and sums as one
          if (round > 0 && group == 0 && g == 0 && t - kHalves < tiles) {
            const int64_t before = flat - kHalves * kRowsTile;
            if (before < rows) {
              float m = kNegInf, l = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) m = fmaxf(m, found[turn ^ 1][half][i][r].x);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = found[turn ^ 1][half][i][r];
                l += f.x == kNegInf ? f.y : f.y * __builtin_amdgcn_exp2f(f.x - m);
              }
              a.parts[(int64_t)kb * all_rows + row0 + before] = make_float2(m, l);
            }
          }
        }
        if (!real) continue;
        const uint8_t* tile = &tiles_lds[half][turn][0];
        v16f lat, rot;
#pragma unroll
        for (int i = 0; i < 16; ++i) lat[i] = rot[i] = 0.f;
#pragma unroll
        for (int s = 0; s < 32; ++s) {
          // key piece s: codes 16 (2 (s / 2) + g) + 8 (s % 2) .. + 7
          const v8bf x = row_piece(tile, 4 * (s >> 1) + 2 * g + (s & 1));
          lat = kMass ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, keys[s], lat, 0, 0, 0)
                      : __builtin_amdgcn_mfma_f32_32x32x16_bf16(keys[s], x, lat, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const v8bf x = row_piece(tile, 64 + 2 * s + g);
          rot = kMass ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, rope[s], rot, 0, 0, 0)
                      : __builtin_amdgcn_mfma_f32_32x32x16_bf16(rope[s], x, rot, 0, 0, 0);
        }
        if constexpr (kMass) {
          // rows 8 (i / 4) + 4 g + i % 4 of the lane's key
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const v4f lse = *reinterpret_cast<const v4f*>(&row_lse[turn][half][8 * i4 + 4 * g]);
            const v4i lim = *reinterpret_cast<const v4i*>(&row_limit[turn][half][8 * i4 + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = fmaf(lat[4 * i4 + i], units[0], fmaf(rot[4 * i4 + i], c, -lse[i]));
              const float p = __builtin_amdgcn_exp2f(x);
              total += key < lim[i] ? p : 0.f;
            }
          }
        } else {
          float x[16], m = kNegInf, l = 0.f;
          const int left = limit - (key0 + group * 32 + 4 * g);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            x[i] = fmaf(lat[i], units[i], rot[i] * c);
            if (8 * (i >> 2) + (i & 3) >= left) x[i] = kNegInf;
            m = fmaxf(m, x[i]);
          }
          m = fmaxf(m, __shfl_xor(m, 32));
          const float ref = m == kNegInf ? 0.f : m;
#pragma unroll
          for (int i = 0; i < 16; ++i) l += __builtin_amdgcn_exp2f(x[i] - ref);
          l += __shfl_xor(l, 32);
          if (g == 0) found[turn][half][group][r] = make_float2(m, l);
        }
      }
      if constexpr (!kMass) {
        lds_barrier();
        const int64_t flat = (int64_t)((rounds - 1) * kHalves + half) * kRowsTile + r;
        if (group == 0 && g == 0 && flat < rows) {
          const int turn = (rounds - 1) & 1;
          float m = kNegInf, l = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) m = fmaxf(m, found[turn][half][i][r].x);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = found[turn][half][i][r];
            l += f.x == kNegInf ? f.y : f.y * __builtin_amdgcn_exp2f(f.x - m);
          }
          a.parts[(int64_t)kb * all_rows + row0 + flat] = make_float2(m, l);
        }
      }
      lds_barrier();  // the tiles and the lists are free for the next block of keys
    }
    if constexpr (kMass) {
      total += __shfl_xor(total, 32);
      if (g == 0) sums[half][group * 32 + r] = total;
      lds_barrier();
      if (half == 0 && g == 0 && key < a.width) {
#pragma unroll
        for (int h = 1; h < kHalves; ++h) total += sums[h][group * 32 + r];
        // tokens that are new in this call start at zero; past the sequence there are none
        const float before = a.mass_in != nullptr && key < seq.len - seq.n ? a.mass_in[(int64_t)b * a.in_stride + key] : 0.f;
        a.mass[(int64_t)b * a.out_stride + key] = key < seq.reach ? before + total : 0.f;
      }
      lds_barrier();
    }
  }
}

// The log2 of each row's sum over all its keys.
__global__ __launch_bounds__(256) void latent_lse_kernel(LatentMassArgs a) {
  const int b = (int)(blockIdx.x / (unsigned)a.each), first = (int)(blockIdx.x - (unsigned)b * a.each);
  const Seq seq = sequence(a, b);
  const int64_t rows = (int64_t)seq.n * a.H, all_rows = (int64_t)a.T * a.H, row0 = (int64_t)seq.q0 * a.H;
  const int blocks = (seq.reach + kKeys - 1) / kKeys;
  for (int64_t row = (int64_t)first * 256 + threadIdx.x; row < rows; row += (int64_t)a.each * 256) {
    const float2* p = a.parts + row0 + row;
    float m = kNegInf, l = 0.f;
    for (int i = 0; i < blocks; ++i) {
      const float2 f = p[(int64_t)i * all_rows];
      const float top = fmaxf(m, f.x);
      if (top == kNegInf) {
        l += f.y;  // (no key seen so far, or NaN)
      } else {
        l = l * __builtin_amdgcn_exp2f(m - top) + f.y * __builtin_amdgcn_exp2f(f.x - top);
        m = top;
      }
    }
    if (sees(seq, (int)(row / a.H)) > seq.reach) l = __builtin_nanf("");
    a.lse[row0 + row] = l == 0.f ? __builtin_inff() : m + __builtin_amdgcn_logf(l);  // (logf: base 2)
  }
}

template <int kHalves>
hipError_t launch(LatentMassArgs a, hipStream_t stream) {
  // Workgroups a sequence: one a block of keys, but a page table may reach much further than its sequences do.
  const int64_t most = 8192 / a.B + 1;
  auto each = [&](int64_t n) { return (int)std::max<int64_t>(std::min(n, most), 1); };
  const int64_t reach = (int64_t)a.cache.table_width * a.cache.page_size;
  if (reach > 0) {
    a.each = each((reach + kKeys - 1) / kKeys);
    hipLaunchKernelGGL((latent_mass_kernel<kHalves, false>), dim3((unsigned)(a.each * a.B)), dim3(kHalves * 256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  a.each = each(((int64_t)a.T * a.H / a.B + 255) / 256);
  hipLaunchKernelGGL(latent_lse_kernel, dim3((unsigned)(a.each * a.B)), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.width < 1) return e;
  a.each = each((a.width + kKeys - 1) / kKeys);
  hipLaunchKernelGGL((latent_mass_kernel<kHalves, true>), dim3((unsigned)(a.each * a.B)), dim3(kHalves * 256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

LatentMassPlan plan_latent_mass(int64_t T, int64_t H, int64_t max_keys) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  return {up((size_t)((max_keys + kKeys - 1) / kKeys) * (size_t)(T * H) * sizeof(float2)), up((size_t)(T * H) * sizeof(float))};
}

hipError_t launch_latent_mass(const LatentMassArgs& a, hipStream_t stream) {
  return (int64_t)a.T * a.H <= (int64_t)a.B * kRowsTile ? launch<1>(a, stream) : launch<2>(a, stream);
}

}  // namespace bfp8
