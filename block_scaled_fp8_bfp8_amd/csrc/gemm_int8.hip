// Product of 8-bit integers with a scale for each token and each channel:
//   C[m, n] = round16((sum_k A[m, k] B[n, k]) As[m] Bs[n] + bias[n])
// The sum runs in 32-bit integers on the matrix cores and is exact (K <= 65536), so its order does not matter; it is
// converted to float32 (an error of 2^-24 at most), scaled and biased there, and rounded once to bf16 or fp16.
//
// As the scales are those of whole rows, nothing but the product happens along K. Both kernels form C^T = B A^T
// (weight rows on the matrix instruction's first operand, so that a lane's results are neighbours in a row of C), and
// copy operands to LDS in pieces of 8 rows x 128 bytes, whose 16-byte columns are XORed by the row (lds_swizzle), so
// that fragment reads are free of bank conflicts. Rows past M or N repeat the last one and are not stored. Where the
// last 128-byte block holds fewer bytes, its missing pieces are read from its first one (nothing past K is touched) and
// cleared in the activations' fragments: an integer product with zero is zero whatever stands on the other side.
//   * K-split (few rows; reading the weights is the work): the 8 waves of a workgroup take the K blocks of a small
//     tile in turn, each from slots of its own, and add their sums through LDS.
//   * tiled: a workgroup's waves share stages of a K block, two to four of them, with one barrier a block.
//
// Measured (cold weights): 8192 x 10240 x 5120 345 us, 2.49 * 10^15 operations a second, bound by power (with operands of zeros, which
// switch nothing, 280 us; the library's product of the same operands 430); 1000 x 4096 x 4096 21 us, bound by the copies into LDS (256
// workgroups, one round); 1 x 4096 x 4096 5.9 us and 5 x 5120 x 8192 12.1 (3.5 TB/s), bound by reading the weights once, start-up
// included; 83 x 576 x 7168 6.6 us, 216 workgroups whose waves take 7 of the 56 K blocks each, two of them in flight: about four memory
// latencies one after another.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device_int8.h"
#include "int8.h"
#include "launch.h"

namespace bfp8 {

namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

// One output: the sum times the scales, plus the bias, as 16 bits.
template <bool kF16>
__device__ __forceinline__ float bias_value(uint16_t b) {
  if constexpr (kF16) return f16_value(b);
  else return __uint_as_float((uint32_t)b << 16);
}
template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kF16) return f32_to_f16_rne(lo) | f32_to_f16_rne(hi) << 16;
  else return pack_bf16(lo, hi);
}

// An output is fl(sum * token's scale) * channel's scale + bias. The sum (2^30 at most) times the scale of a token whose largest element
// passes 2^104 or so may pass float32 though the channel's brings the output back: such a token's outputs are formed 2^32 times smaller first.
__device__ __forceinline__ bool scale_is_far(float ms) { return fabsf(ms) >= 0x1p97f; }
// Four of a row's outputs, packed. In fp16 the compiler makes the sum with the bias and the rounding one instruction; where a branch formed
// both kinds before a common rounding it would not, and the last bit would go by the kernel: so each kind is packed where it is formed.
template <bool kF16>
__device__ __forceinline__ uint2 outputs4(const int* sum, float ms, const float* ns, const float* add) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = fmaf((float)sum[e] * ms, ns[e], add[e]);
  return make_uint2(pack16<kF16>(y[0], y[1]), pack16<kF16>(y[2], y[3]));
}
template <bool kF16>
__device__ __forceinline__ uint2 far_outputs4(const int* sum, float ms, const float* ns, const float* add) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = fmaf((float)sum[e] * (ms * 0x1p-32f) * ns[e], 0x1p32f, add[e]);
    asm volatile("" : "+v"(y[e]));
  }
  uint2 p = make_uint2(pack16<kF16>(y[0], y[1]), pack16<kF16>(y[2], y[3]));
  asm volatile("" : "+v"(p.x), "+v"(p.y));
  return p;
}

// 4 neighbouring outputs n .. n + 3 of a row.
__device__ __forceinline__ void store4(uint16_t* c, int n, int N, bool vec_ok, uint32_t p0, uint32_t p1) {
  if (vec_ok && n + 3 < N) {
    *reinterpret_cast<uint2*>(c) = make_uint2(p0, p1);
  } else {
    if (n < N) c[0] = (uint16_t)p0;
    if (n + 1 < N) c[1] = (uint16_t)(p0 >> 16);
    if (n + 2 < N) c[2] = (uint16_t)p1;
    if (n + 3 < N) c[3] = (uint16_t)(p1 >> 16);
  }
}

// Clears the pieces of a fragment past K: `piece` is its 16-byte column in a block that has `bytes` of them.
__device__ __forceinline__ v4i keep_valid(v4i f, int piece, int bytes) {
  const bool in = 16 * piece < bytes;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = in ? f[i] : 0;
  return f;
}

constexpr int kWaves = 8;
constexpr int kFusedCodes = 16384;  // codes of all tokens that the linear layer's small-batch kernel holds (two workgroups on a compute unit)

// ---------------------------------------------------------------- few rows: the waves split K

// A workgroup's tile is BN = 16 TN weight rows x BM = 16 TM activation rows.
template <int TN, int TM, int SLOTS, bool kF16>
__global__ __launch_bounds__(kWaves * 64) void gemm_int8_ksplit_kernel(Int8GemmArgs args) {
  constexpr int BN = 16 * TN, BM = 16 * TM;
  constexpr int kPieces = (BN + BM) / 8;
  constexpr int kSlot = (BN + BM) * kBlock;
  static_assert(BN * BM * 4 <= SLOTS * kSlot, "the sums of a wave fit its slots");
  static_assert((SLOTS - 1) * kPieces < 64, "copies in flight that a wait can count");
  __shared__ __attribute__((aligned(1024))) uint8_t slots[kWaves][SLOTS][kSlot];

  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kc = lane >> 4;
  const int n0 = blockIdx.x * BN, m0 = blockIdx.y * BM;
  const int M = args.M, N = args.N;
  const int KB = (args.K + kBlock - 1) / kBlock;
  const int last_bytes = args.K - (KB - 1) * kBlock;
  const int nkb = KB > w ? (KB - w + kWaves - 1) / kWaves : 0;  // this wave's blocks: w + 8 i

  // piece j: rows 8 j .. 8 j + 7 of the tile, lane l at row 8 j + l / 8, physical column l % 8
  uint32_t off[kPieces];
  const int8_t* bmat = args.b + (int64_t)n0 * args.ldb;
  const int8_t* amat = args.a + (int64_t)m0 * args.lda;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int row = j * 8 + (lane >> 3);
    const int col = (lane & 7) ^ lds_swizzle(row);
    off[j] = (j * 8 < BN ? (uint32_t)min(row, N - 1 - n0) * (uint32_t)args.ldb
                         : (uint32_t)min(row - BN, M - 1 - m0) * (uint32_t)args.lda) + (uint32_t)(col * 16);
  }
  auto issue = [&](int slot, int kb) __attribute__((always_inline)) {
    const uint32_t dst = lds_addr(&slots[w][slot][0]);
    const bool part = kb == KB - 1 && last_bytes < kBlock;  // uniform
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int col = (lane & 7) ^ lds_swizzle(j * 8 + (lane >> 3));
      const uint32_t o = part && 16 * col >= last_bytes ? off[j] - (uint32_t)(col * 16) : off[j];
      copy16_m0((j * 8 < BN ? bmat : amat) + (int64_t)kb * kBlock, o, dst + (uint32_t)(j * 1024));
    }
  };
  const int sw = lds_swizzle(r);
  const uint32_t at_lo = (uint32_t)(r * kBlock + (((2 * kc) ^ sw) << 4)), at_hi = (uint32_t)(r * kBlock + (((2 * kc + 1) ^ sw) << 4));

  v4i acc[TN][TM];
#pragma unroll
  for (int tn = 0; tn < TN; ++tn)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) acc[tn][tm] = v4i{0, 0, 0, 0};

  // workgroups with the same weight rows start at different blocks: one fetches a block from HBM, the others find
  // it in L2
  const int rot = nkb > 0 ? (int)((int64_t)blockIdx.y * nkb / gridDim.y) : 0;
  auto block_of = [&](int i) __attribute__((always_inline)) { return w + (i + rot < nkb ? i + rot : i + rot - nkb) * kWaves; };
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
    if (s < nkb) issue(s, block_of(s));
  int slot = 0;
  for (int i = 0; i < nkb; ++i) {
    const int kb = block_of(i);
    if (i + SLOTS - 1 < nkb) wait_copies_upto<(SLOTS - 1) * kPieces>();
    else wait_copies();
    const uint8_t* sl = &slots[w][slot][0];
    const bool part = kb == KB - 1 && last_bytes < kBlock;
    v4i fb[TN][2], fa[TM][2];
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      fb[tn][0] = *reinterpret_cast<const v4i*>(sl + at_lo + tn * 16 * kBlock);
      fb[tn][1] = *reinterpret_cast<const v4i*>(sl + at_hi + tn * 16 * kBlock);
    }
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      fa[tm][0] = *reinterpret_cast<const v4i*>(sl + at_lo + (BN + tm * 16) * kBlock);
      fa[tm][1] = *reinterpret_cast<const v4i*>(sl + at_hi + (BN + tm * 16) * kBlock);
      if (part) {
        fa[tm][0] = keep_valid(fa[tm][0], 2 * kc, last_bytes);
        fa[tm][1] = keep_valid(fa[tm][1], 2 * kc + 1, last_bytes);
      }
    }
    // the slot is refilled after this wave's reads of it have returned
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (i + SLOTS < nkb) issue(slot, block_of(i + SLOTS));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
          acc[tn][tm] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[tn][h], fa[tm][h], acc[tn][tm], 0, 0, 0);
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
  }

  // result register i of lane l: weight row 4 (l / 16) + i, activation row l % 16
  int* sums = reinterpret_cast<int*>(&slots[w][0][0]);  // (no copy of this wave is in flight)
#pragma unroll
  for (int tn = 0; tn < TN; ++tn)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) *reinterpret_cast<v4i*>(sums + ((tn * TM + tm) * 64 + lane) * 4) = acc[tn][tm];
  __syncthreads();
  const bool vec_ok = (args.ldc & 3) == 0 && (reinterpret_cast<uintptr_t>(args.c) & 7) == 0;
  for (int q = threadIdx.x; q < TN * TM * 64; q += kWaves * 64) {
    const int ln = q & 63, tile = q >> 6;
    const int m = m0 + (tile % TM) * 16 + (ln & 15), n = n0 + (tile / TM) * 16 + 4 * (ln >> 4);
    if (m >= M || n >= N) continue;
    const float ms = args.as[m];
    float ns[4], add[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = min(n + e, N - 1);
      ns[e] = args.bs[at];
      add[e] = args.bias != nullptr ? bias_value<kF16>(args.bias[at]) : 0.f;
    }
    v4i v = {0, 0, 0, 0};
#pragma unroll
    for (int ww = 0; ww < kWaves; ++ww) v += *reinterpret_cast<const v4i*>(reinterpret_cast<const int*>(&slots[ww][0][0]) + q * 4);
    const int sum[4] = {v[0], v[1], v[2], v[3]};
    uint2 out = outputs4<kF16>(sum, ms, ns, add);
    if (__builtin_expect(scale_is_far(ms), 0)) out = far_outputs4<kF16>(sum, ms, ns, add);
    store4(args.c + (int64_t)m * args.ldc + n, n, N, vec_ok, out.x, out.y);
  }
}

// ---------------------------------------------------------------- one to eight rows, quantized here

// The linear layer of kRows tokens at most: every workgroup quantizes the tokens into LDS while its first weights are on
// their way, and then is the kernel above (16 weight rows a workgroup), with activations that are there already. Each workgroup repeats the
// quantization, which for few codes costs less than a launch of its own.
template <int kIn, int kRows>
__global__ __launch_bounds__(kWaves * 64) void linear_int8_kernel(Int8GemmArgs args, const uint16_t* x, int64_t ldx) {
  constexpr bool kF16 = kIn == kInF16;
  constexpr int BN = 16, SLOTS = 3;
  constexpr int kPieces = BN / 8, kSlot = BN * kBlock;
  constexpr int kShare = kWaves / kRows;  // waves that share a token
  static_assert(kRows * kShare == kWaves && 16 * BN * 4 <= SLOTS * kSlot, "tokens share the waves evenly, sums fit the slots");
  __shared__ __attribute__((aligned(1024))) uint8_t slots[kWaves][SLOTS][kSlot];
  __shared__ __attribute__((aligned(1024))) uint8_t codes[kFusedCodes];  // [K block][kRows][128], columns XORed as elsewhere
  __shared__ float top[kWaves];
  __shared__ float scales[kRows];

  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kc = lane >> 4;
  const int n0 = blockIdx.x * BN, M = args.M, N = args.N, K = args.K;
  const int KB = (K + kBlock - 1) / kBlock, last_bytes = K - (KB - 1) * kBlock;
  const int nkb = KB > w ? (KB - w + kWaves - 1) / kWaves : 0;

  // ---- a share of a token (a row past the last is it again)
  const int token = w / kShare, share = w - token * kShare;
  const uint16_t* row = x + (int64_t)min(token, M - 1) * ldx;
  // (read twice, in loops: code for pieces held in registers takes longer to fetch than they take to come from L2 again)
  const int pieces = (K + kShare * 512 - 1) / (kShare * 512);
  float amax = 0.f;
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const int col = ((i * kShare + share) * 64 + lane) * 8;
    Piece<kIn> v = {};
    if (col < K) v = load_piece<kIn>(row, col);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(element<kIn>(v, e)));
  }
  // ---- the first weights
  uint32_t off[kPieces];
  const int8_t* bmat = args.b + (int64_t)n0 * args.ldb;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int at = j * 8 + (lane >> 3);
    off[j] = (uint32_t)min(at, N - 1 - n0) * (uint32_t)args.ldb + (uint32_t)(((lane & 7) ^ lds_swizzle(at)) * 16);
  }
  auto issue = [&](int slot, int kb) __attribute__((always_inline)) {
    const uint32_t dst = lds_addr(&slots[w][slot][0]);
    const bool part = kb == KB - 1 && last_bytes < kBlock;  // uniform
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int col = (lane & 7) ^ lds_swizzle(j * 8 + (lane >> 3));
      copy16_m0(bmat + (int64_t)kb * kBlock, part && 16 * col >= last_bytes ? off[j] - (uint32_t)(col * 16) : off[j],
                dst + (uint32_t)(j * 1024));
    }
  };
#pragma unroll
  for (int s = 0; s < SLOTS; ++s)
    if (s < nkb) issue(s, w + s * kWaves);
  // ---- codes and scales
  amax = wave_max(amax);
  if constexpr (kShare > 1) {
    if (lane == 0) top[w] = amax;
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kShare; ++i) amax = max_nan(amax, top[token * kShare + i]);
  }
  const Int8Scale scale(amax);
  if (share == 0 && lane == 0) scales[token] = scale.value();
#pragma unroll 2
  for (int i = 0; i < pieces; ++i) {
    const int col = ((i * kShare + share) * 64 + lane) * 8;
    Piece<kIn> v = {};
    if (col < K) v = load_piece<kIn>(row, col);
    if (col < KB * kBlock)  // (zeros past K)
      *reinterpret_cast<uint2*>(codes + ((col >> 7) * kRows + token) * kBlock + ((((col >> 4) & 7) ^ lds_swizzle(token)) << 4) + (col & 8)) =
          row_codes(v, scale);
  }
  lds_barrier();

  const int sw = lds_swizzle(r);
  const uint32_t at_lo = (uint32_t)(r * kBlock + (((2 * kc) ^ sw) << 4)), at_hi = (uint32_t)(r * kBlock + (((2 * kc + 1) ^ sw) << 4));
  const int ra = r % kRows, swa = lds_swizzle(ra);
  const uint32_t a_lo = (uint32_t)(ra * kBlock + (((2 * kc) ^ swa) << 4)), a_hi = (uint32_t)(ra * kBlock + (((2 * kc + 1) ^ swa) << 4));
  v4i acc = {0, 0, 0, 0};
  int slot = 0;
  for (int i = 0; i < nkb; ++i) {
    const int kb = w + i * kWaves;
    if (i + SLOTS - 1 < nkb) wait_copies_upto<(SLOTS - 1) * kPieces>();
    else wait_copies();
    const uint8_t* sl = &slots[w][slot][0];
    const uint8_t* block = codes + kb * kRows * kBlock;
    const v4i fb[2] = {*reinterpret_cast<const v4i*>(sl + at_lo), *reinterpret_cast<const v4i*>(sl + at_hi)};
    const v4i fa[2] = {*reinterpret_cast<const v4i*>(block + a_lo), *reinterpret_cast<const v4i*>(block + a_hi)};
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot has been read
    if (i + SLOTS < nkb) issue(slot, kb + SLOTS * kWaves);
#pragma unroll
    for (int h = 0; h < 2; ++h) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[h], fa[h], acc, 0, 0, 0);
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
  }
  *reinterpret_cast<v4i*>(reinterpret_cast<int*>(&slots[w][0][0]) + lane * 4) = acc;  // (no copy of this wave is in flight)
  __syncthreads();
  const bool vec_ok = (args.ldc & 3) == 0 && (reinterpret_cast<uintptr_t>(args.c) & 7) == 0;
  const int m = r, n = n0 + 4 * kc;
  if (w == 0 && m < M && n < N) {
    const float ms = scales[m];
    v4i v = {0, 0, 0, 0};
#pragma unroll
    for (int ww = 0; ww < kWaves; ++ww) v += *reinterpret_cast<const v4i*>(reinterpret_cast<const int*>(&slots[ww][0][0]) + lane * 4);
    const int sum[4] = {v[0], v[1], v[2], v[3]};
    float ns[4], add[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = min(n + e, N - 1);
      ns[e] = args.bs[at];
      add[e] = args.bias != nullptr ? bias_value<kF16>(args.bias[at]) : 0.f;
    }
    uint2 out = outputs4<kF16>(sum, ms, ns, add);
    if (__builtin_expect(scale_is_far(ms), 0)) out = far_outputs4<kF16>(sum, ms, ns, add);
    store4(args.c + (int64_t)m * args.ldc + n, n, N, vec_ok, out.x, out.y);
  }
}

// ---------------------------------------------------------------- tiles of LDS stages

// A BN x BM tile of C^T, WGN x WGM waves of 32 TN x 32 TM. A K block is four steps of 32x32x32 products; the fragments
// of a step are read while the one before is multiplied. At the end of a block's third step its last fragments have
// been read and the next block has landed; past the barrier there its stage is refilled, and the next block's first
// fragments are read. With two stages (kEarly) that leaves a block's time for its copies to arrive in; so the activations
// are read ahead, all by the end of the first step, and their half of the stage is refilled past a barrier there.
template <int BN, int BM, int WGN, int WGM, int STAGES, bool kPart, bool kF16>
__global__ __launch_bounds__(WGN * WGM * 64) void gemm_int8_tiled_kernel(Int8GemmArgs args) {
  constexpr int kNumWaves = WGN * WGM;
  constexpr int WN = BN / WGN, WM = BM / WGM, TN = WN / 32, TM = WM / 32;
  constexpr int kStage = (BN + BM) * kBlock;
  constexpr int kCopiesB = BN / 8 / kNumWaves, kCopiesA = BM / 8 / kNumWaves;  // pieces of a block that a wave copies
  constexpr int kCopies = kCopiesB + kCopiesA;
  constexpr bool kEarly = STAGES == 2;
  static_assert(BN % (8 * kNumWaves) == 0 && BM % (8 * kNumWaves) == 0 && WN % 32 == 0 && WM % 32 == 0, "whole pieces and products");
  static_assert(STAGES >= 2 && (STAGES - 2) * kCopies < 64, "stages");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * kStage];
  __shared__ __attribute__((aligned(16))) float channel[2][BN];  // scale and bias

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = w % WGN, wm = w / WGN;
  const int r = lane & 31, g = lane >> 5;
  const int M = args.M, N = args.N;
  const int KB = (args.K + kBlock - 1) / kBlock;
  const int last_bytes = args.K - (KB - 1) * kBlock;
  int tile_n, tile_m;
  map_tile(blockIdx.x, (N + BN - 1) / BN, (M + BM - 1) / BM, 8, tile_n, tile_m);
  const int n0 = __builtin_amdgcn_readfirstlane(tile_n * BN), m0 = __builtin_amdgcn_readfirstlane(tile_m * BM);

  const int8_t* bmat = args.b + (int64_t)n0 * args.ldb;
  const int8_t* amat = args.a + (int64_t)m0 * args.lda;
  // a wave's pieces: kCopiesB of the weights' rows, then kCopiesA of the activations'
  uint32_t off[kCopies];
  auto row_of = [&](int j) __attribute__((always_inline)) {  // of the stage
    return j < kCopiesB ? (w * kCopiesB + j) * 8 : BN + (w * kCopiesA + j - kCopiesB) * 8;
  };
#pragma unroll
  for (int j = 0; j < kCopies; ++j) {
    const int row = row_of(j) + (lane >> 3);
    const int col = (lane & 7) ^ lds_swizzle(row);
    off[j] = (j < kCopiesB ? (uint32_t)min(row, N - 1 - n0) * (uint32_t)args.ldb
                           : (uint32_t)min(row - BN, M - 1 - m0) * (uint32_t)args.lda) + (uint32_t)(col * 16);
  }
  const uint32_t lds = lds_addr(smem);
  auto issue_piece = [&](int stage, int kb, int j) __attribute__((always_inline)) {
    uint32_t o = off[j];
    if (kPart && kb == KB - 1) {  // uniform
      const uint32_t col = (uint32_t)((lane & 7) ^ lds_swizzle(row_of(j) + (lane >> 3)));
      if ((int)(16 * col) >= last_bytes) o -= 16 * col;
    }
    copy16_m0((j < kCopiesB ? bmat : amat) + (int64_t)kb * kBlock, o,
              __builtin_amdgcn_readfirstlane(lds + (uint32_t)(stage * kStage + row_of(j) * kBlock)));
  };

  v16i acc[TN][TM];
#pragma unroll
  for (int tn = 0; tn < TN; ++tn)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[tn][tm][i] = 0;

  // fragments: lane l holds row l % 32 and, in step s, the 16-byte column 2 s + l / 32
  const int sw = lds_swizzle(r);
  uint32_t at[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) at[s] = (uint32_t)(r * kBlock + (((2 * s + g) ^ sw) << 4));
  v4i fb[2][TN], fa[kEarly ? 4 : 2][TM];
  auto read_b = [&](const uint8_t* stage, int s, int tn) __attribute__((always_inline)) {
    fb[s & 1][tn] = *reinterpret_cast<const v4i*>(stage + at[s] + (wn * WN + tn * 32) * kBlock);
  };
  auto read_a = [&](const uint8_t* stage, int s, int tm, bool part) __attribute__((always_inline)) {
    v4i& f = fa[kEarly ? s : s & 1][tm];
    f = *reinterpret_cast<const v4i*>(stage + at[s] + (BN + wm * WM + tm * 32) * kBlock);
    if (kPart && part) f = keep_valid(f, 2 * s + g, last_bytes);
  };

  constexpr int kProducts = TN * TM;
  auto block = [&](int kb, int stage, auto steady) __attribute__((always_inline)) {
    constexpr bool kSteady = decltype(steady)::value;  // block kb + STAGES exists
    const int next = stage + 1 == STAGES ? 0 : stage + 1;
    const uint8_t* here = smem + stage * kStage;
    const uint8_t* then = smem + next * kStage;  // (after the last block: stale bytes, not used)
    const bool part_here = kb == KB - 1, part_then = kb + 1 == KB - 1;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      // the fragments read in this step: kEarly: activations of the next block's steps 0 to 2 in the last step, those of
      // step 3 in the first; else each a step ahead
      const int reads_a = !kEarly ? TM : s == 3 ? 3 * TM : s == 0 ? TM : 0, reads = reads_a + TN;
#pragma unroll
      for (int p = 0; p < kProducts; ++p) {
        const int tm = p / TN, tn = p % TN;
        acc[tn][tm] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[s & 1][tn], fa[kEarly ? s : s & 1][tm], acc[tn][tm], 0, 0, 0);
#pragma unroll
        for (int x = 0; x < reads; ++x)
          if (x * kProducts / reads == p) {
            // (weights first: the next step needs them whole)
            if (x < TN) read_b(s < 3 ? here : then, (s + 1) & 3, x);
            else if (!kEarly) read_a(s < 3 ? here : then, (s + 1) & 3, x - TN, s < 3 ? part_here : part_then);
            else if (s == 3) read_a(then, (x - TN) / TM, (x - TN) % TM, part_then);
            else read_a(here, 3, x - TN, part_here);
          }
        if constexpr (kSteady) {
          if (kEarly ? s == 3 || s == 1 : s == 3) {
            const int from = kEarly && s == 1 ? kCopiesB : 0, to = kEarly && s == 3 ? kCopiesB : kCopies;
#pragma unroll
            for (int j = from; j < to; ++j)
              if ((j - from) * kProducts / (to - from) == p) issue_piece(stage, kb + STAGES, j);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (kEarly && s == 0) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        lds_barrier();
      }
      if (s == 2) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        // what may be under way past the next block: its successors, and of the refill begun above the activations
        constexpr int kLater = kEarly ? kCopiesA : (STAGES - 2) * kCopies;
        if (kSteady) wait_copies_upto<kLater>();
        else wait_copies();
        lds_barrier();
      }
    }
    return next;
  };

#pragma unroll
  for (int i = 0; i < STAGES; ++i)
#pragma unroll
    for (int j = 0; j < kCopies; ++j) issue_piece(i, min(i, KB - 1), j);
  wait_copies_upto<(STAGES - 1) * kCopies>();
  lds_barrier();
#pragma unroll
  for (int s = 0; s < (kEarly ? 3 : 1); ++s)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) read_a(smem, s, tm, KB == 1);
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) read_b(smem, 0, tn);
  int stage = 0, kb = 0;
  for (; kb + STAGES < KB; ++kb) stage = block(kb, stage, std::true_type{});
  for (; kb < KB; ++kb) stage = block(kb, stage, std::false_type{});
  lds_barrier();  // every wave is done with the stages (no copy is in flight: the last block waited for all)

  for (int i = tid; i < BN; i += kNumWaves * 64) {
    const int n = min(n0 + i, N - 1);
    channel[0][i] = args.bs[n];
    channel[1][i] = args.bias != nullptr ? bias_value<kF16>(args.bias[n]) : 0.f;
  }
  __syncthreads();

  // result register v of lane l: weight row 8 (v / 4) + 4 (l / 32) + v % 4, activation row l % 32. A wave's 32 rows go through LDS (rows
  // padded by 16 bytes) so that neighbouring lanes store neighbours of a row: 16 bytes each where rows of C allow it, else 4 or 2 (1569
  // tokens, 4826 channels, K = 288: 14 us, 31 with the 8 bytes that a lane holds of each row).
  constexpr int kRowBytes = WN * 2 + 16;
  static_assert(kNumWaves * 32 * kRowBytes <= STAGES * kStage, "staged output");
  uint8_t* staged = smem + w * 32 * kRowBytes;
  const bool vec16 = (args.ldc & 7) == 0 && (reinterpret_cast<uintptr_t>(args.c) & 15) == 0;
  const bool vec4 = (args.ldc & 1) == 0 && (reinterpret_cast<uintptr_t>(args.c) & 3) == 0;
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const float ms = args.as[min(m0 + wm * WM + tm * 32 + r, M - 1)];
    auto stage = [&](auto outputs) __attribute__((always_inline)) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = tn * 32 + 8 * q + 4 * g;
          const v4f s = *reinterpret_cast<const v4f*>(&channel[0][wn * WN + col]);
          const v4f b = *reinterpret_cast<const v4f*>(&channel[1][wn * WN + col]);
          int sum[4];
          float ns[4], add[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = acc[tn][tm][4 * q + e], ns[e] = s[e], add[e] = b[e];
          *reinterpret_cast<uint2*>(staged + r * kRowBytes + col * 2) = outputs(sum, ms, ns, add);
        }
    };
    if (__builtin_expect(scale_is_far(ms), 0)) stage([](auto... v) __attribute__((always_inline)) { return far_outputs4<kF16>(v...); });
    else stage([](auto... v) __attribute__((always_inline)) { return outputs4<kF16>(v...); });
    // (LDS executes a wave's accesses in order; this keeps the compiler to it)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    // pieces of kUnit columns, a lane each
    auto rows_out = [&](auto type, auto store) __attribute__((always_inline)) {
      using T = decltype(type);
      constexpr int kUnit = sizeof(T) / 2, kLanes = WN / kUnit;
#pragma unroll 4
      for (int i = lane; i < 32 * kLanes; i += 64) {
        const int row = i / kLanes, seg = i % kLanes;
        const int m = m0 + wm * WM + tm * 32 + row, n = n0 + wn * WN + seg * kUnit;
        if (m < M && n < N) store(args.c + (int64_t)m * args.ldc + n, n, *reinterpret_cast<const T*>(staged + row * kRowBytes + seg * sizeof(T)));
      }
    };
    if (vec16) {
      rows_out(v4i{}, [&](uint16_t* c, int n, const v4i& v) {
        if (n + 8 <= N) {
          *reinterpret_cast<v4i*>(c) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < N) c[e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
        }
      });
    } else if (vec4) {
      rows_out(uint32_t{}, [&](uint16_t* c, int n, uint32_t v) {
        if (n + 2 <= N) *reinterpret_cast<uint32_t*>(c) = v;
        else c[0] = (uint16_t)v;
      });
    } else {
      rows_out(uint16_t{}, [&](uint16_t* c, int, uint16_t v) { c[0] = v; });
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
  }
}

template <int TN, int TM, int SLOTS>
hipError_t ksplit(const Int8GemmArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 16 * TN - 1) / (16 * TN)), (unsigned)((a.M + 16 * TM - 1) / (16 * TM)));
  if (a.out_f16) hipLaunchKernelGGL((gemm_int8_ksplit_kernel<TN, TM, SLOTS, true>), grid, dim3(kWaves * 64), 0, stream, a);
  else hipLaunchKernelGGL((gemm_int8_ksplit_kernel<TN, TM, SLOTS, false>), grid, dim3(kWaves * 64), 0, stream, a);
  return hipGetLastError();
}

template <int BN, int BM, int WGN, int WGM, int STAGES, bool kPart>
hipError_t tiled_as(const Int8GemmArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)(a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM))), threads(WGN * WGM * 64);
  if (a.out_f16) hipLaunchKernelGGL((gemm_int8_tiled_kernel<BN, BM, WGN, WGM, STAGES, kPart, true>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((gemm_int8_tiled_kernel<BN, BM, WGN, WGM, STAGES, kPart, false>), grid, threads, 0, stream, a);
  return hipGetLastError();
}
template <int BN, int BM, int WGN, int WGM, int STAGES>
hipError_t tiled(const Int8GemmArgs& a, hipStream_t stream) {
  return a.K % kBlock ? tiled_as<BN, BM, WGN, WGM, STAGES, true>(a, stream) : tiled_as<BN, BM, WGN, WGM, STAGES, false>(a, stream);
}

// A kernel's predicted time in microseconds, as sums of what it moves and does, fitted to times measured with cold weights
// over 19 weight shapes from 12 x 25600 to 51200 x 5120 and 1 to 8192 tokens, rows as long as K: the choice by it takes 1.1 % longer than the
// fastest of the 13 on (geometric) average over 151 of them, 32 % at worst. (A round is counted as 256 workgroups, one a compute unit; kernels of which
// several share one run more at once, for which their fitted terms stand. That a row pitch of no whole 128-byte lines costs up to 45 % is not in it.)
struct Shape {
  int bn, bm;
  hipError_t (*launch)(const Int8GemmArgs&, hipStream_t);
  // a launch, a K block of a round and a round; MB copied by all workgroups, MB of weights, 10^6 outputs
  double base, per_block, per_round, copied, weights, outputs;
};
constexpr Shape kTiled[] = {
    {256, 256, tiled<256, 256, 2, 4, 2>, 3.00, 0.797, 4.77, 0.0461, 0.0155, 0.208},
    {256, 128, tiled<256, 128, 4, 2, 3>, 2.49, 0.614, 3.09, 0.0267, 0.0680, 0.211},
    {128, 256, tiled<128, 256, 2, 4, 3>, 2.70, 0.508, 2.99, 0.0340, 0.0500, 0.224},
    {128, 128, tiled<128, 128, 2, 4, 4>, 2.75, 0.404, 0.68, 0.0191, 0.0743, 0.568},
    {64, 128, tiled<64, 128, 2, 4, 4>, 1.55, 0.289, 1.49, 0.0152, 0.0453, 0.452},
    {64, 64, tiled<64, 64, 2, 2, 4>, 2.48, 0.217, 0.40, 0.0, 0.0922, 0.523},
};
struct SplitShape {
  int bn, bm;
  hipError_t (*launch)(const Int8GemmArgs&, hipStream_t);
};
constexpr SplitShape kSplit[] = {{16, 16, ksplit<1, 1, 2>}, {16, 32, ksplit<1, 2, 2>}, {32, 16, ksplit<2, 1, 3>}, {32, 32, ksplit<2, 2, 2>},
                                 {64, 16, ksplit<4, 1, 1>}, {32, 64, ksplit<2, 4, 1>}, {64, 64, ksplit<4, 4, 1>}};

struct Choice {
  Int8Choice kernel;
  hipError_t (*launch)(const Int8GemmArgs&, hipStream_t);
};
Choice choose(int64_t M, int64_t N, int64_t K) {
  const double blocks = (double)((K + kBlock - 1) / kBlock), weights = 1e-6 * N * (double)K, outputs = 1e-6 * N * (double)M;
  double best = 1e30;
  Choice choice{};
  auto tiles = [&](int bn, int bm) { return (double)((N + bn - 1) / bn) * (double)((M + bm - 1) / bm); };
  for (const SplitShape& s : kSplit) {
    if ((M + s.bm - 1) / s.bm > 65535) continue;  // the grid's second dimension
    const double n = tiles(s.bn, s.bm), rounds = std::ceil(n / 256), mb = 1e-6 * kBlock * (s.bn + s.bm) * blocks;
    const double us = 1.91 + 0.107 * weights + 9.02 * rounds * mb + 0.0146 * n * mb + 0.354 * rounds +
                      0.000238 * rounds * s.bn * s.bm + 0.893 * outputs;
    if (us < best) best = us, choice = {{s.bn, s.bm, true}, s.launch};
  }
  for (const Shape& s : kTiled) {
    const double n = tiles(s.bn, s.bm), rounds = std::ceil(n / 256), mb = 1e-6 * kBlock * (s.bn + s.bm) * blocks;
    const double us = s.base + rounds * (s.per_block * blocks + s.per_round) + s.copied * n * mb + s.weights * weights + s.outputs * outputs;
    if (us < best) best = us, choice = {{s.bn, s.bm, false}, s.launch};
  }
  return choice;
}

}  // namespace

Int8Choice choose_gemm_int8(int64_t M, int64_t N, int64_t K) { return choose(M, N, K).kernel; }
hipError_t launch_gemm_int8(const Int8GemmArgs& a, hipStream_t stream) { return choose(a.M, a.N, a.K).launch(a, stream); }

namespace {
template <int kIn, int kRows>
hipError_t linear_rows(const Int8GemmArgs& a, const uint16_t* x, int64_t ldx, hipStream_t stream) {
  hipLaunchKernelGGL((linear_int8_kernel<kIn, kRows>), dim3((unsigned)((a.N + 15) / 16)), dim3(kWaves * 64), 0, stream, a, x, ldx);
  return hipGetLastError();
}
template <int kIn>
hipError_t linear_small(const Int8GemmArgs& a, const uint16_t* x, int64_t ldx, hipStream_t stream) {
  if (a.M == 1) return linear_rows<kIn, 1>(a, x, ldx, stream);
  if (a.M == 2) return linear_rows<kIn, 2>(a, x, ldx, stream);
  if (a.M <= 4) return linear_rows<kIn, 4>(a, x, ldx, stream);
  return linear_rows<kIn, 8>(a, x, ldx, stream);
}
}  // namespace

// Where one launch is faster (bf16, cold weights, us for one launch and for two, 1 and 8 tokens): 1024 x 1024 3.4 and 5.0, 4.2 and 5.2;
// 4096 x 4096 7.3 and 9.5 (3 tokens 8.9 and 8.9); 7168 x 2048 6.0 and 7.9, 8.3 and 8.2. Not past one round of workgroups, two a compute unit:
// 25600 x 1600 15.9 and 13.0, 22.0 and 13.3.
bool linear_int8_fuses(int64_t M, int64_t N, int64_t K) {
  const int64_t rows = M <= 2 ? M : M <= 4 ? 4 : 8;
  return M >= 1 && M <= 8 && N <= 16 * 512 && rows * ((K + kBlock - 1) / kBlock * kBlock) <= kFusedCodes;
}

hipError_t launch_linear_int8(const Int8GemmArgs& a, const uint16_t* x, int64_t ldx, hipStream_t stream) {
  return a.out_f16 ? linear_small<kInF16>(a, x, ldx, stream) : linear_small<kInBf16>(a, x, ldx, stream);
}

}  // namespace bfp8
