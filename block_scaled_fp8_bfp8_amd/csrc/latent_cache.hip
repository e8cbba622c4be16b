// The paged FP8 latent cache of latent attention: writing tokens, reading them back.
//
// A cached token is one row of kLatentRow = 640 bytes: the 512 latents as e4m3 codes, then the 64
// values of the rotary key in bf16; and one UE8M0 scale code in a separate array. A page holds
// page_size rows. The scale of a token is its 1x512 group's max(amax, 1e-10) / 448 rounded up to
// a power of two, held within 2^-42 .. 2^40 (the codes saturate beyond): one code serves the
// token in the hardware-scaled products of attention, and repeated four times it is the token's
// row of 1x128 scales for the UE8M0 GEMM. A token whose latents hold a NaN or an infinity is
// stored as zero codes with scale code 255 (NaN): rows that see it become NaN, rows that do not
// multiply it by a zero weight and stay finite.
//
// All three kernels are HBM-bound (a token: 1152 bytes read and 641 written, or the reverse) once there are enough
// tokens; 16384 written tokens take 9.5 us (3.1 TB/s), most of it the latency of a wave's load, fold and store.
#include "device_latent.h"
#include "latent.h"
#include "launch.h"

namespace bfp8 {

namespace {

constexpr int kTokensPerBlock = 4;  // one wave a token

__global__ __launch_bounds__(256) void latent_write_kernel(const uint16_t* __restrict__ kv, int64_t ld_kv,
                                                           const uint16_t* __restrict__ w, float eps,
                                                           const int64_t* __restrict__ slots, int T, LatentCache cache,
                                                           uint8_t* __restrict__ rows, uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * kTokensPerBlock + (threadIdx.x >> 6);
  if (t >= T) return;
  const int64_t slot = slots[t];
  // negative: a padding token; past the cache: nothing there to write
  if (slot < 0 || slot >= (int64_t)cache.pages * cache.page_size) return;
  const int page = (int)slot / cache.page_size;
  const int off = (int)slot - page * cache.page_size;
  uint8_t* row = rows + page * cache.page_stride + (int64_t)off * kLatentRow;
  const uint16_t* src = kv + t * ld_kv;

  const uint4 r = *reinterpret_cast<const uint4*>(src + lane * 8);
  uint4 rope = make_uint4(0, 0, 0, 0);
  if (lane < 8) rope = *reinterpret_cast<const uint4*>(src + kLatentDim + lane * 8);
  float y[8];
  bf16x8_values(r, y);
  if (w != nullptr) {
    auto token_mean = [&] {  // of the y^2
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(y[i], y[i], sum);
      return wave_sum(sum) / (float)kLatentDim;
    };
    float mean = token_mean() + eps;
    // squares that pass float32 or come near its least: the token again, times a power of two
    const float by = !(mean < __builtin_inff()) ? 0x1p-80f : mean < 0x1p-96f ? 0x1p100f : 1.0f;
    if (by != 1.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= by;
      mean = token_mean() + eps * by * by;
    }
    const float rstd = 1.0f / sqrtf(mean);
    float f[8];
    bf16x8_values(*reinterpret_cast<const uint4*>(w + lane * 8), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (y[i] * rstd) * f[i];
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(y[i]));
  amax = wave_max(amax);
  uint32_t code = 255;
  uint2 codes = make_uint2(0, 0);
  if (amax < __builtin_inff()) {
    code = (__float_as_uint(max_nan(amax, 1e-10f) / 448.0f) + 0x7fffffu) >> 23;
    code = min(max(code, kLatentMinCode), kLatentMaxCode);
    const float inv = __uint_as_float((254u - code) << 23);  // exact
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = clamp_e4m3(y[i] * inv);
    codes = make_uint2(pack_e4m3(y), pack_e4m3(y + 4));
  }
  *reinterpret_cast<uint2*>(row + lane * 8) = codes;
  if (lane < 8) *reinterpret_cast<uint4*>(row + kLatentDim + lane * 16) = rope;
  if (lane == 0) scales[page * cache.scale_stride + off] = (uint8_t)code;
}

constexpr int kTokensPerWave = 8;  // 5 loads of 16 bytes a lane

// Reads tokens cu[b] .. cu[b+1) of the sequences b back in order. kRaw: codes, the scale code
// four times and the rotary key as stored; otherwise bf16(code * scale) and the rotary key.
// A token whose page the table does not name (an entry outside the cache, or a position past the
// table) reads as NaN; tokens past cu[B] are left unwritten.
//
// A wave takes 8 neighbouring tokens: its first 8 lanes look them up, then the 8 x 40 pieces of 16 bytes
// are spread over all lanes, 5 each, all in flight at once (a wave a token with 8-byte pieces: 33 us for
// 16 sequences of 2000 to 8192 tokens gathered; this: 19.4 us, 5.5 TB/s).
template <bool kRaw>
__global__ __launch_bounds__(256) void latent_read_kernel(LatentCache cache, const int32_t* __restrict__ cu, int B,
                                                          int T, uint8_t* __restrict__ q, int64_t ldq,
                                                          uint8_t* __restrict__ e, int64_t ld_e,
                                                          uint16_t* __restrict__ out, int64_t ld_out) {
  constexpr int kPieces = kLatentRow / 16, kCodePieces = kLatentDim / 16;
  const int lane = threadIdx.x & 63;
  const int t0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * kTokensPerWave;
  if (t0 >= T) return;
  // ---- lane i < 8: where token t0 + i lies
  const int mine = t0 + (lane & (kTokensPerWave - 1));
  int seq = -1, first = 0;  // the last sequence that starts at or before it, and that start
  for (int b = 0; b < B; b += 64) {
    const int start = b + lane < B ? cu[b + lane] : INT32_MAX;
#pragma unroll
    for (int i = 0; i < kTokensPerWave; ++i) {
      const int n = __popcll(__ballot(start <= t0 + i));  // (starts rise)
      const int at = __shfl(start, max(n - 1, 0));
      if ((lane & (kTokensPerWave - 1)) == i && n > 0) seq = b + n - 1, first = at;
    }
  }
  const bool there = seq >= 0 && mine < T && mine < cu[B];
  const int pos = there ? max(mine - first, 0) : 0;
  const int col = pos / cache.page_size;
  const int page = there && col < cache.table_width ? cache.table[seq * cache.table_stride + col] : -1;
  const bool bad = page < 0 || page >= cache.pages;
  const int off = pos - col * cache.page_size;
  const int64_t place = bad ? 0 : page * cache.page_stride + (int64_t)off * kLatentRow;
  const int code = bad ? 255 : (int)cache.scales[page * cache.scale_stride + off];
  if constexpr (kRaw) {
    if (there && lane < 32) e[(lane >> 3) * ld_e + mine] = (uint8_t)code;
  }
  const int flags = (there ? 1 : 0) | (bad ? 2 : 0) | code << 8;
  // ---- the pieces
  constexpr int kEach = kTokensPerWave * kPieces / 64;
  static_assert(kTokensPerWave * kPieces % 64 == 0, "whole rounds of the lanes");
  uint4 data[kEach];
  int flag[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int c = lane + 64 * i, token = c / kPieces;
    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)place, token), hi = (uint32_t)__shfl((int)(place >> 32), token);
    flag[i] = __shfl(flags, token);
    data[i] = *reinterpret_cast<const uint4*>(cache.rows + (((uint64_t)hi << 32) | lo) + (c - token * kPieces) * 16);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int c = lane + 64 * i, token = c / kPieces, piece = c - token * kPieces;
    if (!(flag[i] & 1)) continue;
    const int64_t t = t0 + token;
    const bool none = flag[i] & 2;
    uint4 d = data[i];
    if (piece >= kCodePieces) {
      if (none) d = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      *reinterpret_cast<uint4*>(out + t * ld_out + (kRaw ? 0 : kLatentDim) + (piece - kCodePieces) * 8) = d;
    } else if constexpr (kRaw) {
      if (none) d = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(q + t * ldq + piece * 16) = d;
    } else {
      if (none) d = make_uint4(0, 0, 0, 0);
      const float s = e8_value((uint32_t)flag[i] >> 8);
      float f[16];
      e4m3x8_values(make_uint2(d.x, d.y), f);
      e4m3x8_values(make_uint2(d.z, d.w), f + 8);
      uint32_t p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = pack_bf16(f[2 * j] * s, f[2 * j + 1] * s);
      uint4* dst = reinterpret_cast<uint4*>(out + t * ld_out + piece * 16);
      dst[0] = make_uint4(p[0], p[1], p[2], p[3]);
      dst[1] = make_uint4(p[4], p[5], p[6], p[7]);
    }
  }
}

}  // namespace

hipError_t launch_latent_write(const uint16_t* kv, int64_t T, int64_t ld_kv, const uint16_t* w, float eps,
                               const int64_t* slots, const LatentCache& cache, uint8_t* rows, uint8_t* scales,
                               hipStream_t stream) {
  hipLaunchKernelGGL(latent_write_kernel, dim3((unsigned)((T + kTokensPerBlock - 1) / kTokensPerBlock)), dim3(256), 0,
                     stream, kv, ld_kv, w, eps, slots, (int)T, cache, rows, scales);
  return hipGetLastError();
}

hipError_t launch_latent_read(const LatentCache& cache, const int32_t* cu, int64_t B, int64_t T, uint16_t* out,
                              int64_t ld_out, hipStream_t stream) {
  hipLaunchKernelGGL((latent_read_kernel<false>), dim3((unsigned)((T + 4 * kTokensPerWave - 1) / (4 * kTokensPerWave))),
                     dim3(256), 0, stream, cache, cu, (int)B, (int)T, nullptr, 0, nullptr, 0, out, ld_out);
  return hipGetLastError();
}

hipError_t launch_latent_gather(const LatentCache& cache, const int32_t* cu, int64_t B, int64_t T, uint8_t* q,
                                int64_t ldq, uint8_t* e, int64_t ld_e, uint16_t* rope, int64_t ld_rope,
                                hipStream_t stream) {
  hipLaunchKernelGGL((latent_read_kernel<true>), dim3((unsigned)((T + 4 * kTokensPerWave - 1) / (4 * kTokensPerWave))),
                     dim3(256), 0, stream, cache, cu, (int)B, (int)T, q, ldq, e, ld_e, rope, ld_rope);
  return hipGetLastError();
}

}  // namespace bfp8
