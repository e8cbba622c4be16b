// Per-token quantization of activations to 8-bit integers.
//
// For every row m of x [M][K]:  a = max(max_k |x|, 1e-10),  s = a / 127 (correctly rounded),
// q = 127 x / a rounded to the nearest integer, ties to even, of the exact quotient.
// In float32, t = x * (127 / a) is off by at most 2^-23 of |t| <= 127 and so is decided unless it lies
// within 2^-16 of the middle of two integers; there 127 x and (middle) a, both exact in 64 bits, are
// compared. (bf16 and fp16 tokens hold many exact middles: a token whose largest element is 127 times a
// power of two, for one.) A row with an infinite or NaN element has a NaN scale and zero codes.
//
// HBM-bound: x is read once, q written once. A row lives in the registers of the waves that share it, 8
// elements a thread and chunk, as loaded; the waves exchange its largest element through LDS.
#include "device_latent.h"
#include "int8.h"
#include "launch.h"

namespace bfp8 {

namespace {

// 8 elements of type kIn, as loaded.
template <int kIn>
struct Piece {
  uint4 v[kIn == kInF32 ? 2 : 1];
};
template <int kIn>
__device__ __forceinline__ Piece<kIn> load_piece(const void* row, int col) {
  Piece<kIn> p;
  const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + (int64_t)col * (kIn == kInF32 ? 4 : 2));
  p.v[0] = at[0];
  if constexpr (kIn == kInF32) p.v[1] = at[1];
  return p;
}
template <int kIn>
__device__ __forceinline__ float element(const Piece<kIn>& p, int i) {  // (i is known at compile time)
  if constexpr (kIn == kInF32) {
    const uint4& v = p.v[i >> 2];
    return __uint_as_float((i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w);
  } else {
    const uint4& v = p.v[0];
    const uint32_t w = (i >> 1) == 0 ? v.x : (i >> 1) == 1 ? v.y : (i >> 1) == 2 ? v.z : v.w;
    if constexpr (kIn == kInBf16) return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    else return f16_value(i & 1 ? w >> 16 : w & 0xffffu);
  }
}

// x rounded where t, its quotient in float32, is too near the middle of two integers to tell.
__device__ __noinline__ float decide(float x, float a, float t) {
  const float below = floorf(t);
  const double d = 127.0 * (double)x - ((double)below + 0.5) * (double)a;  // both products are exact
  const bool odd = (int)below & 1;
  return d > 0.0 || (d == 0.0 && odd) ? below + 1.0f : below;
}

// kWaves waves share a row (kWaves == 1: four rows a workgroup), kChunks chunks of 8 elements a thread.
template <int kIn, int kWaves, int kChunks>
__global__ __launch_bounds__(kWaves == 1 ? 256 : kWaves * 64) void quant_int8_kernel(
    const void* __restrict__ x, int64_t row_bytes, int8_t* __restrict__ q, int64_t ldq, float* __restrict__ s, int M, int K) {
  constexpr int kRows = kWaves == 1 ? 4 : 1;
  constexpr int kThreads = kWaves * 64;
  const int tid = kWaves == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int m_raw = blockIdx.x * kRows + (kWaves == 1 ? threadIdx.x >> 6 : 0);
  const bool row_ok = m_raw < M;  // a wave past the last row redoes it and stores nothing
  const int64_t m = row_ok ? m_raw : M - 1;
  const uint8_t* row = static_cast<const uint8_t*>(x) + m * row_bytes;

  Piece<kIn> v[kChunks];
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * kThreads + tid) * 8;
    v[c] = {};
    if (col < K) v[c] = load_piece<kIn>(row, col);
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max_nan(amax, fabsf(element<kIn>(v[c], i)));
  amax = wave_max(amax);
  if constexpr (kWaves > 1) {
    __shared__ float part[kWaves];
    if ((tid & 63) == 0) part[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) amax = max_nan(amax, part[i]);
  }
  const bool finite = amax < __builtin_inff();
  const float a = fmaxf(amax, 1e-10f);
  const float f = finite ? 127.0f / a : 0.f;
  if (tid == 0 && row_ok) s[m] = finite ? a / 127.0f : __builtin_nanf("");

#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * kThreads + tid) * 8;
    if (col >= K || !row_ok) continue;
    float r[8];
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = element<kIn>(v[c], i) * f;
      r[i] = rintf(t);
      near |= fabsf(t - r[i]) > 0.5f - 0x1p-16f;
    }
    if (__builtin_expect(near, 0)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = element<kIn>(v[c], i), t = e * f;
        if (fabsf(t - r[i]) > 0.5f - 0x1p-16f) r[i] = decide(e, a, t);
      }
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b0 = finite ? (int)r[4 * h] : 0, b1 = finite ? (int)r[4 * h + 1] : 0;
      const int b2 = finite ? (int)r[4 * h + 2] : 0, b3 = finite ? (int)r[4 * h + 3] : 0;
      w[h] = (b0 & 0xff) | (b1 & 0xff) << 8 | (b2 & 0xff) << 16 | (uint32_t)b3 << 24;
    }
    *reinterpret_cast<uint2*>(q + m * ldq + col) = make_uint2(w[0], w[1]);
  }
}

template <int kIn, int kWaves, int kChunks>
void run(const void* x, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq, float* s, hipStream_t stream) {
  constexpr int kRows = kWaves == 1 ? 4 : 1;
  hipLaunchKernelGGL((quant_int8_kernel<kIn, kWaves, kChunks>), dim3((unsigned)((M + kRows - 1) / kRows)),
                     dim3(kWaves == 1 ? 256 : kWaves * 64), 0, stream, x, ldx * (kIn == kInF32 ? 4 : 2), q, ldq, s, (int)M, (int)K);
}

// By the row's length alone: a wave for every 512 elements, eight at most up to 8192.
template <int kIn>
void choose(const void* x, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq, float* s, hipStream_t stream) {
  const int64_t pieces = (K + 511) / 512;  // 64 lanes of 8 elements
  if (pieces <= 1) run<kIn, 1, 1>(x, M, K, ldx, q, ldq, s, stream);
  else if (pieces <= 2) run<kIn, 2, 1>(x, M, K, ldx, q, ldq, s, stream);
  else if (pieces <= 4) run<kIn, 4, 1>(x, M, K, ldx, q, ldq, s, stream);
  else if (pieces <= 8) run<kIn, 8, 1>(x, M, K, ldx, q, ldq, s, stream);
  else if (pieces <= 16) run<kIn, 8, 2>(x, M, K, ldx, q, ldq, s, stream);
  else if (pieces <= 32) run<kIn, 16, 2>(x, M, K, ldx, q, ldq, s, stream);
  else if (pieces <= 64) run<kIn, 16, 4>(x, M, K, ldx, q, ldq, s, stream);
  else run<kIn, 16, 8>(x, M, K, ldx, q, ldq, s, stream);
}

}  // namespace

hipError_t launch_quant_act_int8(const void* x, int x_dtype, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* s, hipStream_t stream) {
  if (x_dtype == kInBf16) choose<kInBf16>(x, M, K, ldx, q, ldq, s, stream);
  else if (x_dtype == kInF16) choose<kInF16>(x, M, K, ldx, q, ldq, s, stream);
  else choose<kInF32>(x, M, K, ldx, q, ldq, s, stream);
  return hipGetLastError();
}

}  // namespace bfp8
