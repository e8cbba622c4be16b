// Residual addition, root-mean-square norm and FP8 quantization of activations in one pass.
//
// For every row m of x [M][H]:
//   h = round_dtype(x + residual)              (h = x without a residual)
//   r = 1 / sqrt(mean(h^2) + eps),  y = (h * r) * w
//   s = max(amax_128(y), 1e-10) / 448,  q = e4m3_RNE(clamp(y / s, -448, 448))
// with the quantizer's 1x128 groups and group-major scales as[g * ld_as + m], or its UE8M0 form
// (s rounded up to a power of two, stored as the biased exponent byte). The sum of squares, the
// norm and y are float32; y is not rounded between the norm and the quantization. A NaN in a
// group makes its scale and codes NaN (maximum() below propagates it).
//
// HBM-bound: x and the residual are read once, h, q and s written once (7 bytes an element in bf16;
// 8192 rows of 7168 with UE8M0 scales: 76 us, 5.4 TB/s). A row lives in the registers of the threads
// that share it, 8 elements a chunk, so the 16 lanes of a 128-wide group exchange its amax by lane
// shuffles (beyond 32768 columns a few registers of a thread, in float32 66 of them, go to scratch
// memory).
#include "device_latent.h"
#include "launch.h"

namespace bfp8 {

namespace {

template <int kIn>
struct Raw8 {  // 8 elements as loaded
  uint4 v[kIn == kInF32 ? 2 : 1];
};

template <int kIn>
__device__ __forceinline__ Raw8<kIn> load8(const void* base, int64_t elem) {
  Raw8<kIn> r;
  if constexpr (kIn == kInF32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + elem);
    r.v[0] = p[0];
    r.v[1] = p[1];
  } else {
    r.v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem);
  }
  return r;
}

template <int kIn>
__device__ __forceinline__ void widen8(const Raw8<kIn>& r, float* f) {
#pragma unroll
  for (int j = 0; j < (kIn == kInF32 ? 2 : 1); ++j) {
    const uint32_t w[4] = {r.v[j].x, r.v[j].y, r.v[j].z, r.v[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kIn == kInF32) {
        f[4 * j + i] = __uint_as_float(w[i]);
      } else if constexpr (kIn == kInBf16) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        f[2 * i] = f16_value(w[i] & 0xffffu);
        f[2 * i + 1] = f16_value(w[i] >> 16);
      }
    }
  }
}

// kWaves waves share a row (kWaves == 1: four rows a workgroup), kChunks chunks of 8 elements a thread. h_out may be
// x or res: a thread reads its chunks of both before it writes them (a wave that redoes the last row stores nothing of it).
template <int kIn, bool kE8, int kWaves, int kChunks>
__global__ __launch_bounds__(kWaves == 1 ? 256 : kWaves * 64) void rmsnorm_quant_kernel(
    const void* x, int64_t ldx, const void* res, int64_t ld_res, const void* __restrict__ w, float eps,
    void* h_out, int64_t ld_h, uint8_t* __restrict__ q, int64_t ldq, void* __restrict__ as, int64_t ld_as, int M,
    int H) {
  constexpr int kRows = kWaves == 1 ? 4 : 1;
  constexpr int kThreads = kWaves * 64;
  const int tid = kWaves == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int m_raw = blockIdx.x * kRows + (kWaves == 1 ? threadIdx.x >> 6 : 0);
  const bool row_ok = m_raw < M;  // a wave past the last row redoes it and stores nothing
  const int64_t m = row_ok ? m_raw : M - 1;

  float v[kChunks][8];
  Raw8<kIn> wr[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * kThreads + tid) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
    if (col < H) widen8<kIn>(load8<kIn>(x, m * ldx + col), v[c]);
  }
  if (res != nullptr) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int col = (c * kThreads + tid) * 8;
      if (col < H) {
        float f[8];
        widen8<kIn>(load8<kIn>(res, m * ld_res + col), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += f[i];
        Raw8<kIn> o;  // the sum rounded to the stream's type: what is stored is what is normed
        if constexpr (kIn == kInF32) {
          o.v[0] = make_uint4(__float_as_uint(v[c][0]), __float_as_uint(v[c][1]), __float_as_uint(v[c][2]),
                              __float_as_uint(v[c][3]));
          o.v[1] = make_uint4(__float_as_uint(v[c][4]), __float_as_uint(v[c][5]), __float_as_uint(v[c][6]),
                              __float_as_uint(v[c][7]));
        } else {
          uint32_t p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (kIn == kInBf16) p[i] = pack_bf16(v[c][2 * i], v[c][2 * i + 1]);
            else p[i] = f32_to_f16_rne(v[c][2 * i]) | (f32_to_f16_rne(v[c][2 * i + 1]) << 16);
          }
          o.v[0] = make_uint4(p[0], p[1], p[2], p[3]);
          widen8<kIn>(o, v[c]);
        }
        if (row_ok) {
          if constexpr (kIn == kInF32) {
            uint4* p = reinterpret_cast<uint4*>(static_cast<float*>(h_out) + m * ld_h + col);
            p[0] = o.v[0];
            p[1] = o.v[1];
          } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(h_out) + m * ld_h + col) = o.v[0];
          }
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * kThreads + tid) * 8;
    if (col < H) wr[c] = load8<kIn>(w, col);
  }

  __shared__ float part[kWaves > 1 ? 2 : 1][kWaves];
  // the row's sum of v^2
  auto row_sum = [&](int turn) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[c][i], v[c][i], sum);
#pragma unroll
    for (int mask = 1; mask < 64; mask <<= 1) sum += __shfl_xor(sum, mask);
    if constexpr (kWaves > 1) {
      if ((tid & 63) == 0) part[turn][tid >> 6] = sum;
      __syncthreads();
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) sum += part[turn][i];
    }
    return sum;
  };
  float mean = row_sum(0) / (float)H + eps;
  // Squares that pass float32 (|v| of 2^56 or more) or come near its least: the row again, times a power of two
  // with which 65536 squares stay below 2^120. Only an infinite or NaN element still ends in an infinite or NaN sum.
  const float f = !(mean < __builtin_inff()) ? 0x1p-80f : mean < 0x1p-96f ? 0x1p100f : 1.0f;
  if (f != 1.0f) {  // (the same in every thread of the row)
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= f;
    mean = row_sum(kWaves > 1 ? 1 : 0) / (float)H + eps * f * f;
  }
  const float rstd = 1.0f / sqrtf(mean);

#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * kThreads + tid) * 8;
    const bool in = col < H;
    float y[8];
    float amax = 0.f;
    if (in) {
      widen8<kIn>(wr[c], y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = (v[c][i] * rstd) * y[i];
        amax = max_nan(amax, fabsf(y[i]));
      }
    }
#pragma unroll
    for (int mask = 1; mask < 16; mask <<= 1) amax = max_nan(amax, __shfl_xor(amax, mask));
    if (!in || !row_ok) continue;
    float s = max_nan(amax, 1e-10f) / 448.0f;  // correctly rounded divide
    uint32_t code;
    if constexpr (kE8) {
      // up to the next power of two; infinity and NaN become the code of NaN
      code = s < __builtin_inff() ? (__float_as_uint(s) + 0x7fffffu) >> 23 : 255u;
      const float inv = code == 255u ? __builtin_nanf("") : __uint_as_float((254u - code) << 23);  // exact
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = clamp_e4m3(y[i] * inv);
    } else {
      // y / s by a correctly rounded reciprocal and one correction step: the correctly rounded
      // quotient wherever it rounds to a non-zero code (no underflow there).
      const float rcp = 1.0f / s;
      const float back = s < __builtin_inff() ? s : 0.f;  // no step with an infinite scale: y / s = y * 0
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q0 = y[i] * rcp;
        const float e = fmaf(-q0, back, y[i]);
        y[i] = clamp_e4m3(fmaf(e, rcp, q0));
      }
    }
    *reinterpret_cast<uint2*>(q + m * ldq + col) = make_uint2(pack_e4m3(y), pack_e4m3(y + 4));
    if ((tid & 15) == 0) {
      const int64_t at = (int64_t)(col >> 7) * ld_as + m;
      if constexpr (kE8) static_cast<uint8_t*>(as)[at] = (uint8_t)code;
      else static_cast<float*>(as)[at] = s;
    }
  }
}

template <int kIn, bool kE8, int kWaves, int kChunks>
void run(const RmsNormArgs& a, hipStream_t stream) {
  constexpr int kRows = kWaves == 1 ? 4 : 1;
  hipLaunchKernelGGL((rmsnorm_quant_kernel<kIn, kE8, kWaves, kChunks>), dim3((unsigned)((a.M + kRows - 1) / kRows)),
                     dim3(kWaves == 1 ? 256 : kWaves * 64), 0, stream, a.x, a.ldx, a.res, a.ld_res, a.w, a.eps, a.h,
                     a.ld_h, a.q, a.ldq, a.as, a.ld_as, a.M, a.H);
}

// By the row's length alone, so that a row's result does not depend on how many there are. A wave for every 512
// elements answers a single row soonest, and long batches are slower where 16 waves wait for each other (bf16 with a
// residual, us of GPU time for 1 and for 8192 rows): 2048 elements, one wave 5.1 and 22.2, two 3.6 and 21.3, four
// 3.1 and 21.9; 4096, one 8.3 and 42.0, four 3.8 and 38.5, eight 3.3 and 39.3, sixteen 3.3 and 50.2; 7168, four 5.2
// and 83, eight 4.0 and 79, sixteen 3.7 and 86.5; 12288, eight 4.8 and 131, sixteen 4.2 and 135.
template <int kIn, bool kE8>
void choose(const RmsNormArgs& a, hipStream_t stream) {
  const int pieces = (a.H + 511) / 512;  // 64 lanes of 8 elements
  if (pieces <= 1) run<kIn, kE8, 1, 1>(a, stream);
  else if (pieces <= 2) run<kIn, kE8, 2, 1>(a, stream);
  else if (pieces <= 4) run<kIn, kE8, 4, 1>(a, stream);
  else if (pieces <= 8) run<kIn, kE8, 8, 1>(a, stream);
  else if (pieces <= 16) run<kIn, kE8, 8, 2>(a, stream);
  else if (pieces <= 32) run<kIn, kE8, 16, 2>(a, stream);
  else if (pieces <= 64) run<kIn, kE8, 16, 4>(a, stream);
  else run<kIn, kE8, 16, 8>(a, stream);
}

}  // namespace

hipError_t launch_rmsnorm_quant(const RmsNormArgs& a, int x_dtype, bool e8, hipStream_t stream) {
  if (x_dtype == kInBf16) e8 ? choose<kInBf16, true>(a, stream) : choose<kInBf16, false>(a, stream);
  else if (x_dtype == kInF16) e8 ? choose<kInF16, true>(a, stream) : choose<kInF16, false>(a, stream);
  else e8 ? choose<kInF32, true>(a, stream) : choose<kInF32, false>(a, stream);
  return hipGetLastError();
}

}  // namespace bfp8
