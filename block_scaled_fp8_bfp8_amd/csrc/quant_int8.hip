// Per-token quantization of activations to 8-bit integers.
//
// HBM-bound: x is read once, q written once. A row lives in the registers of the waves that share it, 8
// elements a thread and chunk, as loaded; the waves exchange its largest element through LDS. Measured: 8192 x 5120 bf16 22 us (126 MB at
// 5.7 TB/s; a copy of 1 GiB reaches 5.2), one row of 7168 2.0 us in a kernel trace.
#include "device_int8.h"
#include "int8.h"
#include "launch.h"

namespace bfp8 {

namespace {

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
  const Int8Scale scale(amax);
  if (tid == 0 && row_ok) s[m] = scale.value();

#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int col = (c * kThreads + tid) * 8;
    if (col >= K || !row_ok) continue;
    *reinterpret_cast<uint2*>(q + m * ldq + col) = row_codes(v[c], scale);
  }
}

template <int kIn, int kWaves, int kChunks>
void run(const void* x, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq, float* s, hipStream_t stream) {
  constexpr int kRows = kWaves == 1 ? 4 : 1;
  constexpr int64_t kMost = (int64_t)1 << 21;  // rows a launch: its threads stay below 2^32
  const int64_t row_bytes = ldx * (kIn == kInF32 ? 4 : 2);
  for (int64_t m = 0; m < M; m += kMost) {
    const int64_t rows = M - m < kMost ? M - m : kMost;
    hipLaunchKernelGGL((quant_int8_kernel<kIn, kWaves, kChunks>), dim3((unsigned)((rows + kRows - 1) / kRows)),
                       dim3(kWaves == 1 ? 256 : kWaves * 64), 0, stream, static_cast<const uint8_t*>(x) + m * row_bytes, row_bytes,
                       q + m * ldq, ldq, s + m, (int)rows, (int)K);
  }
}

// Many rows (more than run at once): as few waves a row as hold it in two chunks each, so that the fewest lanes have nothing to do and more
// rows are under way. Few: a wave for every 512 elements, eight at most up to 8192. (us in a captured graph, as few and as many waves: 16384 x
// 2560 24.4 and 34.1, 8192 x 4096 20.8 and 23.2, 4096 x 4096 10.5 and 11.9, 2100 x 4096 7.5 and 8.0, 4096 x 512 3.4 and 3.7; 1024 x 4096 5.4 and 5.2,
// 1536 x 1024 4.0 and 3.5. One border for every length: rows of 513 to 1536 elements, of which more fit the card at once, lose up to 0.6 us just past it,
// 2100 x 1024 4.3 and 3.8, 3000 x 1024 4.6 and 4.3, 2049 x 1536 4.7 and 4.4, and gain from about 4096 and 3000 rows on.)
template <int kIn>
void choose(const void* x, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq, float* s, hipStream_t stream) {
  const int64_t pieces = (K + 511) / 512;  // 64 lanes of 8 elements
  if (M > 2048 && pieces <= 14) {
    switch ((pieces + 1) / 2) {
      case 1: return run<kIn, 1, 2>(x, M, K, ldx, q, ldq, s, stream);
      case 2: return run<kIn, 2, 2>(x, M, K, ldx, q, ldq, s, stream);
      case 3: return run<kIn, 3, 2>(x, M, K, ldx, q, ldq, s, stream);
      case 4: return run<kIn, 4, 2>(x, M, K, ldx, q, ldq, s, stream);
      case 5: return run<kIn, 5, 2>(x, M, K, ldx, q, ldq, s, stream);
      case 6: return run<kIn, 6, 2>(x, M, K, ldx, q, ldq, s, stream);
      default: return run<kIn, 7, 2>(x, M, K, ldx, q, ldq, s, stream);
    }
  }
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
