// The 8-bit integer products (internal to libbfp8; arguments are validated by the C-ABI layer before any
// launcher is called).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bfp8 {

constexpr int kInt8MaxK = 65536;  // a sum of 65536 products of codes stays within 2^30

hipError_t launch_quant_act_int8(const void* x, int x_dtype, int64_t M, int64_t K, int64_t ldx, int8_t* q, int64_t ldq,
                                 float* s, hipStream_t stream);

struct Int8GemmArgs {
  const int8_t* a;  // [M][lda] activation codes
  int64_t lda;
  const float* as;  // [M] scale of each token
  const int8_t* b;  // [N][ldb] weight codes
  int64_t ldb;
  const float* bs;       // [N] scale of each channel
  const uint16_t* bias;  // [N] in the output's type, or NULL
  uint16_t* c;           // [M][ldc] bf16, or fp16 with out_f16
  int64_t ldc;
  int M, N, K;
  bool out_f16;
};
hipError_t launch_gemm_int8(const Int8GemmArgs& args, hipStream_t stream);
// The tile of the kernel that launch_gemm_int8 chooses (bn channels x bm tokens), and whether its waves split K.
struct Int8Choice {
  int bn, bm;
  bool splits_k;
};
Int8Choice choose_gemm_int8(int64_t M, int64_t N, int64_t K);
// The linear layer in one launch, for the sizes that linear_int8_fuses accepts (args.a, lda and as unused).
bool linear_int8_fuses(int64_t M, int64_t N, int64_t K);
hipError_t launch_linear_int8(const Int8GemmArgs& args, const uint16_t* x, int64_t ldx, hipStream_t stream);

}  // namespace bfp8
