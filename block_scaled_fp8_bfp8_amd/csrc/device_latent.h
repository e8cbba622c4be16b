// Device-side helpers of the norm, cache and latent-attention kernels, beyond those of device_common.h.
#pragma once

#include "device_common.h"

namespace bfp8 {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

// Two float32 values as a pair of bf16 (low half first), rounded to nearest even by the hardware
// conversion.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2f f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, v2bf));
}

// The larger of two values, NaN if either is NaN (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Clamp to the e4m3 range; NaN stays NaN. The e4m3 conversion does not saturate by itself.
__device__ __forceinline__ float clamp_e4m3(float y) {
  return __builtin_elementwise_minimum(__builtin_elementwise_maximum(y, -448.0f), 448.0f);
}

// Four values as e4m3 codes (round to nearest even), first in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3(const float* y) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
}

// 8 bf16 values as float32.
__device__ __forceinline__ void bf16x8_values(const uint4& r, float* f) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// 8 e4m3 codes as float32.
__device__ __forceinline__ void e4m3x8_values(const uint2& c, float* f) {
  f[0] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 0);
  f[1] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 1);
  f[2] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 2);
  f[3] = __builtin_amdgcn_cvt_f32_fp8((int)c.x, 3);
  f[4] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 0);
  f[5] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 1);
  f[6] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 2);
  f[7] = __builtin_amdgcn_cvt_f32_fp8((int)c.y, 3);
}

// The value 2^(code - 127) of a UE8M0 code (255: NaN; 0: 2^-127, a float32 subnormal).
__device__ __forceinline__ float e8_value(uint32_t code) {
  return code == 255u ? __builtin_nanf("") : code == 0u ? __uint_as_float(0x400000u) : __uint_as_float(code << 23);
}

// 16 bytes of every lane from its own global address, or from sbase + voff, to LDS byte lds + 16 * lane; awaited
// with wait_copies(). For kernels in which nothing else uses M0 (gfx950's LDS instructions do not read it): it is
// not saved.
__device__ __forceinline__ void copy16_m0(const uint8_t* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "s"(lds) : "memory");
}
__device__ __forceinline__ void copy16_m0(const void* sbase, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %1, %0" : : "s"(sbase), "v"(voff), "s"(lds) : "memory");
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // 1, 2, 4, 8 lanes up within 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 to the next 16, of the odd rows
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to the upper half
  return v;
}

template <int kValue>
struct Const {
  static constexpr int v = kValue;
};
// Sum over the lanes of a wave, and the largest of values >= 0 (NaN if one is NaN), in every lane: the
// steps of wave_scan, whose last lane then holds the whole.
template <typename F>
__device__ __forceinline__ float wave_fold(float v, F f) {
  auto moved = [](float x, auto ctrl, auto rows) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), decltype(ctrl)::v, decltype(rows)::v, 0xf, false));
  };
  v = f(v, moved(v, Const<0x111>{}, Const<0xf>{}));
  v = f(v, moved(v, Const<0x112>{}, Const<0xf>{}));
  v = f(v, moved(v, Const<0x114>{}, Const<0xf>{}));
  v = f(v, moved(v, Const<0x118>{}, Const<0xf>{}));
  v = f(v, moved(v, Const<0x142>{}, Const<0xa>{}));
  v = f(v, moved(v, Const<0x143>{}, Const<0xc>{}));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_fold(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_fold(v, [](float a, float b) { return max_nan(a, b); });
}

}  // namespace bfp8
