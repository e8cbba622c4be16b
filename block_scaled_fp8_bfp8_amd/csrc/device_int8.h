// Per-token quantization to 8-bit integers, as the quantizer and the linear layer's small-batch kernel do it (bit for bit alike).
//
// For every row m of x [M][K]:  a = max(max_k |x|, 1e-10),  s = a / 127 (correctly rounded),
// q = 127 x / a rounded to the nearest integer, ties to even, of the exact quotient.
// In float32, t = x * (127 / a) is off by at most 2^-23 of |t| <= 127 and so is decided unless it lies
// within 2^-16 of the middle of two integers; there 127 x and (middle) a are compared exactly. (bf16 and fp16 tokens hold many exact middles: a token whose largest element is 127 times a
// power of two, for one.) A row with an infinite or NaN element has a NaN scale and zero codes.
//
#pragma once

#include "device_latent.h"
#include "launch.h"

namespace bfp8 {

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

// x rounded where t, its quotient in float32, is too near the middle of two integers to tell: the sign of 127 x - middle a, both
// products as a rounded value and what it leaves (a few bits each, so that every difference is exact; over 2^8, as 127 x may pass float32).
__device__ __forceinline__ float decide(float x, float a, float t) {
#pragma clang fp contract(off)
  const float below = floorf(t), middle = below + 0.5f;
  x *= 0x1p-8f, a *= 0x1p-8f;
  const float p = 127.0f * x, q = middle * a;
  const float d = (p - q) + (fmaf(127.0f, x, -p) - fmaf(middle, a, -q));
  return d > 0.0f || (d == 0.0f && ((int)below & 1)) ? below + 1.0f : below;
}

// A row's scale, from its largest magnitude (NaN if an element is NaN).
struct Int8Scale {
  float top, factor;
  bool finite;
  __device__ __forceinline__ explicit Int8Scale(float amax)
      : top(fmaxf(amax, 1e-10f)), factor(0.f), finite(amax < __builtin_inff()) {
    if (finite) factor = 127.0f / top;
  }
  __device__ __forceinline__ float value() const { return finite ? top / 127.0f : __builtin_nanf(""); }
};

// The codes of 8 elements of the row. Adding 1.5 * 2^23 rounds to the nearest integer, ties to even, and leaves its code in the
// low byte.
template <int kIn>
__device__ __forceinline__ uint2 row_codes(const Piece<kIn>& v, const Int8Scale& s) {
#pragma clang fp contract(off)
  constexpr float kMagic = 0x1.8p23f;
  float r[8];
  float far = 0.f;  // the largest distance to a code
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = element<kIn>(v, i) * s.factor;
    r[i] = t + kMagic;
    far = fmaxf(far, fabsf(t - (r[i] - kMagic)));
  }
  if (__builtin_expect(far > 0.5f - 0x1p-16f, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = element<kIn>(v, i), t = e * s.factor;
      if (fabsf(t - (r[i] - kMagic)) > 0.5f - 0x1p-16f) r[i] = decide(e, s.top, t) + kMagic;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t* b = reinterpret_cast<const uint32_t*>(r) + 4 * h;
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
    w[h] = s.finite ? lo | hi << 16 : 0u;
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace bfp8
