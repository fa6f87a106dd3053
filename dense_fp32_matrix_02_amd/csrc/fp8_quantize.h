// Quantisation of a block to e4m3, shared by the quantisers and the kernels whose
// last step it is. For a block with largest magnitude m: s = max(m, 2^-64) / 448
// and q = e4m3(x / s), the quotient rounded to FP32 first.
#pragma once

#include "fp8_internal.h"

namespace sgemm_impl {
namespace {

constexpr float kTop = 448.0f;
constexpr float kLeast = 0x1p-64f;

// The magnitude's bits order like the magnitudes, with infinities and then
// NaNs above all numbers, so their integer maximum keeps a NaN.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale of a block whose largest magnitude has these bits; NaN where the
// block holds a NaN or an infinity.
__device__ __forceinline__ float scale_of(uint32_t most) {
  if (most >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return fmaxf(__uint_as_float(most), kLeast) / kTop;
}

// x / s rounded to FP32, for r = 1 / s rounded: two residual corrections of
// the product x*r. The first brings it within one unit in the last place; the
// second, with r correctly rounded, rounds it correctly (Markstein). With
// s >= 2^-64/448 and |x| <= 448 s no residual that could matter to a quotient
// of 2^-10 or more (the rest round to zero) leaves FP32's range.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  float q = x * r;
  q = __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
  return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
}

// Eight values as e4m3, value i in byte i.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float s) {
  const float r = 1.0f / s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s, r);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return uint2{(uint32_t)lo, (uint32_t)hi};
}

template <bool ONCE = false>
__device__ __forceinline__ void store_bytes(uint8_t* p, uint2 b, int valid) {
  typedef uint32_t words __attribute__((ext_vector_type(2), aligned(1)));
  if (valid >= 8) {
    const words w = {b.x, b.y};
    if constexpr (ONCE) __builtin_nontemporal_store(w, (words*)p);
    else *(words*)p = w;
  } else {
    const uint64_t w = ((uint64_t)b.y << 32) | b.x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = (uint8_t)(w >> (8 * i));
  }
}

}  // namespace
}  // namespace sgemm_impl
