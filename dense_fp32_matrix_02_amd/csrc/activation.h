// Activations and their slopes in FP32.
#pragma once

#include "fp8_internal.h"

namespace sgemm_impl {
namespace {

// exp(x) for x <= 0: the exponent in base 2 as a rounded product and what its
// rounding lost, which enters as a factor 1 + r ln 2. Without it the result
// would be off by |x| half-units in the last place. The hardware's power of two has
// no subnormal results: from x = -87.34 down (2^-126) the result is zero. The bound
// of -104 keeps an infinity out of the fused products.
__device__ __forceinline__ float exp_below(float x) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;
  x = fmaxf(x, -104.0f);
  const float t = x * kLog2e;
  const float r = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(e, r * kLn2, e);
}

// s = 1 / (1 + exp(-x)) and c = 1 - s, each without a difference of like numbers.
__device__ __forceinline__ void sigmoid(float x, float& s, float& c) {
  const float e = exp_below(-fabsf(x));
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  s = x < 0.0f ? e * r : r;
  c = x < 0.0f ? r : e * r;
}

constexpr float kLog2eF = 1.4426950408889634f, kMost = 3.4028234663852886e38f;

// The normal distribution's integral up to p, and its density at p. With
// x = |p|: Phi(-x) = exp(-x^2/2) f(1 / (1 + 0.26 x)), f(t) t times a polynomial
// fitted to erfc(x / sqrt 2) exp(x^2/2) / 2 on 0 <= x <= 14.5 for the least
// relative error, 2.8e-8 (beyond, the exponential is zero). The exponent's
// roundings cost the tail x^2/2 steps of its own size.
__device__ __forceinline__ void normal(float p, float& below, float& density) {
  const float x = fabsf(p);
  const float e = __builtin_amdgcn_exp2f(p * p * (-0.5f * kLog2eF));
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.26f, x, 1.0f));
  float f = 0.030230301335811942f;
  f = __builtin_fmaf(f, t, -0.15149443888002528f);
  f = __builtin_fmaf(f, t, 0.24873321057962977f);
  f = __builtin_fmaf(f, t, -0.1477893502468334f);
  f = __builtin_fmaf(f, t, 0.15875876440857434f);
  f = __builtin_fmaf(f, t, 0.05196482062752984f);
  f = __builtin_fmaf(f, t, 0.10278868211470069f);
  f = __builtin_fmaf(f, t, 0.10305097391778659f);
  f = __builtin_fmaf(f, t, 0.10375702210377379f);
  const float tail = e * (f * t);
  below = p < 0.0f ? tail : 1.0f - tail;
  density = 0.3989422804014327f * e;
}

// p within -most .. most; a NaN becomes a number (one instruction), or stays one.
__device__ __forceinline__ float limited(float p, float most) { return __builtin_amdgcn_fmed3f(p, -most, most); }
__device__ __forceinline__ float within(float p, float most) { return p < -most ? -most : p > most ? most : p; }

// Twice sqrt(2/pi), and the cubic term's share, of GELU's tanh form:
// p s with s = sigmoid(2 u), u = sqrt(2/pi) (p + 0.044715 p^3).
constexpr float kTwoA = 1.5957691216057308f, kB = 0.044715f;

// value = act(p) and slope = act'(p), at the infinities their limits; a NaN
// gives NaN (but NONE's slope, 1). Beyond the bounds below the exponential is zero,
// s, or Phi, 0 or 1, and the other factor is cut, so that no infinity meets a zero. An s
// or Phi under 2^-126 is 0: SiLU of -87.34 to -104 is zero where it is -1.0e-36 to
// -7e-44.
template <int ACT>
__device__ __forceinline__ void activation(float p, float& value, float& slope) {
  if constexpr (ACT == SGEMM_MI355_NONE) {
    value = p, slope = 1.0f;
  } else if constexpr (ACT == SGEMM_MI355_RELU) {
    value = p <= 0.0f ? 0.0f : p;
    slope = p <= 0.0f ? 0.0f : p > 0.0f ? 1.0f : p;
  } else if constexpr (ACT == SGEMM_MI355_SILU) {
    float s, c;
    sigmoid(p, s, c);
    value = (p < -104.0f ? -104.0f : p) * s;
    slope = __builtin_fmaf(within(p, 104.0f) * c, s, s);  // s (1 + p (1 - s))
  } else if constexpr (ACT == SGEMM_MI355_GELU) {
    float below, density;
    normal(p, below, density);
    value = fmaxf(p, -kMost) * below;
    slope = __builtin_fmaf(limited(p, 20.0f), density, below);
  } else {
    const float q = within(p, 12.0f), q2 = q * q;
    float s, c;
    sigmoid(kTwoA * q * __builtin_fmaf(kB, q2, 1.0f), s, c);
    value = (p > 0.0f ? p : q) * s;
    slope = __builtin_fmaf(q * c * (kTwoA * __builtin_fmaf(3.0f * kB, q2, 1.0f)), s, s);
  }
}

// act'(p) for P of 16 bits, in fewer instructions where a sigmoid is all of it
// (8192 x 8192 bf16, an epilogue's way back: SiLU 74 us against 79, the tanh form
// 74 against 78). s = 1 / (1 + exp(-x)) as it stands, so that s and 1 - s lose |x|
// steps of FP32 where they are small, and the slope, which has their product, a few
// steps of 1: the bias' gradient is an FP32 sum of these. (A polynomial for GELU off by
// 8.6e-6 saves 1 us of 76 and puts that sum off by 2.6e-6.)
template <int ACT>
__device__ __forceinline__ float slope16(float p) {
  if constexpr (ACT == SGEMM_MI355_SILU) {
    const float e = __builtin_amdgcn_exp2f(p * -kLog2eF), s = __builtin_amdgcn_rcpf(1.0f + e);
    return __builtin_fmaf(limited(p, 104.0f) * (fminf(e, kMost) * s), s, s);  // an infinite e has s = 0
  } else if constexpr (ACT == SGEMM_MI355_GELU_TANH) {
    constexpr float a = -kTwoA * kLog2eF, b = -kTwoA * kLog2eF * kB;
    const float e = __builtin_amdgcn_exp2f(p * __builtin_fmaf(b, p * p, a)), s = __builtin_amdgcn_rcpf(1.0f + e);
    const float q = limited(p, 12.0f);
    return __builtin_fmaf(q * (fminf(e, kMost) * s) * __builtin_fmaf(3.0f * kTwoA * kB, q * q, kTwoA), s, s);
  } else {
    float value, slope;
    activation<ACT>(p, value, slope);
    return slope;
  }
}

// The values of W arguments of an activation that the whole launch shares, in
// little code: it is fetched once for each tile of a product. SiLU and the tanh
// form of GELU are one expression, p sigmoid(a p + b p^3), with other numbers.
// SHORT: for results of 16 bits, s = 1 / (1 + exp(-x)) as it stands, which loses
// |x| steps of FP32 where it is small and takes a third of the instructions (8192 x 8192
// results with K 4096, the tanh form, with P: 246 us against 257). A residual that
// cancels act(p) shows no more error than with the long form (of act(p) rounded to
// fp16, |p| up to 8: 3.5e-4 on average of what is left, 2.0e-4 (SiLU) and 5.0e-4 (tanh)).
template <bool SHORT, int W>
__device__ __forceinline__ void activate(int act, float (&v)[W]) {
  if (act == SGEMM_MI355_SILU || act == SGEMM_MI355_GELU_TANH) {
    const bool tanh = act == SGEMM_MI355_GELU_TANH;
    if constexpr (SHORT) {
      const float a = tanh ? -kTwoA * kLog2eF : -kLog2eF, b = tanh ? -kTwoA * kLog2eF * kB : 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        // The square is cut, so that SiLU's b = 0 meets no infinity.
        const float p = v[i], q2 = fminf(p * p, kMost);
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(p * __builtin_fmaf(b, q2, a)));
        v[i] = fmaxf(p, -kMost) * s;
      }
    } else {
      const float most = tanh ? 12.0f : 104.0f, a = tanh ? kTwoA : 1.0f, b = tanh ? kB : 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float p = v[i], q = limited(p, most);
        float s, c;
        sigmoid(a * q * __builtin_fmaf(b, q * q, 1.0f), s, c);
        v[i] = (p < -most ? -most : p) * s;
      }
    }
  } else if (act == SGEMM_MI355_GELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      float value, slope;
      activation<SGEMM_MI355_GELU>(v[i], value, slope);
      v[i] = value;
    }
  } else if (act == SGEMM_MI355_RELU) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = v[i] <= 0.0f ? 0.0f : v[i];
  }
}

}  // namespace
}  // namespace sgemm_impl
