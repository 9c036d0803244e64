// Activations of the Linear epilogue and their slopes, in FP32 (gfx950).
//
//   none  z                      gelu       z Phi(z), Phi the normal distribution function
//   relu  max(z, 0)              gelu_tanh  z sigma(2 c (z + a z^3)), c = sqrt(2 / pi), a = 0.044715
//   silu  z sigma(z)             (0.5 (1 + tanh(u)) = sigma(2 u))
//
// The hardware exponential and reciprocal are about 1 ulp each; the
// exponential's argument carries the rounding of x log2(e), so sigma has a
// relative error of about |x| 2^-24 where it is small.  An infinite z follows
// the formulas: +Inf gives +Inf, and -Inf the NaN of -Inf * 0 for gelu,
// gelu_tanh and silu.
#pragma once

#include <hip/hip_runtime.h>

namespace fp8mot {

enum Act { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// 1 / (1 + exp(-x)): exp overflows to +Inf for very negative x and its
// reciprocal is 0.
__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(__fadd_rn(1.0f, __expf(-x)));
}

// Phi(z) = erfc(-z / sqrt 2) / 2 with Abramowitz and Stegun's formula 7.1.26,
// erfc(x) ~ (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 + p x), x >= 0, within
// 1.5e-7: one exponential, one reciprocal and six FMAs, where a library erf
// evaluates two polynomial branches.  The factor exp(-x^2) keeps the tail's
// relative accuracy, which 1 + erf would lose to cancellation.  *e receives
// exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float x = __fmul_rn(__builtin_fabsf(z), 0.70710678f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
  float p = __builtin_fmaf(t, 1.061405429f, -1.453152027f);
  p = __builtin_fmaf(t, p, 1.421413741f);
  p = __builtin_fmaf(t, p, -0.284496736f);
  p = __builtin_fmaf(t, p, 0.254829592f);
  *e = __expf(-__fmul_rn(x, x));
  const float half = __fmul_rn(__fmul_rn(0.5f * t, p), *e);   // erfc(|z| / sqrt 2) / 2
  return z < 0.0f ? half : 1.0f - half;
}

// 2 c (z + a z^3) with z held to [-16, 16] (NaN stays), beyond which sigma of
// it is 0 or 1 to the last bit: keeps z^3 and the slope's z^2 finite.
__device__ __forceinline__ float clamp16(float z) {
  return __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -16.0f), 16.0f);
}
__device__ __forceinline__ float gelu_tanh_arg(float zc) {
  return __fmul_rn(1.5957691f * zc, __builtin_fmaf(0.044715f * zc, zc, 1.0f));
}

__device__ __forceinline__ float act_value(float z, int act) {
  float e;
  switch (act) {
    case kActRelu: return __builtin_elementwise_maximum(z, 0.0f);   // NaN stays NaN
    case kActGelu: return __fmul_rn(z, normal_cdf(z, &e));
    case kActGeluTanh: return __fmul_rn(z, sigmoid_f32(gelu_tanh_arg(clamp16(z))));
    case kActSilu: return __fmul_rn(z, sigmoid_f32(z));
    default: return z;
  }
}

// d act / dz.  relu's slope at 0 is 0; a NaN z gives NaN for every activation
// with a slope of its own.
__device__ __forceinline__ float act_slope(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.0f ? 1.0f : (z == z ? 0.0f : z);
    case kActGelu: {
      float e;
      const float p = normal_cdf(z, &e);
      return __builtin_fmaf(z * 0.39894228f, e, p);
    }
    case kActGeluTanh: {
      const float zc = clamp16(z);
      const float p = sigmoid_f32(gelu_tanh_arg(zc));
      const float du = 1.5957691f * __builtin_fmaf(0.134145f * zc, zc, 1.0f);
      return __builtin_fmaf(__fmul_rn(zc * p, 1.0f - p), du, p);
    }
    case kActSilu: {
      const float p = sigmoid_f32(z);
      return __fmul_rn(p, __builtin_fmaf(z, 1.0f - p, 1.0f));
    }
    default: return 1.0f;
  }
}

}  // namespace fp8mot
