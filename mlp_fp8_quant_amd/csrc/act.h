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

// 1 / (1 + 2^x), for sigma(y) = 1 / (1 + 2^(-y log2 e)): the power overflows
// to +Inf for large x and its reciprocal is 0.
__device__ __forceinline__ float rcp_1p_exp2(float x) {
  return __builtin_amdgcn_rcpf(__fadd_rn(1.0f, __builtin_amdgcn_exp2f(x)));
}
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float sigmoid_f32(float x) { return rcp_1p_exp2(__fmul_rn(x, -kLog2e)); }

// Phi(z) = erfc(-z / sqrt 2) / 2 with Abramowitz and Stegun's formula 7.1.26,
// erfc(x) ~ (a1 t + .. + a5 t^5) exp(-x^2), t = 1 / (1 + p x), x >= 0, within
// 1.5e-7: one exponential, one reciprocal and a dozen operations, where a
// library erf evaluates two polynomial branches.  The factor exp(-x^2) keeps
// the tail's relative accuracy, which 1 + erf would lose to cancellation.
// The constants below are the formula's with 1/sqrt 2, 1/2 and log2 e folded
// in.  *e receives exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.23164190f, __builtin_fabsf(z), 1.0f));
  float p = __builtin_fmaf(t, 0.530702715f, -0.726576014f);
  p = __builtin_fmaf(t, p, 0.710706871f);
  p = __builtin_fmaf(t, p, -0.142248368f);
  p = __builtin_fmaf(t, p, 0.127414796f);
  *e = __builtin_amdgcn_exp2f(__fmul_rn(z, __fmul_rn(z, -0.5f * kLog2e)));
  const float half = __fmul_rn(__fmul_rn(t, p), *e);   // erfc(|z| / sqrt 2) / 2
  return z < 0.0f ? half : 1.0f - half;
}

// sigma(2 c (z + a z^3)) and the slope of its argument.  z is held to
// [-16, 16], beyond which sigma is 0 or 1 to the last bit: that keeps z^3
// and z^2 finite (a NaN z turns into a bound here and is a NaN again in the
// product with z).
__device__ __forceinline__ float gelu_tanh_sigma(float z, float* zc_out) {
  const float zc = __builtin_amdgcn_fmed3f(z, -16.0f, 16.0f);
  *zc_out = zc;
  const float p = __builtin_fmaf(__fmul_rn(zc, zc), -1.5957691f * 0.044715f * kLog2e, -1.5957691f * kLog2e);
  return rcp_1p_exp2(__fmul_rn(zc, p));
}

__device__ __forceinline__ float act_value(float z, int act) {
  float e;   // not needed here
  switch (act) {
    case kActRelu: return __builtin_elementwise_maximum(z, 0.0f);   // NaN stays NaN
    case kActGelu: return __fmul_rn(z, normal_cdf(z, &e));
    case kActGeluTanh: return __fmul_rn(z, gelu_tanh_sigma(z, &e));
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
      float zc;
      const float p = gelu_tanh_sigma(z, &zc);
      const float du = __builtin_fmaf(zc * zc, 1.5957691f * 0.134145f, 1.5957691f);
      const float s = __builtin_fmaf(__fmul_rn(zc * p, 1.0f - p), du, p);
      return z == z ? s : z;
    }
    case kActSilu: {
      const float p = sigmoid_f32(z);
      return __fmul_rn(p, __builtin_fmaf(z, 1.0f - p, 1.0f));
    }
    default: return 1.0f;
  }
}

// The same over n values: the switch is outside the loops, so that only the
// chosen one's instructions are fetched.
template <int n>
__device__ __forceinline__ void act_all(float* z, int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = act_value(z[i], kActRelu);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = act_value(z[i], kActGelu);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = act_value(z[i], kActGeluTanh);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = act_value(z[i], kActSilu);
      break;
    default: break;
  }
}

template <int n>
__device__ __forceinline__ void slope_all(float* z, int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = act_slope(z[i], kActRelu);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = act_slope(z[i], kActGelu);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = act_slope(z[i], kActGeluTanh);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = act_slope(z[i], kActSilu);
      break;
    default:
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] = 1.0f;
  }
}

}  // namespace fp8mot
