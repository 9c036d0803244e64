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

// The normal distribution's tail, Phi(-a) = exp(-a^2 / 2) t Q(t) with t =
// 1 / (a + 2) and Q a minimax fit of degree 9, for all a >= 0 within 5.4e-8 of
// its size: both factors fall with a as the tail does, so that nothing cancels
// where Phi(z) is small.  One exponential, one reciprocal and some fifteen
// operations, without the branches of a library erf.  Returns t Q(t); *e
// receives exp(-a^2 / 2).
//
// gelu(z) = max(z, 0) - a Phi(-a) and gelu'(z) = w for z < 0, 1 - w else, with
// w = exp(-a^2 / 2) (t Q(t) - a / sqrt(2 pi)), a = |z|.  In half steps u = 2^-24
// of the value, Phi(-a) is within 1.25 a^2 + 14 (the exponential's argument
// rounds twice: 1e-5 at a = 12); 1 + erf in FP32 is 1e-5 off at a = 3 and has
// lost all of Phi at 6.  Over normal z, gelu's root mean square error measured
// 0.52 u (0.5 z (1 + erf(z / sqrt 2)) in FP32: 0.65), its slope's 0.72 u.
__device__ __forceinline__ float normal_tail(float a, float* e) {
  const float t = __builtin_amdgcn_rcpf(__fadd_rn(a, 2.0f));
  float q = __builtin_fmaf(t, -28.0450525f, 103.455102f);
  q = __builtin_fmaf(t, q, -156.656782f);
  q = __builtin_fmaf(t, q, 122.406434f);
  q = __builtin_fmaf(t, q, -47.8484196f);
  q = __builtin_fmaf(t, q, 5.761188f);
  q = __builtin_fmaf(t, q, -0.122317093f);
  q = __builtin_fmaf(t, q, 1.26324963f);
  q = __builtin_fmaf(t, q, 0.795226992f);
  q = __builtin_fmaf(t, q, 0.398987228f);
  *e = __builtin_amdgcn_exp2f(__fmul_rn(__fmul_rn(a, a), -0.5f * kLog2e));
  return __fmul_rn(t, q);
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
  float e;
  switch (act) {
    case kActRelu: return __builtin_elementwise_maximum(z, 0.0f);   // NaN stays NaN
    case kActGelu: {
      // -0 for max's bound keeps the sign of z Phi(z); +Inf meets a Phi(-a) = 0
      // as the largest finite a, -Inf as itself (NaN)
      const float p = normal_tail(__builtin_fabsf(z), &e);
      return __builtin_fmaf(-__builtin_fabsf(__builtin_fminf(z, 0x1.fffffep+127f)), __fmul_rn(p, e),
                            __builtin_fmaxf(z, -0.0f));
    }
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
      const float a = __builtin_fabsf(z), p = normal_tail(a, &e);
      const float w = __fmul_rn(e, __builtin_fmaf(a, -0.39894228f, p));
      return z < 0.0f ? w : 1.0f - w;
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
