// FP8 with an FP32 scale for each block of 128 (gfx950): the scale of a block
// from its largest magnitude, and the quotients that its codes encode.
//
//   s = amax / 448,  q = e4m3(v / s), both divisions correctly rounded
//
// A zero block has scale 0 and keeps its signed zeros; a block that holds a
// NaN has a NaN scale and NaN codes, one with an infinity an infinite scale.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace fp8mot {
namespace block {

constexpr int kBlock = 128;

// Magnitudes are compared as integers: in order for numbers, and any NaN above
// them all.
__device__ __forceinline__ int magnitude(float v) { return (int)(__float_as_uint(v) & 0x7FFFFFFFu); }
__device__ __forceinline__ int max8(const float* f) {
  int m = magnitude(f[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) m = max(m, magnitude(f[k]));
  return m;
}

// The largest over each 16 lanes, in each of them.
template <int CTRL>
__device__ __forceinline__ int dpp_max(int v) {
  return max(v, __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ int max16(int v) {
  v = dpp_max<0xB1>(v);        // quad_perm [1,0,3,2]
  v = dpp_max<0x4E>(v);        // quad_perm [2,3,0,1]
  v = dpp_max<0x141>(v);       // row_half_mirror
  return dpp_max<0x140>(v);    // row_mirror
}

__device__ __forceinline__ float scale_of(int amax) { return __int_as_float(amax) / 448.0f; }

// f = f / s for the encoder (see div_by_scale); r = 1 / s.
template <int N>
__device__ __forceinline__ void quotients(float* f, float s, float r) {
  if (div_by_scale_ok(s)) {
    const float lim = 1024.0f * s;
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = div_by_scale(f[k], s, r, lim);
  } else if (s != 0.0f) {
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = f[k] / s;
  }
}

template <int N>
__device__ __forceinline__ void quotients(float* f, float s) {
  quotients<N>(f, s, 1.0f / s);
}

}  // namespace block
}  // namespace fp8mot
