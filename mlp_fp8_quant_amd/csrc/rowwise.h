// Pieces of the kernels that stream rows of floats: groups of eight
// consecutive elements of a row, sums over a wave or a workgroup, E4M3 and BF16
// output.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace fp8mot {
namespace rows {

// Eight elements of a row may start at any element of it: global accesses need
// no alignment beyond the element's on this target.
typedef uint32_t u4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f4a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u2a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

// Raw eight elements: BF16 in one register quad, FP32 in two.
template <bool F32>
struct Raw8 {
  u4 q[F32 ? 2 : 1];
};

// Elements i .. i + 7 of a row of n; past its end zeros, or with LAST the row's
// last element again.  WHOLE: the row does not end before them.
template <bool F32, bool WHOLE = false, bool LAST = false>
__device__ __forceinline__ Raw8<F32> load8(const void* row, int64_t i, int64_t n) {
  Raw8<F32> r;
  if (WHOLE || i + 8 <= n) {
    if constexpr (F32) {
      const float* p = static_cast<const float*>(row) + i;
      r.q[0] = __builtin_bit_cast(u4, (f4)(*reinterpret_cast<const f4a4*>(p)));
      r.q[1] = __builtin_bit_cast(u4, (f4)(*reinterpret_cast<const f4a4*>(p + 4)));
    } else {
      r.q[0] = *reinterpret_cast<const u4a2*>(static_cast<const uint16_t*>(row) + i);
    }
  } else if constexpr (LAST) {
    auto at = [&](int k) { return i + k < n ? i + k : n - 1; };
#pragma unroll
    for (int k = 0; k < (F32 ? 8 : 4); ++k) {
      uint32_t v;
      if constexpr (F32) {
        v = static_cast<const uint32_t*>(row)[at(k)];
      } else {
        v = static_cast<const uint16_t*>(row)[at(2 * k)];
        v |= (uint32_t) static_cast<const uint16_t*>(row)[at(2 * k + 1)] << 16;
      }
      r.q[k >> 2][k & 3] = v;
    }
  } else {
#pragma unroll
    for (int k = 0; k < (F32 ? 8 : 4); ++k) {
      uint32_t v = 0;
      if constexpr (F32) {
        if (i + k < n) v = static_cast<const uint32_t*>(row)[i + k];
      } else {
        if (i + 2 * k < n) v = static_cast<const uint16_t*>(row)[i + 2 * k];
        if (i + 2 * k + 1 < n) v |= (uint32_t) static_cast<const uint16_t*>(row)[i + 2 * k + 1] << 16;
      }
      r.q[k >> 2][k & 3] = v;
    }
  }
  return r;
}

// The same of a row of n >= 8 without a branch: a group that crosses the row's
// end is the row's last eight elements, which shift8 puts in their places once
// they have arrived.  (load8's end is loads that wait for one another: a
// workgroup whose last wave takes it waits for that wave in every row.)  Past
// the row's end shift8 puts zeros, or with LAST the row's last element.
template <bool F32>
__device__ __forceinline__ Raw8<F32> load8_ahead(const void* row, int64_t i, int64_t n) {
  return load8<F32, true>(row, i + 8 <= n ? i : n - 8, n);
}
template <bool F32, bool LAST = false>
__device__ __forceinline__ void shift8(Raw8<F32>& r, int64_t i, int64_t n) {
  if (i + 8 <= n) return;
  const int s = i >= n ? 8 : (int)(i + 8 - n);   // elements past the end
  if constexpr (F32) {
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r.q[k >> 2][k & 3];
    const uint32_t fill = LAST ? v[7] : 0;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
      if (s & d) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k + d < 8 ? v[k + d] : fill;
      }
#pragma unroll
    for (int k = 0; k < 8; ++k) r.q[k >> 2][k & 3] = v[k];
  } else {
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = r.q[0][k];
    const uint32_t fill = LAST ? v[3] >> 16 | (v[3] & 0xFFFF0000u) : 0;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
      if (s & (2 * d)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = k + d < 4 ? v[k + d] : fill;
      }
    if (s & 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = v[k] >> 16 | (k < 3 ? v[k + 1] : fill) << 16;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) r.q[0][k] = v[k];
  }
}

template <bool F32>
__device__ __forceinline__ void values8(const Raw8<F32>& r, float* f) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (F32) {
      f[k] = __uint_as_float(r.q[0][k]);
      f[k + 4] = __uint_as_float(r.q[1][k]);
    } else {
      f[2 * k] = __uint_as_float(r.q[0][k] << 16);
      f[2 * k + 1] = __uint_as_float(r.q[0][k] & 0xFFFF0000u);
    }
  }
}

// The same with the element type known at run time only.
__device__ __forceinline__ void load8_values(const void* row, int f32, int64_t i, int64_t n, float* f) {
  if (f32) values8<true>(load8<true>(row, i, n), f);
  else values8<false>(load8<false>(row, i, n), f);
}

// Stores of elements i .. i + 7 of a row of n, as BF16, FP32 or E4M3.
__device__ __forceinline__ void store8_bf16(void* row, int64_t i, int64_t n, const float* f) {
  uint16_t* p = static_cast<uint16_t*>(row) + i;
  const u4 v = {bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7])};
  if (i + 8 <= n) {
    *reinterpret_cast<u4a2*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[k] = (uint16_t)(v[k >> 1] >> ((k & 1) * 16));
  }
}
__device__ __forceinline__ void store8_f32(void* row, int64_t i, int64_t n, const float* f) {
  float* p = static_cast<float*>(row) + i;
  if (i + 8 <= n) {
    *reinterpret_cast<f4a4*>(p) = (f4){f[0], f[1], f[2], f[3]};
    *reinterpret_cast<f4a4*>(p + 4) = (f4){f[4], f[5], f[6], f[7]};
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[k] = f[k];
  }
}
__device__ __forceinline__ void store8_fp8(void* row, int64_t i, int64_t n, const float* f) {
  uint8_t* p = static_cast<uint8_t*>(row) + i;
  const uint32_t a = e4m3_pack4(f[0], f[1], f[2], f[3]), b = e4m3_pack4(f[4], f[5], f[6], f[7]);
  if (i + 8 <= n) {
    *reinterpret_cast<u2a1*>(p) = (u2a1){a, b};
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[k] = (uint8_t)((k < 4 ? a : b) >> ((k & 3) * 8));
  }
}

// Sum over the wave, the same in every lane: four exchanges inside rows of 16
// lanes (quad permutations, half-row and row mirrors), then the four rows'
// sums in order.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return __fadd_rn(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true)));
}
// (over each 16 lanes alone)
__device__ __forceinline__ float sum16(float v) {
  v = dpp_add<0xB1>(v);        // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);        // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);       // row_half_mirror
  return dpp_add<0x140>(v);    // row_mirror
}
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  const int i = __float_as_int(v);
  const float a = __int_as_float(__builtin_amdgcn_readlane(i, 0)), b = __int_as_float(__builtin_amdgcn_readlane(i, 16));
  const float c = __int_as_float(__builtin_amdgcn_readlane(i, 32)), d = __int_as_float(__builtin_amdgcn_readlane(i, 48));
  return __fadd_rn(__fadd_rn(a, b), __fadd_rn(c, d));
}

// Sum over the threads that share a row, the same in each: TC = 16 or 64
// lanes, or (0) the whole workgroup.  red: 16 floats of LDS that no other sum
// in flight uses.
template <int TC>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if constexpr (TC == 16) return sum16(v);
  v = wave_sum(v);
  if constexpr (TC == 0) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const int waves = blockDim.x >> 6;
    v = red[0];
    for (int w = 1; w < waves; ++w) v = __fadd_rn(v, red[w]);
  }
  return v;
}

// A tree over eight values: fewer roundings in a row than one after another.
__device__ __forceinline__ float sum8(const float* f) {
  return __fadd_rn(__fadd_rn(__fadd_rn(f[0], f[1]), __fadd_rn(f[2], f[3])),
                   __fadd_rn(__fadd_rn(f[4], f[5]), __fadd_rn(f[6], f[7])));
}

// A sum that keeps what its additions round off (of many terms in one thread,
// where the roundings of a plain sum would add up: 2e-5 of rstd at 2^26
// columns).
struct LongSum {
  float s = 0.0f, lost = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float y = __fadd_rn(v, -lost), t = __fadd_rn(s, y);
    lost = __fadd_rn(__fadd_rn(t, -s), -y);
    s = t;
  }
};

}  // namespace rows
}  // namespace fp8mot
