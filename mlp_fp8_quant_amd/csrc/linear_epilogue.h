// The epilogue of fp8_linear_act, shared by its kernels: bias, activation,
// residual and output of groups of four consecutive columns.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "device_common.h"
#include "gemm_parts.h"
#include "kernels.h"

namespace fp8mot {
namespace linear {

typedef uint32_t u2v __attribute__((ext_vector_type(2)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef float f4v __attribute__((ext_vector_type(4)));

// Rows of a [M, N] tensor from row m0 on.  A group of four columns is
// addressed by its element offset from there, row * N + n; groups and elements
// past the matrix get an offset past the buffer's range, where loads read
// zeros and stores are dropped.  VEC (N % 4 == 0): a group lies inside its row
// or past it and moves in one access; otherwise element by element.
struct Rows {
  __amdgpu_buffer_rsrc_t r;
};
__device__ __forceinline__ Rows rows_of(const void* p, int64_t m0, int64_t M, int64_t N, int esz) {
  return {tile::make_rsrc(p == nullptr ? nullptr : static_cast<const uint8_t*>(p) + m0 * N * esz,
                          p == nullptr ? 0 : (M - m0) * N * esz)};
}

// nv: how many of the group's columns lie inside the row.
template <bool VEC>
__device__ __forceinline__ u4v load4(const Rows& t, int f32, int at, int nv) {
  u4v v = {0, 0, 0, 0};
  if constexpr (VEC) {
    if (f32) {
      v = __builtin_bit_cast(u4v, __builtin_amdgcn_raw_buffer_load_b128(t.r, nv > 0 ? at * 4 : tile::kOOB, 0, 0));
    } else {
      const u2v h = __builtin_bit_cast(u2v, __builtin_amdgcn_raw_buffer_load_b64(t.r, nv > 0 ? at * 2 : tile::kOOB, 0, 0));
      v.x = h.x;
      v.y = h.y;
    }
  } else if (f32) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      v[c] = __builtin_amdgcn_raw_buffer_load_b32(t.r, c < nv ? (at + c) * 4 : tile::kOOB, 0, 0);
  } else {
    uint32_t h[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      h[c] = __builtin_amdgcn_raw_buffer_load_b16(t.r, c < nv ? (at + c) * 2 : tile::kOOB, 0, 0);
    v.x = h[0] | h[1] << 16;
    v.y = h[2] | h[3] << 16;
  }
  return v;
}

__device__ __forceinline__ void values4(const u4v v, int f32, float* f) {
  f[0] = __uint_as_float(f32 ? v.x : v.x << 16);
  f[1] = __uint_as_float(f32 ? v.y : v.x & 0xFFFF0000u);
  f[2] = __uint_as_float(f32 ? v.z : v.y << 16);
  f[3] = __uint_as_float(f32 ? v.w : v.y & 0xFFFF0000u);
}

template <bool VEC>
__device__ __forceinline__ void store4_bf16(const Rows& t, int at, int nv, const float* z) {
  const uint32_t a = bf16x2_rne(z[0], z[1]), b = bf16x2_rne(z[2], z[3]);
  if constexpr (VEC) {
    __builtin_amdgcn_raw_buffer_store_b64((tile::v2u){a, b}, t.r, nv > 0 ? at * 2 : tile::kOOB, 0, 0);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)((c < 2 ? a : b) >> ((c & 1) * 16)), t.r,
                                            c < nv ? (at + c) * 2 : tile::kOOB, 0, 0);
  }
}

template <bool VEC>
__device__ __forceinline__ void store4_f32(const Rows& t, int at, int nv, const float* z) {
  if constexpr (VEC) {
    __builtin_amdgcn_raw_buffer_store_b128(
        (tile::v4u){__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3])},
        t.r, nv > 0 ? at * 4 : tile::kOOB, 0, 0);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(z[c]), t.r, c < nv ? (at + c) * 4 : tile::kOOB, 0, 0);
  }
}

template <bool VEC>
__device__ __forceinline__ void store4_fp8(const Rows& t, int at, int nv, const float* z) {
  const uint32_t w = e4m3_pack4(z[0], z[1], z[2], z[3]);
  if constexpr (VEC) {
    __builtin_amdgcn_raw_buffer_store_b32(w, t.r, nv > 0 ? at : tile::kOOB, 0, 0);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(w >> (8 * c)), t.r, c < nv ? at + c : tile::kOOB, 0, 0);
  }
}

// What the epilogue needs of a launch and of a workgroup's rows, read once.
struct Epilogue {
  Rows y, residual, pre;
  float alpha;   // s_x s_w (without row scales)
  float rs;      // 1 / s_y, correctly rounded (FP8 output)
};
__device__ __forceinline__ Epilogue open_epilogue(const LinearActArgs& g, int64_t m0) {
  Epilogue e;
  e.y = rows_of(g.y, m0, g.M, g.N, g.out_kind == 0 ? 2 : (g.out_kind == 1 ? 1 : 4));
  e.residual = rows_of(g.residual, m0, g.M, g.N, g.residual_f32 ? 4 : 2);
  e.pre = rows_of(g.pre, m0, g.M, g.N, 2);
  e.alpha = g.row_scales ? 0.0f : __fmul_rn(*g.sx, *g.sw);
  e.rs = g.out_kind == 1 ? 1.0f / *g.sy : 0.0f;
  return e;
}

// Bias of four columns.
struct Columns {
  float bias[4];
};
template <bool VEC>
__device__ __forceinline__ Columns load_columns(const LinearActArgs& g, int n, int nv) {
  Columns c = {{0.0f, 0.0f, 0.0f, 0.0f}};
  if (g.bias != nullptr) values4(load4<VEC>(rows_of(g.bias, 0, 1, g.N, g.bias_f32 ? 4 : 2), g.bias_f32, n, nv), g.bias_f32, c.bias);
  return c;
}

// Residual of G groups in rows `row`, row + dm, .. (counted from m0), columns
// n .. n + 3: raw dwords.
template <int G, bool VEC>
__device__ __forceinline__ void load_residual(const LinearActArgs& g, const Epilogue& e, int row, int dm, int n,
                                              int nv, u4v* r) {
#pragma unroll
  for (int k = 0; k < G; ++k) r[k] = load4<VEC>(e.residual, g.residual_f32, (row + k * dm) * (int)g.N + n, nv);
}

// Outputs of G such groups from their sums z (overwritten):
// z = fma(acc, alpha, bias), pre, act, + residual, y.  FP8 values are
// multiplied by 1 / s_y, as in the SwiGLU kernels.  next() runs once the
// residual has been used, before the outputs' stores: the place to load the
// next groups' residual.
template <int G, bool VEC, class Next>
__device__ __forceinline__ void finish(const LinearActArgs& g, const Epilogue& e, const Columns& col, int64_t m0,
                                       int row, int dm, int n, int nv, const u4v* residual, float (*z)[4],
                                       Next next) {
  const int N = (int)g.N;
  if (g.row_scales) {
    float sw[4];
    values4(load4<VEC>(rows_of(g.sw, 0, 1, g.N, 4), 1, n, nv), 1, sw);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int64_t m = m0 + row + k * dm;
      const float sx = m < g.M ? g.sx[m] : 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) z[k][c] = __builtin_fmaf(z[k][c], __fmul_rn(sx, sw[c]), col.bias[c]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) z[k][c] = __builtin_fmaf(z[k][c], e.alpha, col.bias[c]);
  }
  if (g.pre != nullptr) {
#pragma unroll
    for (int k = 0; k < G; ++k) store4_bf16<VEC>(e.pre, (row + k * dm) * N + n, nv, z[k]);
  }
  act_all<4 * G>(&z[0][0], g.act);
  if (g.residual != nullptr) {
#pragma unroll
    for (int k = 0; k < G; ++k) {
      float r[4];
      values4(residual[k], g.residual_f32, r);
#pragma unroll
      for (int c = 0; c < 4; ++c) z[k][c] = __fadd_rn(z[k][c], r[c]);
    }
  }
  next();
  if (g.out_kind == 0) {
#pragma unroll
    for (int k = 0; k < G; ++k) store4_bf16<VEC>(e.y, (row + k * dm) * N + n, nv, z[k]);
  } else if (g.out_kind == 1) {
#pragma unroll
    for (int k = 0; k < G; ++k) {
#pragma unroll
      for (int c = 0; c < 4; ++c) z[k][c] = __fmul_rn(z[k][c], e.rs);
      store4_fp8<VEC>(e.y, (row + k * dm) * N + n, nv, z[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < G; ++k) store4_f32<VEC>(e.y, (row + k * dm) * N + n, nv, z[k]);
  }
}

}  // namespace linear
}  // namespace fp8mot
