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

// Vectors of a row whose start may not be a multiple of their size: global
// accesses need no alignment beyond the element's on this target.
typedef uint32_t u2a __attribute__((ext_vector_type(2), aligned(2)));
typedef float f4a __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u1a __attribute__((aligned(1)));

// Rows of a [M, N] tensor from row m0 on.  A group of four columns is
// addressed by its element offset from there, row * N + n; loads of groups and
// elements past the matrix give zeros and their stores are dropped: with VEC
// (N % 4 == 0: a group lies inside its row or past it) by the buffer's range
// check, otherwise by comparison, four elements at once inside a row and one
// by one at its end.
struct Rows {
  __amdgpu_buffer_rsrc_t r;
  void* base;
  int64_t limit;   // elements from row m0 to the matrix's end
};
__device__ __forceinline__ Rows rows_of(const void* p, int64_t m0, int64_t M, int64_t N, int esz) {
  Rows t;
  t.base = p == nullptr ? nullptr : const_cast<uint8_t*>(static_cast<const uint8_t*>(p)) + m0 * N * esz;
  t.limit = p == nullptr ? 0 : (M - m0) * N;
  t.r = tile::make_rsrc(t.base, t.limit * esz);
  return t;
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
  } else if (at < t.limit) {
    if (f32) {
      const float* p = static_cast<const float*>(t.base) + at;
      if (nv >= 4) {
        v = __builtin_bit_cast(u4v, (f4v)(*reinterpret_cast<const f4a*>(p)));
      } else {
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (c < nv) v[c] = __float_as_uint(p[c]);
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(t.base) + at;
      if (nv >= 4) {
        const u2a h = *reinterpret_cast<const u2a*>(p);
        v.x = h.x;
        v.y = h.y;
      } else {
        if (nv > 0) v.x = p[0];
        if (nv > 1) v.x |= (uint32_t)p[1] << 16;
        if (nv > 2) v.y = p[2];
      }
    }
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
  } else if (at < t.limit) {
    uint16_t* p = static_cast<uint16_t*>(t.base) + at;
    if (nv >= 4) {
      *reinterpret_cast<u2a*>(p) = (u2a){a, b};
    } else {
      if (nv > 0) p[0] = (uint16_t)a;
      if (nv > 1) p[1] = (uint16_t)(a >> 16);
      if (nv > 2) p[2] = (uint16_t)b;
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store4_f32(const Rows& t, int at, int nv, const float* z) {
  if constexpr (VEC) {
    __builtin_amdgcn_raw_buffer_store_b128(
        (tile::v4u){__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3])},
        t.r, nv > 0 ? at * 4 : tile::kOOB, 0, 0);
  } else if (at < t.limit) {
    float* p = static_cast<float*>(t.base) + at;
    if (nv >= 4) {
      *reinterpret_cast<f4a*>(p) = (f4a){z[0], z[1], z[2], z[3]};
    } else {
#pragma unroll
      for (int c = 0; c < 3; ++c)
        if (c < nv) p[c] = z[c];
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store4_fp8(const Rows& t, int at, int nv, const float* z) {
  const uint32_t w = e4m3_pack4(z[0], z[1], z[2], z[3]);
  if constexpr (VEC) {
    __builtin_amdgcn_raw_buffer_store_b32(w, t.r, nv > 0 ? at : tile::kOOB, 0, 0);
  } else if (at < t.limit) {
    uint8_t* p = static_cast<uint8_t*>(t.base) + at;
    if (nv >= 4) {
      *reinterpret_cast<u1a*>(p) = w;
    } else {
#pragma unroll
      for (int c = 0; c < 3; ++c)
        if (c < nv) p[c] = (uint8_t)(w >> (8 * c));
    }
  }
}

// What the epilogue needs of a launch and of a workgroup's rows, read once.
struct Epilogue {
  Rows y, residual, pre;
  float alpha;   // s_x s_w (without row scales)
  float rs;      // 1 / s_y, correctly rounded (FP8 output)
};
__device__ __forceinline__ Epilogue open_outputs(const LinearActArgs& g, int64_t m0) {   // of sums scaled already
  Epilogue e;
  e.y = rows_of(g.y, m0, g.M, g.N, g.out_kind == 0 ? 2 : (g.out_kind == 1 ? 1 : 4));
  e.residual = rows_of(g.residual, m0, g.M, g.N, g.residual_f32 ? 4 : 2);
  e.pre = rows_of(g.pre, m0, g.M, g.N, 2);
  e.alpha = 1.0f;
  e.rs = g.out_kind == 1 ? 1.0f / *g.sy : 0.0f;
  return e;
}
__device__ __forceinline__ Epilogue open_epilogue(const LinearActArgs& g, int64_t m0) {
  Epilogue e = open_outputs(g, m0);
  e.alpha = g.row_scales ? 0.0f : __fmul_rn(*g.sx, *g.sw);
  return e;
}

// Bias and (with row scales) weight scales of four columns, as raw dwords: what
// loads them does not wait for them.
struct Columns {
  u4v bias, sw;
};
template <bool VEC>
__device__ __forceinline__ Columns load_columns(const LinearActArgs& g, int n, int nv) {
  Columns c = {{0, 0, 0, 0}, {0, 0, 0, 0}};
  if (g.bias != nullptr) c.bias = load4<VEC>(rows_of(g.bias, 0, 1, g.N, g.bias_f32 ? 4 : 2), g.bias_f32, n, nv);
  if (g.row_scales) c.sw = load4<VEC>(rows_of(g.sw, 0, 1, g.N, 4), 1, n, nv);
  return c;
}

// What G groups in rows `row`, row + dm, .. (counted from m0), columns
// n .. n + 3, need of their own: the residual as raw dwords and the rows'
// scales.
template <int G>
struct Operands {
  u4v residual[G];
  float sx[G];
};
template <int G, bool VEC>
__device__ __forceinline__ void load_operands(const LinearActArgs& g, const Epilogue& e, int64_t m0, int row, int dm,
                                              int n, int nv, Operands<G>* o) {
  if (g.residual != nullptr) {
#pragma unroll
    for (int k = 0; k < G; ++k)
      o->residual[k] = load4<VEC>(e.residual, g.residual_f32, (row + k * dm) * (int)g.N + n, nv);
  }
  if (g.row_scales) {
#pragma unroll
    for (int k = 0; k < G; ++k) o->sx[k] = m0 + row + k * dm < g.M ? g.sx[m0 + row + k * dm] : 0.0f;
  }
}

// Outputs of G such groups from their sums z (overwritten):
// z = fma(acc, alpha, bias), pre, act, + residual, y.  FP8 values are
// multiplied by 1 / s_y, as in the SwiGLU kernels.  next() runs once the
// operands have been used, before the outputs' stores: the place to load the
// next groups'.
template <int G, bool VEC, class Next>
__device__ __forceinline__ void finish(const LinearActArgs& g, const Epilogue& e, const Columns& col, int row,
                                       int dm, int n, int nv, const Operands<G>& o, float (*z)[4], Next next) {
  const int N = (int)g.N;
  float bias[4], sw[4];
  values4(col.bias, g.bias_f32, bias);
  if (g.row_scales) {
    values4(col.sw, 1, sw);
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) z[k][c] = __builtin_fmaf(z[k][c], __fmul_rn(o.sx[k], sw[c]), bias[c]);
  } else {
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) z[k][c] = __builtin_fmaf(z[k][c], e.alpha, bias[c]);
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
      values4(o.residual[k], g.residual_f32, r);
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
