// Layer norm over the last dimension and its backward pass (declared in
// include/fp8mot.h as fp8_layer_norm and fp8_layer_norm_backward).
//
//   mean = sum x / H,  var = sum (x - mean)^2 / H,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh w + b  -> BF16, E4M3(y / s_y) or FP32
//   g = dy w:  dx = rstd (g - sum g / H - xh sum(g xh) / H) + dres
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// All sums are FP32; the variance is taken about the mean (not from the
// squares' mean, which cancels where the mean is large).  Bound by memory: a
// row is read once and kept in registers over its sums.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "kernels.h"
#include "rowwise.h"

namespace fp8mot {

namespace {

using namespace rows;

// Sum over T threads that share a row (16 lanes, or whole waves), the same in
// each.  red: T / 64 floats of LDS that no other sum in flight uses.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* red) {
  if constexpr (T == 16) return sum16(v);
  v = wave_sum(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v = __fadd_rn(v, red[w]);
  }
  return v;
}

// A tree over eight values: fewer roundings in a row than one after another.
__device__ __forceinline__ float sum8(const float* f) {
  return __fadd_rn(__fadd_rn(__fadd_rn(f[0], f[1]), __fadd_rn(f[2], f[3])),
                   __fadd_rn(__fadd_rn(f[4], f[5]), __fadd_rn(f[6], f[7])));
}

__device__ __forceinline__ void emit8(const LayerNormArgs& g, int64_t base, int64_t i, float rs, float* y) {
  if (g.out_kind == 0) {
    store8_bf16(static_cast<uint16_t*>(g.y) + base, i, g.H, y);
  } else if (g.out_kind == 1) {
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = __fmul_rn(y[k], rs);
    store8_fp8(static_cast<uint8_t*>(g.y) + base, i, g.H, y);
  } else {
    store8_f32(static_cast<float*>(g.y) + base, i, g.H, y);
  }
}

// Weight and bias of eight columns: ones and zeros where there are none.
__device__ __forceinline__ void affine8(const LayerNormArgs& g, int64_t i, float* w, float* b) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    w[k] = 1.0f;
    b[k] = 0.0f;
  }
  if (g.w != nullptr) load8_values(g.w, g.wb_f32, i, g.H, w);
  if (g.b != nullptr) load8_values(g.b, g.wb_f32, i, g.H, b);
}

// T threads per row, U groups of eight elements per thread (group j * T + t of
// the row): a row of up to 8 T U elements in registers.  Workgroups of 256
// threads hold 256 / T rows where T < 256.  A workgroup walks rows: the next
// row is on its way while this one is summed, and (U <= 3) weight and bias
// stay in registers.
template <bool F32, int T, int U>
__global__ __launch_bounds__(T < 256 ? 256 : T) void layer_norm_kernel(LayerNormArgs g) {
  __shared__ float red[2][T < 64 ? 1 : T / 64];
  constexpr int RPB = T < 256 ? 256 / T : 1;
  constexpr bool KEEP = U <= 3;
  const int t = T < 256 ? threadIdx.x % T : threadIdx.x;
  const float inv_h = 1.0f / (float)g.H;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t r = (int64_t)blockIdx.x * RPB + (T < 256 ? threadIdx.x / T : 0);
  if (r >= g.rows) return;   // with T > 64 whole workgroups
  Raw8<F32> next[U];
  auto load = [&](int64_t row) {
    const void* xr = static_cast<const uint8_t*>(g.x) + row * g.H * (F32 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < U; ++j) next[j] = load8<F32>(xr, 8 * (int64_t)(j * T + t), g.H);
  };
  load(r);
  float w[KEEP ? U : 1][8], b[KEEP ? U : 1][8];
  if constexpr (KEEP) {
#pragma unroll
    for (int j = 0; j < U; ++j) affine8(g, 8 * (int64_t)(j * T + t), w[j], b[j]);
  }
  const float rs = g.out_kind == 1 ? 1.0f / *g.sy : 0.0f;
  // (the two sums' LDS takes turns, so a row's never meets the row before)
  for (; r < g.rows; r += step) {
    float x[U][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      values8<F32>(next[j], x[j]);
      s = __fadd_rn(s, sum8(x[j]));
    }
    if (r + step < g.rows) load(r + step);
    const float mean = __fmul_rn(row_sum<T>(s, red[0]), inv_h);
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[j][k] = __fadd_rn(x[j][k], -mean);
      if (i + 8 <= g.H) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v = __builtin_fmaf(x[j][k], x[j][k], v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i + k < g.H) v = __builtin_fmaf(x[j][k], x[j][k], v);
      }
    }
    const float var = __fmul_rn(row_sum<T>(v, red[1]), inv_h);
    const float rstd = 1.0f / __fsqrt_rn(__fadd_rn(var, g.eps));
    if (t == 0) {
      if (g.mean != nullptr) g.mean[r] = mean;
      if (g.rstd != nullptr) g.rstd[r] = rstd;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
      if (i < g.H) {
        if constexpr (!KEEP) affine8(g, i, w[0], b[0]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[j][k] = __builtin_fmaf(__fmul_rn(x[j][k], rstd), w[KEEP ? j : 0][k], b[KEEP ? j : 0][k]);
        emit8(g, r * g.H, i, rs, x[j]);
      }
    }
  }
}

// Rows too long for registers: read three times, from cache after the first.
template <bool F32>
__global__ __launch_bounds__(1024) void layer_norm_long_kernel(LayerNormArgs g) {
  __shared__ float red[2][16];
  const float inv_h = 1.0f / (float)g.H;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
  const int64_t base = r * g.H;
  const void* xr = static_cast<const uint8_t*>(g.x) + base * (F32 ? 4 : 2);
  float s = 0.0f;
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    float f[8];
    values8<F32>(load8<F32>(xr, i, g.H), f);
    s = __fadd_rn(s, sum8(f));
  }
  const float mean = __fmul_rn(row_sum<1024>(s, red[0]), inv_h);
  float v = 0.0f;
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    float f[8];
    values8<F32>(load8<F32>(xr, i, g.H), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = i + k < g.H ? __fadd_rn(f[k], -mean) : 0.0f;
      v = __builtin_fmaf(d, d, v);
    }
  }
  const float var = __fmul_rn(row_sum<1024>(v, red[1]), inv_h);
  const float rstd = 1.0f / __fsqrt_rn(__fadd_rn(var, g.eps));
  if (threadIdx.x == 0) {
    if (g.mean != nullptr) g.mean[r] = mean;
    if (g.rstd != nullptr) g.rstd[r] = rstd;
  }
  const float rs = g.out_kind == 1 ? 1.0f / *g.sy : 0.0f;
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    float f[8];
    values8<F32>(load8<F32>(xr, i, g.H), f);
    float w[8], b[8];
    affine8(g, i, w, b);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __builtin_fmaf(__fmul_rn(__fadd_rn(f[k], -mean), rstd), w[k], b[k]);
    emit8(g, base, i, rs, f);
  }
  }
}

// Backward pass.  T threads cover a row, U groups of eight columns each (TC:
// 16 or 64, and as many rows side by side as the workgroup holds; or 0: the
// whole workgroup, any number of waves).  They walk the rows of the workgroup's slab:
// the row's two sums through one barrier, dx, and the columns' sums of dy xh
// and dy in registers, which go to part[slab, 0:H) and [H:2H) at the end.  The
// next row's x, dy and dres are on their way during this row's sums.
template <bool XF, bool DF, int TC, int U>
__global__ __launch_bounds__(1024) void layer_norm_backward_kernel(LayerNormBwdArgs g, int64_t slab_rows,
                                                                   float* __restrict__ part) {
  const int G = TC > 0 ? (int)blockDim.x / TC : 1;   // rows side by side
  __shared__ float red[2][2][16];
  __shared__ float cols[TC > 0 ? 1024 * 8 : 1];      // [G][8 TC]
  const int T = TC > 0 ? TC : blockDim.x, waves = T >> 6, t = TC > 0 ? threadIdx.x % TC : threadIdx.x;
  const float inv_h = 1.0f / (float)g.H;
  const int64_t r0 = (int64_t)blockIdx.x * slab_rows;
  const int64_t r1 = r0 + slab_rows < g.rows ? r0 + slab_rows : g.rows;
  float w[U][8], sw[U][8], sb[U][8];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = 8 * (int64_t)(j * T + t);
    if (g.w != nullptr) load8_values(g.w, g.w_f32, i, g.H, w[j]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (g.w == nullptr) w[j][k] = 1.0f;
      sw[j][k] = sb[j][k] = 0.0f;
    }
  }
  Raw8<XF> x[U], rs[U];
  Raw8<DF> d[U];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t r) {
    const int64_t base = r * g.H;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
      x[j] = load8<XF>(static_cast<const uint8_t*>(g.x) + base * (XF ? 4 : 2), i, g.H);
      d[j] = load8<DF>(static_cast<const uint8_t*>(g.dy) + base * (DF ? 4 : 2), i, g.H);
      if (g.dres != nullptr) rs[j] = load8<XF>(static_cast<const uint8_t*>(g.dres) + base * (XF ? 4 : 2), i, g.H);
    }
    mean = g.mean[r];
    rstd = g.rstd[r];
  };
  int64_t r = r0 + (TC > 0 ? threadIdx.x / TC : 0);
  if (r < r1) load(r);
  for (int buf = 0; r < r1; r += G, buf ^= 1) {
    float xh[U][8], gw[U][8], res[U][8];
    const float rstd_r = rstd;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float dy[8];
      values8<XF>(x[j], xh[j]);
      values8<DF>(d[j], dy);
      if (g.dres != nullptr) values8<XF>(rs[j], res[j]);
      // columns past H: dy is 0 there, and whatever xh is falls away
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        xh[j][k] = __fmul_rn(__fadd_rn(xh[j][k], -mean), rstd);
        gw[j][k] = __fmul_rn(dy[k], w[j][k]);
        s1 = __fadd_rn(s1, gw[j][k]);
      }
      if (8 * (int64_t)(j * T + t) + 8 <= g.H) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          s2 = __builtin_fmaf(gw[j][k], xh[j][k], s2);
          sw[j][k] = __builtin_fmaf(dy[k], xh[j][k], sw[j][k]);
        }
      } else {
        const int64_t left = g.H - 8 * (int64_t)(j * T + t);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < left) {
            s2 = __builtin_fmaf(gw[j][k], xh[j][k], s2);
            sw[j][k] = __builtin_fmaf(dy[k], xh[j][k], sw[j][k]);
          }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sb[j][k] = __fadd_rn(sb[j][k], dy[k]);
    }
    if (r + G < r1) load(r + G);
    if constexpr (TC == 16) {
      s1 = sum16(s1);
      s2 = sum16(s2);
    } else {
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
    }
    if constexpr (TC == 0) {
      if ((t & 63) == 0) {
        red[buf][0][t >> 6] = s1;
        red[buf][1][t >> 6] = s2;
      }
      __syncthreads();   // the other buffer's readers are past the barrier before this one
      s1 = red[buf][0][0];
      s2 = red[buf][1][0];
      for (int v = 1; v < waves; ++v) {
        s1 = __fadd_rn(s1, red[buf][0][v]);
        s2 = __fadd_rn(s2, red[buf][1][v]);
      }
    }
    const float c1 = __fmul_rn(s1, inv_h), c2 = __fmul_rn(s2, inv_h);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
      if (i < g.H) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          y[k] = __fmul_rn(rstd_r, __builtin_fmaf(-xh[j][k], c2, __fadd_rn(gw[j][k], -c1)));
          if (g.dres != nullptr) y[k] = __fadd_rn(y[k], res[j][k]);
        }
        if constexpr (XF) store8_f32(static_cast<float*>(g.dx) + r * g.H, i, g.H, y);
        else store8_bf16(static_cast<uint16_t*>(g.dx) + r * g.H, i, g.H, y);
      }
    }
  }
  if (part == nullptr) return;
  float* p = part + (int64_t)blockIdx.x * 2 * g.H;
  if constexpr (TC > 0) {
    // the rows side by side are added in order, one kind of sum at a time
    static_assert(U == 1, "");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h > 0) __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) cols[8 * threadIdx.x + k] = h == 0 ? sw[0][k] : sb[0][k];
      __syncthreads();
      for (int c = threadIdx.x; c < TC * 8; c += blockDim.x) {
        float v = cols[c];
        for (int q = 1; q < G; ++q) v = __fadd_rn(v, cols[q * (TC * 8) + c]);
        if (c < g.H) p[h * g.H + c] = v;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
      if (i < g.H) {
        store8_f32(p, i, g.H, sw[j]);
        store8_f32(p + g.H, i, g.H, sb[j]);
      }
    }
  }
}

// Rows too long for that: column sums first (dx may be written over dy or x),
// eight columns per thread over a slab, then dx with two reads of the row.
__global__ __launch_bounds__(256) void layer_norm_dw_long_kernel(LayerNormBwdArgs g, int64_t slab_rows,
                                                                 float* __restrict__ part) {
  const int64_t i = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= g.H) return;
  const int64_t r0 = (int64_t)blockIdx.y * slab_rows;
  const int64_t r1 = r0 + slab_rows < g.rows ? r0 + slab_rows : g.rows;
  float sw[8] = {}, sb[8] = {};
  for (int64_t r = r0; r < r1; ++r) {
    float x[8], d[8];
    load8_values(static_cast<const uint8_t*>(g.x) + r * g.H * (g.x_f32 ? 4 : 2), g.x_f32, i, g.H, x);
    load8_values(static_cast<const uint8_t*>(g.dy) + r * g.H * (g.dy_f32 ? 4 : 2), g.dy_f32, i, g.H, d);
    const float mean = g.mean[r], rstd = g.rstd[r];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      sw[k] = __builtin_fmaf(d[k], __fmul_rn(__fadd_rn(x[k], -mean), rstd), sw[k]);
      sb[k] = __fadd_rn(sb[k], d[k]);
    }
  }
  float* p = part + (int64_t)blockIdx.y * 2 * g.H;
  store8_f32(p, i, g.H, sw);
  store8_f32(p + g.H, i, g.H, sb);
}

__global__ __launch_bounds__(1024) void layer_norm_dx_long_kernel(LayerNormBwdArgs g) {
  __shared__ float red[2][16];
  const float inv_h = 1.0f / (float)g.H;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
  const uint8_t* xr = static_cast<const uint8_t*>(g.x) + r * g.H * (g.x_f32 ? 4 : 2);
  const uint8_t* dr = static_cast<const uint8_t*>(g.dy) + r * g.H * (g.dy_f32 ? 4 : 2);
  const float mean = g.mean[r], rstd = g.rstd[r];
  auto row8 = [&](int64_t i, float* xh, float* gw) {
    load8_values(xr, g.x_f32, i, g.H, xh);
    load8_values(dr, g.dy_f32, i, g.H, gw);
    float w[8];
    if (g.w != nullptr) load8_values(g.w, g.w_f32, i, g.H, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      xh[k] = i + k < g.H ? __fmul_rn(__fadd_rn(xh[k], -mean), rstd) : 0.0f;
      if (g.w != nullptr) gw[k] = __fmul_rn(gw[k], w[k]);
    }
  };
  float s1 = 0.0f, s2 = 0.0f, xh[8], gw[8];
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    row8(i, xh, gw);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s1 = __fadd_rn(s1, gw[k]);
      s2 = __builtin_fmaf(gw[k], xh[k], s2);
    }
  }
  const float c1 = __fmul_rn(row_sum<1024>(s1, red[0]), inv_h), c2 = __fmul_rn(row_sum<1024>(s2, red[1]), inv_h);
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    row8(i, xh, gw);
    float y[8], res[8];
    if (g.dres != nullptr)
      load8_values(static_cast<const uint8_t*>(g.dres) + r * g.H * (g.x_f32 ? 4 : 2), g.x_f32, i, g.H, res);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[k] = __fmul_rn(rstd, __builtin_fmaf(-xh[k], c2, __fadd_rn(gw[k], -c1)));
      if (g.dres != nullptr) y[k] = __fadd_rn(y[k], res[k]);
    }
    if (g.x_f32) store8_f32(static_cast<float*>(g.dx) + r * g.H, i, g.H, y);
    else store8_bf16(static_cast<uint16_t*>(g.dx) + r * g.H, i, g.H, y);
  }
  }
}

// Column sums over slabs: out_a[n] (n < N) and out_b[n - N] (n >= N), either of
// them NULL to leave it out, of part [slabs, cols] in an order that depends on
// (slabs, cols) alone.  A workgroup takes 4 Q columns, four per thread, and L
// threads share a column's slabs, R of them in flight each.
template <int Q>
__global__ __launch_bounds__(256) void sum_slabs_kernel(const float* __restrict__ part, float* __restrict__ out_a,
                                                        float* __restrict__ out_b, int64_t slabs, int64_t N,
                                                        int64_t cols) {
  constexpr int R = 4, L = 256 / Q, C = 4 * Q, P = 256 / C;
  __shared__ float red[L][C + 1], red2[P][C + 1];
  const int q = threadIdx.x % Q, s = threadIdx.x / Q;
  const int64_t n = (int64_t)blockIdx.x * C + 4 * q;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* v = part + n;
  if (n + 4 <= cols) {
    int64_t p = s;
    for (; p + L * (R - 1) < slabs; p += L * R) {
      f4 x[R];
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] = *reinterpret_cast<const f4a4*>(v + (p + L * r) * cols);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) a[k] = __fadd_rn(a[k], x[r][k]);
    }
    for (; p < slabs; p += L) {
      const f4 x = *reinterpret_cast<const f4a4*>(v + p * cols);
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = __fadd_rn(a[k], x[k]);
    }
  } else {
    for (int64_t p = s; p < slabs; p += L)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (n + k < cols) a[k] = __fadd_rn(a[k], v[p * cols + k]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) red[s][4 * q + k] = a[k];
  __syncthreads();
  {
    static_assert(L / P == 4, "four rows of red per thread");
    const int c = threadIdx.x % C, h = threadIdx.x / C;
    red2[h][c] = __fadd_rn(__fadd_rn(red[4 * h][c], red[4 * h + 1][c]), __fadd_rn(red[4 * h + 2][c], red[4 * h + 3][c]));
  }
  __syncthreads();
  if (threadIdx.x < C) {
    float t = red2[0][threadIdx.x];
#pragma unroll
    for (int p = 1; p < P; ++p) t = __fadd_rn(t, red2[p][threadIdx.x]);
    const int64_t c = (int64_t)blockIdx.x * C + threadIdx.x;
    if (c < N) {
      if (out_a != nullptr) out_a[c] = t;
    } else if (c < cols) {
      if (out_b != nullptr) out_b[c - N] = t;
    }
  }
}

// Workgroups of a grid over rows: up to `most`, which walk the rest.
unsigned row_grid(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

template <bool F32, int T, int U>
hipError_t run_norm(const LayerNormArgs& g, hipStream_t stream) {
  constexpr int rpb = T < 256 ? 256 / T : 1, threads = T < 256 ? 256 : T;
  // as many workgroups as are resident at once (256 CUs): 4 to 8 waves a SIMD
  constexpr int64_t most = 256 * ((U <= 1 ? 32 : U == 2 ? 24 : 16) * 64 / threads);
  hipLaunchKernelGGL((layer_norm_kernel<F32, T, U>), dim3(row_grid((g.rows + rpb - 1) / rpb, most)), dim3(threads), 0,
                     stream, g);
  return hipGetLastError();
}

template <bool F32>
hipError_t norm_of_type(const LayerNormArgs& g, hipStream_t stream) {
  const int64_t units = (g.H + 7) / 8;
  if (units <= 16) return run_norm<F32, 16, 1>(g, stream);
  if (units <= 64) return run_norm<F32, 64, 1>(g, stream);
  if (units <= 128 && g.rows > 512) return run_norm<F32, 64, 2>(g, stream);
  if (units <= 256) return run_norm<F32, 256, 1>(g, stream);
  if (units <= 512 && g.rows > 512) return run_norm<F32, 256, 2>(g, stream);
  if (units <= 768 && g.rows > 512) return run_norm<F32, 256, 3>(g, stream);
  if (units <= 1024) return run_norm<F32, 1024, 1>(g, stream);
  if (units <= 2048) return run_norm<F32, 1024, 2>(g, stream);
  if (units <= 4096) return run_norm<F32, 1024, 4>(g, stream);
  hipLaunchKernelGGL((layer_norm_long_kernel<F32>), dim3(row_grid(g.rows, 1 << 20)), dim3(1024), 0, stream, g);
  return hipGetLastError();
}

// rows of up to this many elements go through layer_norm_backward_kernel
constexpr int64_t kBwdRegs = 1024 * 8 * 2;

// How the backward pass covers rows of H elements: threads of a workgroup,
// rows side by side in it, groups of eight per thread, and slabs: as many
// workgroups as are resident at once (256 CUs, 16 to 20 waves each), but at
// least two rows one after another in each.  Narrow rows go 1024 threads to a
// workgroup where there are enough of them, which keeps the slabs few.
struct BwdShape {
  int threads, side, groups;
  int64_t slabs;
};
BwdShape bwd_shape(int64_t rows, int64_t H) {
  const int64_t units = (H + 7) / 8;
  BwdShape b{0, 1, 1, 0};
  if (units <= 64) {
    const int tc = units <= 16 ? 16 : 64;
    b.threads = rows >= 256 * 4 * (1024 / tc) ? 1024 : 256;
    b.side = b.threads / tc;
  } else {
    b.groups = units <= 1024 ? 1 : 2;
    const int64_t t = (units + b.groups - 1) / b.groups;
    b.threads = t < 1024 ? (int)((t + 63) / 64 * 64) : 1024;
  }
  const int waves = b.threads / 64;
  b.slabs = 256 * (waves > 10 ? 1 : waves > 4 ? 20 / waves : 4);
  const int64_t most = (rows + 2 * b.side - 1) / (2 * b.side);
  if (b.slabs > most) b.slabs = most;
  return b;
}

template <bool XF, bool DF, int TC, int U>
hipError_t run_backward_kernel(const LayerNormBwdArgs& g, int threads, int64_t slabs, float* part,
                               hipStream_t stream) {
  hipLaunchKernelGGL((layer_norm_backward_kernel<XF, DF, TC, U>), dim3((unsigned)slabs), dim3(threads), 0, stream, g,
                     (g.rows + slabs - 1) / slabs, part);
  return hipGetLastError();
}

template <bool XF, bool DF>
hipError_t run_backward(const LayerNormBwdArgs& g, int64_t slabs, float* part, hipStream_t stream) {
  const BwdShape b = bwd_shape(g.rows, g.H);
  if (g.H <= 128) return run_backward_kernel<XF, DF, 16, 1>(g, b.threads, slabs, part, stream);
  if (g.H <= 512) return run_backward_kernel<XF, DF, 64, 1>(g, b.threads, slabs, part, stream);
  if (b.groups == 1) return run_backward_kernel<XF, DF, 0, 1>(g, b.threads, slabs, part, stream);
  return run_backward_kernel<XF, DF, 0, 2>(g, b.threads, slabs, part, stream);
}

}  // namespace

hipError_t launch_sum_slabs(const float* part, float* out_a, float* out_b, int64_t slabs, int64_t N, int64_t cols,
                            hipStream_t stream) {
  // 64 columns a workgroup read whole 256-byte pieces, but few columns then
  // leave most CUs idle: 8192 columns of 256 slabs in 64s 2.8 us less than in
  // 16s, 2054 columns of 766 slabs 7.7 us more
  if (cols >= 8192)
    hipLaunchKernelGGL(sum_slabs_kernel<16>, dim3((unsigned)((cols + 63) / 64)), dim3(256), 0, stream, part, out_a,
                       out_b, slabs, N, cols);
  else
    hipLaunchKernelGGL(sum_slabs_kernel<4>, dim3((unsigned)((cols + 15) / 16)), dim3(256), 0, stream, part, out_a,
                       out_b, slabs, N, cols);
  return hipGetLastError();
}

hipError_t launch_layer_norm(const LayerNormArgs& g, hipStream_t stream) {
  return g.x_f32 ? norm_of_type<true>(g, stream) : norm_of_type<false>(g, stream);
}

int64_t layer_norm_backward_slabs(int64_t rows, int64_t H) { return rows == 0 ? 0 : bwd_shape(rows, H).slabs; }

hipError_t launch_layer_norm_backward(const LayerNormBwdArgs& g, float* dw, float* db, float* part,
                                      hipStream_t stream) {
  const int64_t slabs = layer_norm_backward_slabs(g.rows, g.H);
  const bool sums = dw != nullptr || db != nullptr;
  hipError_t e = hipSuccess;
  if (slabs > 0 && g.H <= kBwdRegs) {
    float* p = sums ? part : nullptr;
    if (g.x_f32) e = g.dy_f32 ? run_backward<true, true>(g, slabs, p, stream) : run_backward<true, false>(g, slabs, p, stream);
    else e = g.dy_f32 ? run_backward<false, true>(g, slabs, p, stream) : run_backward<false, false>(g, slabs, p, stream);
  } else if (slabs > 0) {
    if (sums)
      hipLaunchKernelGGL(layer_norm_dw_long_kernel, dim3((unsigned)((g.H + 2047) / 2048), (unsigned)slabs), dim3(256),
                         0, stream, g, (g.rows + slabs - 1) / slabs, part);
    hipLaunchKernelGGL(layer_norm_dx_long_kernel, dim3(row_grid(g.rows, 1 << 20)), dim3(1024), 0, stream, g);
    e = hipGetLastError();
  }
  if (e != hipSuccess || !sums) return e;
  return launch_sum_slabs(part, dw, db, slabs, g.H, 2 * g.H, stream);
}

}  // namespace fp8mot
