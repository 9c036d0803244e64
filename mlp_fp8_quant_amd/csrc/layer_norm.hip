// Layer norm over the last dimension and its backward pass (declared in
// include/fp8mot.h as fp8_layer_norm and fp8_layer_norm_backward).
//
//   mean = sum x / H,  var = sum (x - mean)^2 / H,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh w + b  -> BF16, E4M3(y / s_y) or FP32
//   g = dy w:  dx = rstd (g - sum g / H - xh sum(g xh) / H) + dres
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// All sums are FP32.  The variance is taken about the mean (not from the
// squares' mean, which cancels where the mean is large).  A first mean is off by
// some 2^-24 of itself (an ulp at 1000 is 6e-5, which the rstd of a constant
// row, 316, makes 0.02): where the mean is far above the spread, the
// differences from it are summed too, and that sum corrects mean, variance and
// xh.  Bound by memory: a row is read once and kept in registers over its sums.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "rowwise.h"

namespace fp8mot {

namespace {

using namespace rows;

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

// Whether a row's mean needs the correction, from the mean square d2 of the
// differences from it: below four standard deviations some 2^-24 of it is less
// than the other roundings of (x - mean) rstd.  Equal in the threads that share a
// row.  (A third sum in every row costs 2 to 7%: 16384x5120 BF16 -> E4M3 60.3
// -> 64.4 us.)
__device__ __forceinline__ bool off_centre(float mean, float d2, float eps) {
  return __fmul_rn(mean, mean) > 16.0f * __fadd_rn(d2, eps);
}
// The variance about mean + off (0 where roundings would make it negative).
__device__ __forceinline__ float centred(float d2, float off) {
  return __builtin_fmaxf(__builtin_fmaf(-off, off, d2), 0.0f);
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

// T threads cover a row, U groups of eight elements each (group j * T + t of
// the row), in registers.  TC: 16 or 64 of them, 256 / TC rows side by side in
// a workgroup; or 0: the whole workgroup, any number of waves.  A workgroup
// walks rows: the next row is on its way while this one is summed, and weight
// and bias stay in registers.  FULL: the groups are exactly the row (512x4096
// BF16 -> E4M3 4.1 us with its loads unguarded, 4.4 with the guards).
// 16384x5120 BF16 -> BF16 67 us, 5.0 TB/s, bound by memory; -> E4M3 60 us, 4.2
// TB/s, by the arithmetic between the row's sums (loads two rows ahead: slower).
// The bound of 1024 threads holds every whole-workgroup kernel to 128 registers;
// that of three FP32 groups spills 32, which does not show: 16384x5120 FP32 ->
// BF16 97 us, 8000x12288 113, both 5.2 TB/s.
template <bool F32, int TC, int U, bool FULL>
__global__ __launch_bounds__(TC > 0 ? 256 : 1024) void layer_norm_kernel(LayerNormArgs g) {
  __shared__ float red[3][16];
  constexpr int RPB = TC > 0 ? 256 / (TC > 0 ? TC : 1) : 1;
  constexpr bool KEEP = U <= 3;   // more would not fit beside the row
  const int T = TC > 0 ? TC : blockDim.x, t = TC > 0 ? threadIdx.x % T : threadIdx.x;
  const float inv_h = 1.0f / (float)g.H;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t r = (int64_t)blockIdx.x * RPB + (TC > 0 ? threadIdx.x / T : 0);
  if (r >= g.rows) return;   // with TC = 0 whole workgroups
  Raw8<F32> next[U];
  auto load = [&](int64_t row) {
    const void* xr = static_cast<const uint8_t*>(g.x) + row * g.H * (F32 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < U; ++j) next[j] = load8<F32, FULL>(xr, 8 * (int64_t)(j * T + t), g.H);
  };
  load(r);
  float w[KEEP ? U : 1][8], b[KEEP ? U : 1][8];
  if constexpr (KEEP) {
#pragma unroll
    for (int j = 0; j < U; ++j) affine8(g, 8 * (int64_t)(j * T + t), w[j], b[j]);
  }
  const float rs = g.out_kind == 1 ? 1.0f / *g.sy : 0.0f;
  // (the sums' LDS takes turns, so a row's never meets the row before)
  for (; r < g.rows; r += step) {
    float x[U][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      values8<F32>(next[j], x[j]);
      s = __fadd_rn(s, sum8(x[j]));
    }
    if (r + step < g.rows) load(r + step);
    float mean = __fmul_rn(row_sum<TC>(s, red[0]), inv_h);
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[j][k] = __fadd_rn(x[j][k], -mean);
      if (FULL || i + 8 <= g.H) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v = __builtin_fmaf(x[j][k], x[j][k], v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i + k < g.H) v = __builtin_fmaf(x[j][k], x[j][k], v);
      }
    }
    float var = __fmul_rn(row_sum<TC>(v, red[1]), inv_h);
    if (__builtin_expect(off_centre(mean, var, g.eps), 0)) {
      float c = 0.0f;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t i = 8 * (int64_t)(j * T + t);
        if (FULL || i + 8 <= g.H) {
          c = __fadd_rn(c, sum8(x[j]));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i + k < g.H) c = __fadd_rn(c, x[j][k]);
        }
      }
      const float off = __fmul_rn(row_sum<TC>(c, red[2]), inv_h);
      var = centred(var, off);
      mean = __fadd_rn(mean, off);
      const bool flat = __fadd_rn(var, g.eps) == 0.0f;   // 0 * Inf below, whatever off's roundings left
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[j][k] = flat ? 0.0f : __fadd_rn(x[j][k], -off);
    }
    const float rstd = 1.0f / __fsqrt_rn(__fadd_rn(var, g.eps));
    if (t == 0) {
      if (g.mean != nullptr) g.mean[r] = mean;
      if (g.rstd != nullptr) g.rstd[r] = rstd;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
      if (FULL || i < g.H) {
        if constexpr (!KEEP) affine8(g, i, w[0], b[0]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[j][k] = __builtin_fmaf(__fmul_rn(x[j][k], rstd), w[KEEP ? j : 0][k], b[KEEP ? j : 0][k]);
        emit8(g, r * g.H, i, rs, x[j]);
      }
    }
  }
}

// Rows too long for registers: read three times (four where the
// mean is corrected), from cache after the first.
template <bool F32>
__global__ __launch_bounds__(1024) void layer_norm_long_kernel(LayerNormArgs g) {
  __shared__ float red[3][16];
  const float inv_h = 1.0f / (float)g.H;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
  const int64_t base = r * g.H;
  const void* xr = static_cast<const uint8_t*>(g.x) + base * (F32 ? 4 : 2);
  LongSum s, v;
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    float f[8];
    values8<F32>(load8<F32>(xr, i, g.H), f);
    s.add(sum8(f));
  }
  const float mean = __fmul_rn(row_sum<0>(s.s, red[0]), inv_h);
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    float f[8];
    values8<F32>(load8<F32>(xr, i, g.H), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = i + k < g.H ? __fadd_rn(f[k], -mean) : 0.0f;
      f[k] = __fmul_rn(d, d);
    }
    v.add(sum8(f));
  }
  float var = __fmul_rn(row_sum<0>(v.s, red[1]), inv_h), off = 0.0f;
  if (off_centre(mean, var, g.eps)) {
    LongSum c;
    for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
      float f[8];
      values8<F32>(load8<F32>(xr, i, g.H), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = i + k < g.H ? __fadd_rn(f[k], -mean) : 0.0f;
      c.add(sum8(f));
    }
    off = __fmul_rn(row_sum<0>(c.s, red[2]), inv_h);
    var = centred(var, off);
  }
  const float rstd = 1.0f / __fsqrt_rn(__fadd_rn(var, g.eps));
  const bool flat = off != 0.0f && __fadd_rn(var, g.eps) == 0.0f;   // 0 * Inf below, whatever off's roundings left
  if (threadIdx.x == 0) {
    if (g.mean != nullptr) g.mean[r] = __fadd_rn(mean, off);
    if (g.rstd != nullptr) g.rstd[r] = rstd;
  }
  const float rs = g.out_kind == 1 ? 1.0f / *g.sy : 0.0f;
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    float f[8];
    values8<F32>(load8<F32>(xr, i, g.H), f);
    float w[8], b[8];
    affine8(g, i, w, b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float d = flat ? 0.0f : __fadd_rn(__fadd_rn(f[k], -mean), -off);
      f[k] = __builtin_fmaf(__fmul_rn(d, rstd), w[k], b[k]);
    }
    emit8(g, base, i, rs, f);
  }
  }
}

// Backward pass.  T threads cover a row, U groups of eight columns each (TC:
// 16 or 64, and as many rows side by side as the workgroup holds; or 0: the
// whole workgroup, any number of waves).  They walk the rows of the workgroup's
// slab: the row's two sums through one barrier, dx, and the columns' sums of
// dy xh and dy, which go to rows `slab` of out_w and out_b (2 H floats apart;
// NULL: not needed) at the end.  The next row's x, dy and dres are on their way
// during this row's sums; the guards of a row that ends inside a group must not
// make a wave wait for each load in turn (8000x6000 BF16 123 us so, 91 with
// load8_ahead).  FULL: the groups are exactly the row.  16384x5120 BF16 with
// dres: 141 us, 4.7 TB/s.
template <bool XF, bool DF, int TC, int U, bool FULL>
__global__ __launch_bounds__(1024) void layer_norm_backward_kernel(LayerNormBwdArgs g, int64_t slab_rows,
                                                                    float* out_w, float* out_b) {
  // two groups: a row stays in its raw form over its sums and is worked out
  // again for dx, and FP32 rows are not loaded ahead: 128 registers hold no more
  constexpr bool AGAIN = U > 1, AHEAD = U == 1 || (!XF && !DF);
  const int G = TC > 0 ? (int)blockDim.x / TC : 1;   // rows side by side
  __shared__ float red[2][2][16];
  __shared__ f4 cols[TC > 0 ? 4 * 512 : 1];          // half the threads' sums
  __shared__ f4 sums[AGAIN ? 4 * U * 1024 : 1];      // [dw, db][U][half][threads]: each thread's own
  const int T = TC > 0 ? TC : blockDim.x, waves = T >> 6, t = TC > 0 ? threadIdx.x % TC : threadIdx.x;
  const float inv_h = 1.0f / (float)g.H;
  const int64_t r0 = (int64_t)blockIdx.x * slab_rows;
  const int64_t r1 = r0 + slab_rows < g.rows ? r0 + slab_rows : g.rows;
  float w[U][8], sw[AGAIN ? 1 : U][8], sb[AGAIN ? 1 : U][8];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = 8 * (int64_t)(j * T + t);
    if (g.w != nullptr) load8_values(g.w, g.w_f32, i, g.H, w[j]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (g.w == nullptr) w[j][k] = 1.0f;
      if constexpr (!AGAIN) sw[j][k] = sb[j][k] = 0.0f;
    }
    if constexpr (AGAIN)
      for (int q = 0; q < 4; ++q) sums[(4 * j + q) * 1024 + t] = (f4){0.0f, 0.0f, 0.0f, 0.0f};
  }
  Raw8<XF> x[U], rs[U];
  Raw8<DF> d[U];
  float mean = 0.0f, rstd = 0.0f;
  // last: what a group holds past the row's end, its last element or zeros
  auto load8_of = [&](auto& to, const void* from, int64_t base, int64_t i, auto last) {
    constexpr bool F = sizeof(to) == 32;
    const void* row = static_cast<const uint8_t*>(from) + base * (F ? 4 : 2);
    to = TC == 16 || FULL ? load8<F, FULL, decltype(last)::value>(row, i, g.H) : load8_ahead<F>(row, i, g.H);
  };
  auto load_res = [&](int64_t r) {
    if (g.dres == nullptr) return;
#pragma unroll
    for (int j = 0; j < U; ++j) load8_of(rs[j], g.dres, r * g.H, 8 * (int64_t)(j * T + t), std::false_type{});
  };
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      load8_of(x[j], g.x, r * g.H, 8 * (int64_t)(j * T + t), std::true_type{});
      load8_of(d[j], g.dy, r * g.H, 8 * (int64_t)(j * T + t), std::false_type{});
    }
    mean = g.mean[r];
    rstd = g.rstd[r];
  };
  // xh and g of a group, from its raw elements
  auto group = [&](const Raw8<XF>& xr, const Raw8<DF>& dr, float mean_r, float rstd_r, int j, float* dy, float* xh,
                   float* gw) {
    values8<XF>(xr, xh);
    values8<DF>(dr, dy);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      xh[k] = __fmul_rn(__fadd_rn(xh[k], -mean_r), rstd_r);
      gw[k] = __fmul_rn(dy[k], w[j][k]);
    }
  };
  int64_t r = r0 + (TC > 0 ? threadIdx.x / TC : 0);
  if (r < r1) {
    load(r);
    if constexpr (!AGAIN) load_res(r);
  }
  for (int buf = 0; r < r1; r += G, buf ^= 1) {
    float xh[U][8], gw[U][8], res[U][8];
    Raw8<XF> x_now[U];
    Raw8<DF> d_now[U];
    const float mean_r = mean, rstd_r = rstd;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float dy[8];
      const int64_t i = 8 * (int64_t)(j * T + t);
      if constexpr (TC != 16 && !FULL) {
        shift8<XF, true>(x[j], i, g.H);
        shift8<DF>(d[j], i, g.H);
        if (!AGAIN && g.dres != nullptr) shift8<XF>(rs[j], i, g.H);
      }
      x_now[j] = x[j];
      d_now[j] = d[j];
      if (!AGAIN && g.dres != nullptr) values8<XF>(rs[j], res[j]);
      // columns past H: dy is 0 there and xh the row's last, as finite as that
      // (of x = 0, -mean rstd could overflow and 0 Inf reach the sums), so they
      // add nothing to the row's sums
      group(x[j], d[j], mean_r, rstd_r, j, dy, xh[j], gw[j]);
#pragma unroll
      for (int k = 0; k < 8; ++k) s1 = __fadd_rn(s1, gw[j][k]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s2 = __builtin_fmaf(gw[j][k], xh[j][k], s2);
        if constexpr (!AGAIN) {
          sw[j][k] = __builtin_fmaf(dy[k], xh[j][k], sw[j][k]);
          sb[j][k] = __fadd_rn(sb[j][k], dy[k]);
        }
      }
      if constexpr (AGAIN) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f4 a = sums[(4 * j + q) * 1024 + t];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float dk = dy[4 * (q & 1) + k];
            a[k] = q < 2 ? __builtin_fmaf(dk, xh[j][4 * (q & 1) + k], a[k]) : __fadd_rn(a[k], dk);
          }
          sums[(4 * j + q) * 1024 + t] = a;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (AGAIN) load_res(r);
    if constexpr (AHEAD) {
      if (r + G < r1) {
        load(r + G);
        if constexpr (!AGAIN) load_res(r + G);
      }
    }
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
      if (FULL || i < g.H) {
        float y[8];
        if constexpr (AGAIN) {
          float dy[8];
          for (u4& q : x_now[j].q) asm volatile("" : "+v"(q));   // not kept from above
          for (u4& q : d_now[j].q) asm volatile("" : "+v"(q));
          group(x_now[j], d_now[j], mean_r, rstd_r, j, dy, xh[j], gw[j]);
          if (g.dres != nullptr) {
            if constexpr (!FULL) shift8<XF>(rs[j], i, g.H);
            values8<XF>(rs[j], res[j]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          y[k] = __fmul_rn(rstd_r, __builtin_fmaf(-xh[j][k], c2, __fadd_rn(gw[j][k], -c1)));
          if (g.dres != nullptr) y[k] = __fadd_rn(y[k], res[j][k]);
        }
        if constexpr (XF) store8_f32(static_cast<float*>(g.dx) + r * g.H, i, g.H, y);
        else store8_bf16(static_cast<uint16_t*>(g.dx) + r * g.H, i, g.H, y);
      }
    }
    if constexpr (!AHEAD) {
      if (r + G < r1) load(r + G);
    }
  }
  const int64_t at = (int64_t)blockIdx.x * 2 * g.H;
  if constexpr (TC > 0) {
    // the rows side by side (a power of two) are added in a tree
    static_assert(U == 1, "");
    if (out_w == nullptr && out_b == nullptr) return;
    const int q = threadIdx.x / TC;
    for (int h = G >> 1; h > 0; h >>= 1) {
      const int at4 = (q & (h - 1)) * TC + t, n4 = h * TC;
      if (q >= h && q < 2 * h) {
        cols[at4] = (f4){sw[0][0], sw[0][1], sw[0][2], sw[0][3]};
        cols[n4 + at4] = (f4){sw[0][4], sw[0][5], sw[0][6], sw[0][7]};
        cols[2 * n4 + at4] = (f4){sb[0][0], sb[0][1], sb[0][2], sb[0][3]};
        cols[3 * n4 + at4] = (f4){sb[0][4], sb[0][5], sb[0][6], sb[0][7]};
      }
      __syncthreads();
      if (q < h) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sw[0][k] = __fadd_rn(sw[0][k], cols[(k >> 2) * n4 + at4][k & 3]);
          sb[0][k] = __fadd_rn(sb[0][k], cols[(2 + (k >> 2)) * n4 + at4][k & 3]);
        }
      }
      __syncthreads();
    }
    if (q == 0 && 8 * t < g.H) {
      if (out_w != nullptr) store8_f32(out_w + at, 8 * t, g.H, sw[0]);
      if (out_b != nullptr) store8_f32(out_b + at, 8 * t, g.H, sb[0]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
      if (i < g.H) {
        if constexpr (AGAIN) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            sw[0][k] = sums[(4 * j + k / 4) * 1024 + t][k & 3];
            sb[0][k] = sums[(4 * j + 2 + k / 4) * 1024 + t][k & 3];
          }
        }
        if (out_w != nullptr) store8_f32(out_w + at, i, g.H, sw[AGAIN ? 0 : j]);
        if (out_b != nullptr) store8_f32(out_b + at, i, g.H, sb[AGAIN ? 0 : j]);
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
  LongSum s1, s2;
  float xh[8], gw[8];
  for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
    row8(i, xh, gw);
    s1.add(sum8(gw));
#pragma unroll
    for (int k = 0; k < 8; ++k) xh[k] = __fmul_rn(gw[k], xh[k]);
    s2.add(sum8(xh));
  }
  const float c1 = __fmul_rn(row_sum<0>(s1.s, red[0]), inv_h), c2 = __fmul_rn(row_sum<0>(s2.s, red[1]), inv_h);
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

template <bool F32, int TC, int U>
hipError_t run_norm(const LayerNormArgs& g, int threads, hipStream_t stream) {
  const int rpb = TC > 0 ? 256 / (TC > 0 ? TC : 1) : 1;
  // as many workgroups as are resident at once (256 CUs, 16 or 20 waves each)
  const int waves = threads / 64, room = U <= 2 ? 20 : 16;
  const int64_t most = 256 * (waves > room ? 1 : room / waves);
  const dim3 grid(row_grid((g.rows + rpb - 1) / rpb, most));
  if (TC == 0 && g.H == (int64_t)threads * U * 8)
    hipLaunchKernelGGL((layer_norm_kernel<F32, TC, U, TC == 0>), grid, dim3(threads), 0, stream, g);
  else
    hipLaunchKernelGGL((layer_norm_kernel<F32, TC, U, false>), grid, dim3(threads), 0, stream, g);
  return hipGetLastError();
}

// Few rows: one group of eight per thread, so that a row's latency is least.
// Many: two or three, which halves the sums over waves, in workgroups of four
// waves or a multiple: five or six would load the SIMDs unevenly (8000x6000
// BF16 -> E4M3 in 256 threads of three groups 35 us, in 384 of two 47;
// 4096x4096 in 256 of two 14.2, in 128 of four 15.5, in 512 of one 16.1).
template <bool F32>
hipError_t norm_of_type(const LayerNormArgs& g, hipStream_t stream) {
  const int64_t units = (g.H + 7) / 8;
  if (units <= 16) return run_norm<F32, 16, 1>(g, 256, stream);
  if (units <= 64) return run_norm<F32, 64, 1>(g, 256, stream);
  if (g.rows <= 512) {
    if (units <= 1024) return run_norm<F32, 0, 1>(g, (int)((units + 63) / 64 * 64), stream);
  } else {
    if (units <= 128) return run_norm<F32, 64, 2>(g, 256, stream);
    if (units <= 256) return run_norm<F32, 0, 1>(g, 256, stream);
    if (units <= 512) return run_norm<F32, 0, 2>(g, 256, stream);
    if (units <= 768) return run_norm<F32, 0, 3>(g, 256, stream);
    if (units <= 1024) return run_norm<F32, 0, 2>(g, 512, stream);
    if (units <= 1536) return run_norm<F32, 0, 3>(g, 512, stream);
  }
  if (units <= 2048) return run_norm<F32, 0, 2>(g, 1024, stream);
  if (units <= 4096) return run_norm<F32, 0, 4>(g, 1024, stream);
  hipLaunchKernelGGL((layer_norm_long_kernel<F32>), dim3(row_grid(g.rows, 1 << 20)), dim3(1024), 0, stream, g);
  return hipGetLastError();
}

// rows of up to this many elements go through layer_norm_backward_kernel
constexpr int64_t kBwdRegs = 1024 * 8 * 2;

// How the backward pass covers rows of H elements: threads of a workgroup,
// rows side by side in it, groups of eight per thread (one up to 8192 columns,
// then two), and slabs.  One workgroup of eight waves or more per CU, two of
// three to seven, three of fewer: more slabs cost more in partial sums than
// they hide (4096x4096 FP32 41.7 us with 256 slabs, 44.3 with 512; 4000x2600
// BF16 38.5, 29.6; 4096x1024 18.8, 14.4).  For the same reason a slab's rows
// are one, two or at least four one after another (64x4096 6.5, 7.0, 8.6;
// 256x4096 11.3, 9.0, 9.7; 512x4096 13.6, 13.6, 12.5; 777x2053 17.7, 16.2,
// 14.1); narrow rows, which go side by side, need no second (5000x100 8.2, 9.2,
// 11.6).  They take 1024 threads to a workgroup where there are enough of them.
// A few rows are one slab, whose sums need no second launch: that takes 3.3 us
// of the host and more of the GPU's time than four rows of 4096 save side by
// side (a call 9.8 -> 6.8 us, its kernels 5.3 -> 6.3; 6x256 5.2 -> 3.7).
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
    b.threads = (int)((units + 64 * b.groups - 1) / (64 * b.groups) * 64);
  }
  // (rows beyond registers: eight workgroups per CU over columns and slabs)
  if (H > kBwdRegs) {
    const int64_t across = (H + 2047) / 2048, room = 2048 / across;
    b.slabs = room < 1 ? 1 : room < 256 ? room : 256;
    const int64_t most = (rows + 3) / 4;
    if (b.slabs > most) b.slabs = most;
    return b;
  }
  const int waves = b.threads / 64;
  b.slabs = waves >= 8 ? 256 : waves >= 3 ? 512 : 768;
  if (rows <= (H <= 4096 ? 4 : 2) * b.side) {
    b.slabs = 1;
    return b;
  }
  const int64_t walk = b.side > 1 || rows <= 64 ? 1 : rows <= 256 ? 2 : 4;
  const int64_t most = (rows + walk * b.side - 1) / (walk * b.side);
  if (b.slabs > most) b.slabs = most;
  return b;
}

template <bool XF, bool DF, int TC, int U>
hipError_t run_backward_kernel(const LayerNormBwdArgs& g, int threads, int64_t slabs, float* out_w, float* out_b,
                               hipStream_t stream) {
  const int64_t slab_rows = (g.rows + slabs - 1) / slabs;
  if (TC == 0 && g.H == (int64_t)threads * U * 8)
    hipLaunchKernelGGL((layer_norm_backward_kernel<XF, DF, TC, U, TC == 0>), dim3((unsigned)slabs), dim3(threads), 0,
                       stream, g, slab_rows, out_w, out_b);
  else
    hipLaunchKernelGGL((layer_norm_backward_kernel<XF, DF, TC, U, false>), dim3((unsigned)slabs), dim3(threads), 0,
                       stream, g, slab_rows, out_w, out_b);
  return hipGetLastError();
}

template <bool XF, bool DF>
hipError_t run_backward(const LayerNormBwdArgs& g, int64_t slabs, float* out_w, float* out_b, hipStream_t stream) {
  const BwdShape b = bwd_shape(g.rows, g.H);
  if (g.H <= 128) return run_backward_kernel<XF, DF, 16, 1>(g, b.threads, slabs, out_w, out_b, stream);
  if (g.H <= 512) return run_backward_kernel<XF, DF, 64, 1>(g, b.threads, slabs, out_w, out_b, stream);
  if (b.groups == 1) return run_backward_kernel<XF, DF, 0, 1>(g, b.threads, slabs, out_w, out_b, stream);
  return run_backward_kernel<XF, DF, 0, 2>(g, b.threads, slabs, out_w, out_b, stream);
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

// (one slab's sums are the results, where registers hold the row)
int64_t layer_norm_backward_partials(int64_t rows, int64_t H) {
  const int64_t slabs = rows == 0 || H == 0 ? 0 : bwd_shape(rows, H).slabs;
  return slabs == 1 && H <= kBwdRegs ? 0 : slabs;
}

hipError_t launch_layer_norm_backward(const LayerNormBwdArgs& g, float* dw, float* db, float* part,
                                      hipStream_t stream) {
  const int64_t slabs = g.rows == 0 ? 0 : bwd_shape(g.rows, g.H).slabs;
  const bool sums = dw != nullptr || db != nullptr;
  hipError_t e = hipSuccess;
  if (slabs > 0 && g.H <= kBwdRegs) {
    const bool direct = slabs == 1;
    float* ow = dw == nullptr ? nullptr : (direct ? dw : part);
    float* ob = db == nullptr ? nullptr : (direct ? db : part + g.H);
    if (g.x_f32) e = g.dy_f32 ? run_backward<true, true>(g, slabs, ow, ob, stream) : run_backward<true, false>(g, slabs, ow, ob, stream);
    else e = g.dy_f32 ? run_backward<false, true>(g, slabs, ow, ob, stream) : run_backward<false, false>(g, slabs, ow, ob, stream);
    if (direct) return e;
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
