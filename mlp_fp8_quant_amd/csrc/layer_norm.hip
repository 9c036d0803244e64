// Layer norm over the last dimension and its backward pass (declared in
// include/fp8mot.h as fp8_layer_norm and fp8_layer_norm_backward).
//
//   mean = sum x / H,  var = sum (x - mean)^2 / H,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh w + b  -> BF16, E4M3(y / s_y) or FP32
//   g = dy w:  dx = rstd (g - sum g / H - xh sum(g xh) / H) + dres
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// All sums are FP32; the variance is taken about the mean (not from the
// squares' mean, which cancels where the mean is large).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "kernels.h"

namespace fp8mot {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_elem(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ uint16_t bf16_of(float v) { return (uint16_t)bf16x2_rne(v, v); }

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = __fadd_rn(v, __shfl_xor(v, off, 64));
  __syncthreads();   // red may still be read from the sum before
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) s = __fadd_rn(s, red[w]);
  return s;
}

// One workgroup per row, which it reads three times (from cache after the first).
__global__ __launch_bounds__(kThreads) void layer_norm_kernel(LayerNormArgs g) {
  __shared__ float red[kThreads / 64];
  const float inv_h = 1.0f / (float)g.H;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    const int64_t base = r * g.H;
    float s = 0.0f;
    for (int64_t i = threadIdx.x; i < g.H; i += kThreads) s = __fadd_rn(s, load_elem(g.x, g.x_f32, base + i));
    const float mean = __fmul_rn(block_sum(s, red), inv_h);
    float v = 0.0f;
    for (int64_t i = threadIdx.x; i < g.H; i += kThreads) {
      const float d = __fadd_rn(load_elem(g.x, g.x_f32, base + i), -mean);
      v = __builtin_fmaf(d, d, v);
    }
    const float var = __fmul_rn(block_sum(v, red), inv_h);
    const float rstd = 1.0f / __fsqrt_rn(__fadd_rn(var, g.eps));
    for (int64_t i = threadIdx.x; i < g.H; i += kThreads) {
      float y = __fmul_rn(__fadd_rn(load_elem(g.x, g.x_f32, base + i), -mean), rstd);
      if (g.w != nullptr) y = __fmul_rn(y, load_elem(g.w, g.wb_f32, i));
      if (g.b != nullptr) y = __fadd_rn(y, load_elem(g.b, g.wb_f32, i));
      if (g.out_kind == 0) static_cast<uint16_t*>(g.y)[base + i] = bf16_of(y);
      else if (g.out_kind == 1) static_cast<uint8_t*>(g.y)[base + i] = (uint8_t)e4m3_encode(y / *g.sy);
      else static_cast<float*>(g.y)[base + i] = y;
    }
    if (threadIdx.x == 0) {
      if (g.mean != nullptr) g.mean[r] = mean;
      if (g.rstd != nullptr) g.rstd[r] = rstd;
    }
  }
}

// dx: one workgroup per row.
__global__ __launch_bounds__(kThreads) void layer_norm_dx_kernel(LayerNormBwdArgs g) {
  __shared__ float red[kThreads / 64];
  const float inv_h = 1.0f / (float)g.H;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    const int64_t base = r * g.H;
    const float mean = g.mean[r], rstd = g.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t i = threadIdx.x; i < g.H; i += kThreads) {
      const float xh = __fmul_rn(__fadd_rn(load_elem(g.x, g.x_f32, base + i), -mean), rstd);
      float d = load_elem(g.dy, g.dy_f32, base + i);
      if (g.w != nullptr) d = __fmul_rn(d, load_elem(g.w, g.w_f32, i));
      s1 = __fadd_rn(s1, d);
      s2 = __builtin_fmaf(d, xh, s2);
    }
    const float c1 = __fmul_rn(block_sum(s1, red), inv_h), c2 = __fmul_rn(block_sum(s2, red), inv_h);
    for (int64_t i = threadIdx.x; i < g.H; i += kThreads) {
      const float xh = __fmul_rn(__fadd_rn(load_elem(g.x, g.x_f32, base + i), -mean), rstd);
      float d = load_elem(g.dy, g.dy_f32, base + i);
      if (g.w != nullptr) d = __fmul_rn(d, load_elem(g.w, g.w_f32, i));
      float v = __fmul_rn(rstd, __builtin_fmaf(-xh, c2, __fadd_rn(d, -c1)));
      if (g.dres != nullptr) v = __fadd_rn(v, load_elem(g.dres, g.x_f32, base + i));
      if (g.x_f32) static_cast<float*>(g.dx)[base + i] = v;
      else static_cast<uint16_t*>(g.dx)[base + i] = bf16_of(v);
    }
  }
}

// Column sums of dy xh and dy over a slab of rows: part[slab, 0:H) and [H:2H).
__global__ __launch_bounds__(kThreads) void layer_norm_dw_kernel(LayerNormBwdArgs g, int64_t slab_rows,
                                                                 float* __restrict__ part) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= g.H) return;
  const int64_t r0 = (int64_t)blockIdx.y * slab_rows;
  const int64_t r1 = r0 + slab_rows < g.rows ? r0 + slab_rows : g.rows;
  float sw = 0.0f, sb = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const float xh = __fmul_rn(__fadd_rn(load_elem(g.x, g.x_f32, r * g.H + i), -g.mean[r]), g.rstd[r]);
    const float d = load_elem(g.dy, g.dy_f32, r * g.H + i);
    sw = __builtin_fmaf(d, xh, sw);
    sb = __fadd_rn(sb, d);
  }
  float* p = part + (int64_t)blockIdx.y * 2 * g.H;
  p[i] = sw;
  p[g.H + i] = sb;
}

// out[n] = sum over slabs of part[slab, n], in slab order (row stride ld).
__global__ __launch_bounds__(kThreads) void sum_slabs_kernel(const float* __restrict__ part,
                                                             float* __restrict__ out, int64_t slabs,
                                                             int64_t N, int64_t ld) {
  const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (n >= N) return;
  float s = 0.0f;
  for (int64_t p = 0; p < slabs; ++p) s = __fadd_rn(s, part[p * ld + n]);
  out[n] = s;
}

}  // namespace

hipError_t launch_sum_slabs(const float* part, float* out, int64_t slabs, int64_t N, hipStream_t stream) {
  hipLaunchKernelGGL(sum_slabs_kernel, dim3((unsigned)((N + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                     stream, part, out, slabs, N, N);
  return hipGetLastError();
}

hipError_t launch_layer_norm(const LayerNormArgs& g, int num_cus, hipStream_t stream) {
  const int64_t most = (int64_t)num_cus * 64;
  hipLaunchKernelGGL(layer_norm_kernel, dim3((unsigned)(g.rows < most ? g.rows : most)), dim3(kThreads), 0,
                     stream, g);
  return hipGetLastError();
}

int64_t layer_norm_backward_slabs(int64_t rows, int64_t H) {
  (void)H;
  return rows < 32 ? (rows > 0 ? 1 : 0) : (rows / 32 < 256 ? rows / 32 : 256);
}

hipError_t launch_layer_norm_backward(const LayerNormBwdArgs& g, float* dw, float* db, float* part,
                                      int num_cus, hipStream_t stream) {
  const int64_t slabs = layer_norm_backward_slabs(g.rows, g.H);
  const unsigned gx = (unsigned)((g.H + kThreads - 1) / kThreads);
  if (slabs > 0) {
    const int64_t most = (int64_t)num_cus * 64;
    // the column sums first: dx may be written over dy or x
    if (dw != nullptr || db != nullptr)
      hipLaunchKernelGGL(layer_norm_dw_kernel, dim3(gx, (unsigned)slabs), dim3(kThreads), 0, stream, g,
                         (g.rows + slabs - 1) / slabs, part);
    hipLaunchKernelGGL(layer_norm_dx_kernel, dim3((unsigned)(g.rows < most ? g.rows : most)),
                       dim3(kThreads), 0, stream, g);
  }
  if (dw != nullptr)
    hipLaunchKernelGGL(sum_slabs_kernel, dim3(gx), dim3(kThreads), 0, stream, part, dw, slabs, g.H, 2 * g.H);
  if (db != nullptr)
    hipLaunchKernelGGL(sum_slabs_kernel, dim3(gx), dim3(kThreads), 0, stream, part + g.H, db, slabs, g.H,
                       2 * g.H);
  return hipGetLastError();
}

}  // namespace fp8mot
