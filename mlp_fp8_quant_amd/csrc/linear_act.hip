// FP8 Linear with bias, activation and residual in its epilogue, and that
// epilogue's backward pass (declared in include/fp8mot.h as fp8_linear_act
// and fp8_linear_act_backward).
//
//   acc[m,n] = sum_k dec(qx[m,k]) dec(qw[n,k])          (FP32 accumulation)
//   z        = fp32(acc * alpha) + bias[n],  alpha = fp32(s_x s_w)
//   y        = act(z) + residual[m,n]  -> BF16, E4M3(y / s_y) or FP32
//   dz       = dy act'(z),  dbias[n] = sum_m dz[m,n]
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "device_common.h"
#include "kernels.h"

namespace fp8mot {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Eight E4M3 codes (two dwords) -> eight F16 values with the gfx950 packed
// conversion at scale 1.0: every E4M3 value is exactly an F16 value, and the
// NaN codes become an F16 NaN.
__device__ __forceinline__ f16x8 decode8(int lo, int hi) {
  return __builtin_bit_cast(
      f16x8, (v4i){__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)lo, 1.0f, false)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)lo, 1.0f, true)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)hi, 1.0f, false)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)hi, 1.0f, true))});
}

__device__ __forceinline__ float load_elem(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

__device__ __forceinline__ uint16_t bf16_of(float v) { return (uint16_t)bf16x2_rne(v, v); }

// One output element from its sum.
__device__ __forceinline__ void finish(const LinearActArgs& g, int64_t m, int64_t n, float acc) {
  const float alpha = g.row_scales ? __fmul_rn(g.sx[m], g.sw[n]) : __fmul_rn(*g.sx, *g.sw);
  float z = __fmul_rn(acc, alpha);
  if (g.bias != nullptr) z = __fadd_rn(z, load_elem(g.bias, g.bias_f32, n));
  const int64_t i = m * g.N + n;
  if (g.pre != nullptr) g.pre[i] = bf16_of(z);
  float y = act_value(z, g.act);
  if (g.residual != nullptr) y = __fadd_rn(y, load_elem(g.residual, g.residual_f32, i));
  if (g.out_kind == 0) static_cast<uint16_t*>(g.y)[i] = bf16_of(y);
  else if (g.out_kind == 1) static_cast<uint8_t*>(g.y)[i] = (uint8_t)e4m3_encode(y / *g.sy);   // IEEE division
  else static_cast<float*>(g.y)[i] = y;
}

// A workgroup computes 16 * MB rows of X against 16 rows of W, straight from
// memory: its NW waves take the 64-K chunks in turn and their sums are added
// through LDS in wave order.  A lane reads 16 bytes of one row of W and of
// each 16-row block of X (row lane % 16, K position 16 * (lane / 16) of the
// chunk) and feeds bytes 0..7 to one 16x16x32 F16 MFMA and bytes 8..15 to the
// next, W as its first operand: accumulator register v of lane l is then
// column n = 4 * (l / 16) + v of row m = l % 16.
constexpr int kWaves = 8;

template <int MB>
__global__ __launch_bounds__(kWaves * 64) void linear_rows_kernel(LinearActArgs g) {
  __shared__ v4f red[kWaves][MB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l15 = lane & 15, kq = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const bool n_ok = n0 + l15 < g.N;
  const uint8_t* wrow = g.qw + (n_ok ? n0 + l15 : 0) * g.K;
  for (int64_t m0 = (int64_t)blockIdx.y * (16 * MB); m0 < g.M; m0 += (int64_t)gridDim.y * (16 * MB)) {
  const uint8_t* xrow[MB];
  bool m_ok[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int64_t m = m0 + 16 * b + l15;
    m_ok[b] = m < g.M;
    xrow[b] = g.qx + (m_ok[b] ? m : 0) * g.K;
  }
  v4f acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t k0 = (int64_t)wave * 64; k0 < g.K; k0 += kWaves * 64) {
    const int64_t k = k0 + 16 * kq;
    const bool k_ok = k < g.K;   // K % 16 == 0: a chunk of 16 lies inside K or past it
    const v4i zero = {0, 0, 0, 0};
    const v4i w = n_ok && k_ok ? *reinterpret_cast<const v4i*>(wrow + k) : zero;
    const f16x8 w0 = decode8(w[0], w[1]), w1 = decode8(w[2], w[3]);
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const v4i x = m_ok[b] && k_ok ? *reinterpret_cast<const v4i*>(xrow[b] + k) : zero;
      acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0, decode8(x[0], x[1]), acc[b], 0, 0, 0);
      acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1, decode8(x[2], x[3]), acc[b], 0, 0, 0);
    }
  }
#pragma unroll
  for (int b = 0; b < MB; ++b) red[wave][b][lane] = acc[b];
  __syncthreads();
  for (int t = threadIdx.x; t < MB * 64; t += kWaves * 64) {
    const int b = t >> 6, l = t & 63;
    v4f s = red[0][b][l];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      const v4f o = red[w][b][l];
#pragma unroll
      for (int v = 0; v < 4; ++v) s[v] = __fadd_rn(s[v], o[v]);
    }
    const int64_t m = m0 + 16 * b + (l & 15), n = n0 + 4 * (l >> 4);
    if (m < g.M) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (n + v < g.N) finish(g, m, n + v, s[v]);
    }
  }
  __syncthreads();   // red is reused by the next rows
  }
}

// dz = dy act'(pre) for kActRows rows of 256 columns, one column per thread,
// with the column's sum over those rows (of dz before its rounding to BF16)
// into part[slab, n].
constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void act_backward_kernel(
    const uint16_t* __restrict__ dy, const uint16_t* __restrict__ pre, int act,
    uint16_t* __restrict__ dz, float* __restrict__ part, int64_t M, int64_t N, int64_t slab_rows) {
  const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (n >= N) return;
  const int64_t r0 = (int64_t)blockIdx.y * slab_rows;
  const int64_t r1 = r0 + slab_rows < M ? r0 + slab_rows : M;
  float s = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    const int64_t i = r * N + n;
    float d = bf16_to_f32(dy[i]);
    if (act != kActNone) d = __fmul_rn(d, act_slope(bf16_to_f32(pre[i]), act));
    if (dz != nullptr) dz[i] = bf16_of(d);
    s = __fadd_rn(s, d);
  }
  if (part != nullptr) part[(int64_t)blockIdx.y * N + n] = s;
}

}  // namespace

size_t linear_act_workspace(int64_t M, int64_t N, int64_t K) {
  (void)M;
  (void)N;
  (void)K;
  return 0;
}

hipError_t launch_linear_act(const LinearActArgs& g, int accum, float* ws, int num_cus, hipStream_t stream) {
  (void)accum;
  (void)ws;
  (void)num_cus;
  const unsigned gx = (unsigned)((g.N + 15) / 16);
  if (g.M <= 16)
    hipLaunchKernelGGL((linear_rows_kernel<1>), dim3(gx, 1), dim3(kWaves * 64), 0, stream, g);
  else
    hipLaunchKernelGGL((linear_rows_kernel<4>), dim3(gx, (unsigned)(g.M < 64 * 4096 ? (g.M + 63) / 64 : 4096)),
                       dim3(kWaves * 64), 0, stream, g);
  return hipGetLastError();
}

int64_t act_backward_slabs(int64_t M, int64_t N) {
  (void)N;
  return M < 64 ? (M > 0 ? 1 : 0) : (M / 64 < 64 ? M / 64 : 64);
}

hipError_t launch_act_backward(const uint16_t* dy, const uint16_t* pre, int act, uint16_t* dz,
                               float* dbias, int64_t M, int64_t N, float* part, hipStream_t stream) {
  const int64_t slabs = act_backward_slabs(M, N);
  if (slabs > 0) {
    const int64_t slab_rows = (M + slabs - 1) / slabs;
    hipLaunchKernelGGL(act_backward_kernel, dim3((unsigned)((N + kThreads - 1) / kThreads), (unsigned)slabs),
                       dim3(kThreads), 0, stream, dy, pre, act, dz, dbias != nullptr ? part : nullptr, M, N,
                       slab_rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (dbias == nullptr) return hipSuccess;
  return launch_sum_slabs(part, dbias, slabs, N, stream);
}

}  // namespace fp8mot
