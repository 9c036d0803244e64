// The norms before and after a block, fused with the block's gate and residual
// scale, and their backward pass (declared in include/fp8mot.h as
// fp8_residual_norm and fp8_residual_norm_backward).
//
//   forward   z = h rs_h (or h),  rs_h = 1 / sqrt(sum h^2 / H + eps)
//             r = x + z (alpha gate pw)               the residual stream
//             y = r rs w,  rs = 1 / sqrt(sum r^2 / H + eps)
//   backward  g = dy w,  n = r rs,  z = h rs_h (or h)
//             dx = rs (g - n sum(g n) / H) + dr,  p = dx (alpha gate pw)
//             dh = rs_h (p - z sum(p z) / H)  (or p)
//             dw = sum_rows dy n,  A = sum of dx z over a gate's rows:
//             dgate = alpha pw A,  dpw = sum_gates alpha gate A
//
// Everything between the reads and the stores is FP32; y and rs are taken from
// r before its rounding to the stream's type.  Bound by memory: a row is read
// once and kept in registers over its sums.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "block_scale.h"
#include "device_common.h"
#include "kernels.h"
#include "rowwise.h"

namespace fp8mot {

namespace {

using namespace rows;
using block::kBlock;

template <bool F32>
__device__ __forceinline__ const void* row_at(const void* p, int64_t at) {
  return static_cast<const uint8_t*>(p) + at * (F32 ? 4 : 2);
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t at, int64_t i, int64_t n, const float* f) {
  if constexpr (F32) store8_f32(static_cast<float*>(p) + at, i, n, f);
  else store8_bf16(static_cast<uint16_t*>(p) + at, i, n, f);
}
// Eight values of a parameter of n columns, ones where there is none.
__device__ __forceinline__ void param8(const void* p, int f32, int64_t i, int64_t n, float* f) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 1.0f;
  } else {
    load8_values(p, f32, i, n, f);
  }
}
__device__ __forceinline__ float param1(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ const void* gate_at(const void* gate, int f32, int64_t at) {
  return gate == nullptr ? nullptr : static_cast<const uint8_t*>(gate) + at * (f32 ? 4 : 2);
}

// Sums over the threads that share a row, the same in each (as rows::row_sum, TC
// = 0 the whole workgroup).  Every 16 lanes read the waves' sums side by side,
// zeros where there is no wave, and add them as they add their own: one after
// another they took a quarter of the row's time (8000x6000 BF16 89 -> 85 us,
// backward 512x4096 16.0 -> 13).  Two sets take turns, since a wave may be at the
// next sum while others still read this one.
template <int TC>
struct RowSums {
  float* const red;   // [2][16]
  int turn = 0;
  __device__ __forceinline__ explicit RowSums(float* lds) : red(lds) {
    if constexpr (TC == 0) {
      if (threadIdx.x < 32) red[threadIdx.x] = 0.0f;
      __syncthreads();
    }
  }
  __device__ __forceinline__ float operator()(float v) {
    if constexpr (TC == 16) return sum16(v);
    v = wave_sum(v);
    if constexpr (TC == 0) {
      turn ^= 16;
      if ((threadIdx.x & 63) == 0) red[turn + (threadIdx.x >> 6)] = v;
      __syncthreads();
      v = sum16(red[turn + (threadIdx.x & 15)]);
    }
    return v;
  }
};

__device__ __forceinline__ float root(float sum, float inv_h, float eps) {
  return 1.0f / __fsqrt_rn(__builtin_fmaf(sum, inv_h, eps));
}
__device__ __forceinline__ float square8(const float* f) {
  float q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = __fmul_rn(f[k], f[k]);
  return sum8(q);
}

// Columns i .. i + 7 of row r of y.  For block output sixteen lanes hold a
// block's columns, and all of them come here (those past the row's end with
// zeros: they write the padding).
__device__ __forceinline__ void emit8(const ResidualNormArgs& g, int64_t r, int64_t i, float rs, float* y) {
  if (g.out_kind == 3) {
    const float s = block::scale_of(block::max16(block::max8(y)));
    block::quotients<8>(y, s);
    const int64_t Hp = (g.H + 15) / 16 * 16;
    if (i < Hp) store8_fp8(static_cast<uint8_t*>(g.y) + r * Hp, i, Hp, y);
    if (i % kBlock == 0 && i < g.H) g.scales[r * ((g.H + kBlock - 1) / kBlock) + i / kBlock] = s;
  } else if (i < g.H) {
    if (g.out_kind == 0) {
      store8_bf16(static_cast<uint16_t*>(g.y) + r * g.H, i, g.H, y);
    } else if (g.out_kind == 1) {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = __fmul_rn(y[k], rs);
      store8_fp8(static_cast<uint8_t*>(g.y) + r * g.H, i, g.H, y);
    } else {
      store8_f32(static_cast<float*>(g.y) + r * g.H, i, g.H, y);
    }
  }
}

// (alpha gate) pw of eight columns: what the block's output is multiplied by, as
// one factor, which a walk over rows of one gate forms once.
template <class Args>
__device__ __forceinline__ void factor8(const Args& g, int64_t gate, int64_t i, float* f) {
  float pw[8];
  param8(gate_at(g.gate, g.gate_f32, gate * g.H), g.gate_f32, i, g.H, f);
  param8(g.post_w, g.w_f32, i, g.H, pw);
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(__fmul_rn(g.alpha, f[k]), pw[k]);
}

// T threads cover a row, U groups of eight columns each.  TC: 16 or 64 of
// them, NT / TC rows side by side in a workgroup; or 0: the whole workgroup.  A
// workgroup walks `walk` rows (of each side) that lie together, so that a gate is
// seldom another one: the next row is on its way while this one is summed, and
// the norms' weights and the gate stay in registers.  FULL: the groups are exactly
// the row.  16384x5120 BF16 with 8 gates -> BF16 141 us, 4.8 TB/s, bound by memory;
// -> block codes 137 us, 4.3 TB/s, also by what lies between a row's sums and its
// codes; x alone -> BF16 67 us, 5.0 TB/s, -> codes 80.
template <bool XF, bool HF, int TC, int U, int NT, bool FULL>
__global__ __launch_bounds__(NT) void residual_norm_kernel(ResidualNormArgs g, int64_t walk) {
  __shared__ float red[32];
  constexpr int RPB = TC > 0 ? NT / (TC > 0 ? TC : 1) : 1;
  const int T = TC > 0 ? TC : blockDim.x, t = TC > 0 ? threadIdx.x % T : threadIdx.x;
  const bool has_h = g.h != nullptr, post = g.post_w != nullptr;
  const int64_t first = (int64_t)blockIdx.x * RPB * walk + (TC > 0 ? threadIdx.x / T : 0);
  const int64_t end = (int64_t)(blockIdx.x + 1) * RPB * walk < g.rows ? (int64_t)(blockIdx.x + 1) * RPB * walk : g.rows;
  if (first >= end) return;   // with TC = 0 whole workgroups
  Raw8<XF> nx[U];
  Raw8<HF> nh[U];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
      nx[j] = load8<XF, FULL>(row_at<XF>(g.x, r * g.H), i, g.H);
      if (has_h) nh[j] = load8<HF, FULL>(row_at<HF>(g.h, r * g.H), i, g.H);
    }
  };
  load(first);
  float w[U][8], f[U][8];
  auto gate_of = [&](int64_t r) { return (int)((uint32_t)r / (uint32_t)g.gate_rows); };
  int gate = gate_of(first);
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = 8 * (int64_t)(j * T + t);
    param8(g.w, g.w_f32, i, g.H, w[j]);
    if (has_h) factor8(g, gate, i, f[j]);
  }
  const float inv_h = 1.0f / (float)g.H, rs = g.out_kind == 1 ? 1.0f / *g.sy : 0.0f;
  RowSums<TC> total(red);
  for (int64_t r = first; r < end; r += RPB) {
    float v[U][8], h[U][8];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      values8<XF>(nx[j], v[j]);
      if (has_h) values8<HF>(nh[j], h[j]);
    }
    if (r + RPB < end) load(r + RPB);
    if (has_h) {
      float post_rs = 1.0f;
      if (post) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < U; ++j) s = __fadd_rn(s, square8(h[j]));
        post_rs = root(total(s), inv_h, g.eps);
        if (t == 0 && g.post_rstd != nullptr) g.post_rstd[r] = post_rs;
      }
      const int now = gate_of(r);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t i = 8 * (int64_t)(j * T + t);
        if (now != gate) factor8(g, now, i, f[j]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (post) h[j][k] = __fmul_rn(h[j][k], post_rs);
          v[j][k] = __builtin_fmaf(h[j][k], f[j][k], v[j][k]);
        }
        if (FULL || i < g.H) store8<XF>(g.r, r * g.H, i, g.H, v[j]);
      }
      gate = now;
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) s = __fadd_rn(s, square8(v[j]));
    const float rstd = root(total(s), inv_h, g.eps);
    if (t == 0 && g.rstd != nullptr) g.rstd[r] = rstd;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = 8 * (int64_t)(j * T + t);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = __fmul_rn(__fmul_rn(v[j][k], rstd), w[j][k]);
      emit8(g, r, i, rs, v[j]);
    }
  }
}

// Rows too long for registers: x and h are read again for every sum, from cache
// after the first.
template <bool XF, bool HF>
__global__ __launch_bounds__(1024) void residual_norm_long_kernel(ResidualNormArgs g) {
  __shared__ float red[32];
  const float inv_h = 1.0f / (float)g.H, rs = g.out_kind == 1 ? 1.0f / *g.sy : 0.0f;
  const bool has_h = g.h != nullptr, post = g.post_w != nullptr;
  const int64_t end = (g.H + 8 * 1024 - 1) / (8 * 1024) * (8 * 1024);   // whole workgroups, for the block output
  RowSums<0> total(red);
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    const int64_t base = r * g.H;
    float post_rs = 1.0f;
    if (has_h && post) {
      LongSum s;
      for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
        float h[8];
        values8<HF>(load8<HF>(row_at<HF>(g.h, base), i, g.H), h);
        s.add(square8(h));
      }
      post_rs = root(total(s.s), inv_h, g.eps);
      if (threadIdx.x == 0 && g.post_rstd != nullptr) g.post_rstd[r] = post_rs;
    }
    auto stream8 = [&](int64_t i, float* v) {
      values8<XF>(load8<XF>(row_at<XF>(g.x, base), i, g.H), v);
      if (!has_h) return;
      float h[8], f[8];
      values8<HF>(load8<HF>(row_at<HF>(g.h, base), i, g.H), h);
      factor8(g, (int64_t)((uint32_t)r / (uint32_t)g.gate_rows), i, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (post) h[k] = __fmul_rn(h[k], post_rs);
        v[k] = __builtin_fmaf(h[k], f[k], v[k]);
      }
    };
    LongSum s;
    for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
      float v[8];
      stream8(i, v);
      s.add(square8(v));
    }
    const float rstd = root(total(s.s), inv_h, g.eps);
    if (threadIdx.x == 0 && g.rstd != nullptr) g.rstd[r] = rstd;
    for (int64_t i = 8 * (int64_t)threadIdx.x; i < end; i += 8 * 1024) {
      float v[8] = {}, w[8];
      if (i < g.H) {
        stream8(i, v);
        if (has_h) store8<XF>(g.r, base, i, g.H, v);   // over x, where r is x: these columns are done with it
        param8(g.w, g.w_f32, i, g.H, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(__fmul_rn(v[k], rstd), w[k]);
      }
      emit8(g, r, i, rs, v);
    }
  }
}

unsigned row_grid(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

template <bool XF, bool HF, int TC, int U, int NT>
hipError_t run_norm(const ResidualNormArgs& g, int threads, hipStream_t stream) {
  const int rpb = TC > 0 ? NT / (TC > 0 ? TC : 1) : 1;
  // as many workgroups as 24 waves a CU hold (256 CUs) or, but for workgroups of a
  // multiple of three, 20: 4096x4096 BF16 in two of eight waves 26.1, in three 31.2;
  // 8000x6000 in two of twelve 87, in one 114
  const int waves = threads / 64, room = waves % 3 == 0 ? 24 : 20;
  const int64_t most = 256 * (waves > room ? 1 : room / waves), blocks = (g.rows + rpb - 1) / rpb;
  const int64_t walk = (blocks + most - 1) / most;
  const dim3 grid((unsigned)((blocks + walk - 1) / walk));
  if (TC == 0 && g.H == (int64_t)threads * U * 8)
    hipLaunchKernelGGL((residual_norm_kernel<XF, HF, TC, U, NT, TC == 0>), grid, dim3(threads), 0, stream, g, walk);
  else
    hipLaunchKernelGGL((residual_norm_kernel<XF, HF, TC, U, NT, false>), grid, dim3(threads), 0, stream, g, walk);
  return hipGetLastError();
}

// One group of eight per thread while a workgroup holds the row so: two or three
// in fewer threads halve the sums over waves, but leave less in flight
// (16384x5120 BF16 -> block codes 139 us in 640 threads, 158 in 320, 172 in 256).
template <bool XF, bool HF>
hipError_t norm_of_types(const ResidualNormArgs& g, hipStream_t stream) {
  const int64_t units = (g.H + 7) / 8;
  if (units <= 16) return run_norm<XF, HF, 16, 1, 256>(g, 256, stream);
  if (units <= 64) return run_norm<XF, HF, 64, 1, 256>(g, 256, stream);
  if (units <= 512) return run_norm<XF, HF, 0, 1, 512>(g, (int)((units + 63) / 64 * 64), stream);
  if (units <= 1024) return run_norm<XF, HF, 0, 1, 1024>(g, (int)((units + 63) / 64 * 64), stream);
  if (units <= 2048) return run_norm<XF, HF, 0, 2, 1024>(g, 1024, stream);
  hipLaunchKernelGGL((residual_norm_long_kernel<XF, HF>), dim3(row_grid(g.rows, 1 << 20)), dim3(1024), 0, stream, g);
  return hipGetLastError();
}

// ---- backward ----

// The slabs of a launch: per_gate of them cover the rows of each gate, `rows`
// each.  part: [slabs, 2, H up to a multiple of 4] sums over a slab, of dy n and of
// dx z.  Of many gates `together` (else 0) are walked one after another and share
// a slab, whose second sum is then that of alpha gate dx z.
__host__ __device__ inline int64_t part_columns(int64_t H) { return (H + 3) / 4 * 4; }
struct Slabs {
  int64_t per_gate, rows, together, count;
  float* part;
};
// alpha f a: a gradient from the sum a of dx z.
__device__ __forceinline__ void scaled8(float alpha, const float* f, const float* a, float* out) {
#pragma unroll
  for (int k = 0; k < 8; ++k) out[k] = __fmul_rn(__fmul_rn(alpha, f[k]), a[k]);
}
// A slab's column sums go to its part, or, the only slab of all (or of its gate),
// to the results themselves.
__device__ __forceinline__ void put_sums(const ResidualNormBwdArgs& g, const Slabs& s, int64_t slab, int64_t gate,
                                         int64_t i, const float* sw, const float* sa) {
  const bool one = s.count == 1, wanted = g.dpost != nullptr || g.dgate != nullptr;
  float* p = s.part + slab * 2 * part_columns(g.H);
  float f[8];
  if (g.dw != nullptr) store8_f32(one ? g.dw : p, i, g.H, sw);
  if (one && g.dpost != nullptr) {
    param8(gate_at(g.gate, g.gate_f32, gate * g.H), g.gate_f32, i, g.H, f);
    scaled8(g.alpha, f, sa, f);
    store8_f32(g.dpost, i, g.H, f);
  }
  if (s.per_gate == 1 && g.dgate != nullptr) {
    param8(g.post_w, g.w_f32, i, g.H, f);
    scaled8(g.alpha, f, sa, f);
    store8_f32(g.dgate + slab * g.H, i, g.H, f);
  }
  if (!one && wanted) store8_f32(p + part_columns(g.H), i, g.H, sa);
}

// The same where gates share a slab: what a gate's sum of dx z gives, and the
// slab's sums.
__device__ __forceinline__ void put_gate(const ResidualNormBwdArgs& g, int64_t gate, int64_t i, const float* gt,
                                         const float* pw, float* sa, float* sp) {
  float f[8];
  scaled8(g.alpha, pw, sa, f);
  if (g.dgate != nullptr && i < g.H) store8_f32(g.dgate + gate * g.H, i, g.H, f);
  scaled8(g.alpha, gt, sa, f);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    sp[k] = __fadd_rn(sp[k], f[k]);
    sa[k] = 0.0f;
  }
}
__device__ __forceinline__ void put_together(const ResidualNormBwdArgs& g, const Slabs& s, int64_t slab, int64_t i,
                                             const float* sw, const float* sp) {
  float* p = s.part + slab * 2 * part_columns(g.H);
  if (g.dw != nullptr) store8_f32(p, i, g.H, sw);
  if (g.dpost != nullptr) store8_f32(p + part_columns(g.H), i, g.H, sp);
}

struct RowRange {
  int64_t gate, first, end;
};
// The rows of the gates from walk * together on.
__device__ __forceinline__ RowRange rows_together(const ResidualNormBwdArgs& g, const Slabs& s, int64_t walk) {
  const int64_t gate_rows = g.rows / g.gates;
  RowRange r;
  r.gate = walk * s.together;
  r.first = r.gate * gate_rows;
  r.end = (r.gate + s.together) * gate_rows < g.rows ? (r.gate + s.together) * gate_rows : g.rows;
  return r;
}
__device__ __forceinline__ RowRange rows_of_slab(const ResidualNormBwdArgs& g, const Slabs& s, int64_t slab) {
  const int64_t gate_rows = g.rows / g.gates;
  RowRange r;
  r.gate = slab / s.per_gate;
  r.first = r.gate * gate_rows + (slab - r.gate * s.per_gate) * s.rows;
  r.end = r.first + s.rows < (r.gate + 1) * gate_rows ? r.first + s.rows : (r.gate + 1) * gate_rows;
  return r;
}

// T threads cover a row, eight columns each (TC: 16 or 64, and as many rows
// side by side as the workgroup holds; or 0: the whole workgroup).  They walk
// the rows of the workgroup's slab, which lies within one gate's rows, the next
// row's loads on their way during this row's sums.  FULL: the threads' columns
// are exactly the row.  16384x5120 BF16 with 8 gates and dr 203 us, 4.95 TB/s (the
// sums over slabs 6 more), bound by memory; 512x4096 12, by four rows one after
// another.  MANY: gates share a slab, and rows side by side are those of different
// gates, each T threads walking `together` gates of their own.
template <bool XF, bool HF, int TC, int NT, bool FULL, bool MANY>
__global__ __launch_bounds__(NT) void residual_norm_backward_kernel(ResidualNormBwdArgs g, Slabs sl) {
  __shared__ float red[32];
  __shared__ f4 cols[TC > 0 ? 4 * NT / 2 : 1];
  const int G = TC > 0 ? (int)blockDim.x / (TC > 0 ? TC : 1) : 1;   // rows side by side
  const int t = TC > 0 ? threadIdx.x % (TC > 0 ? TC : 1) : threadIdx.x;
  const int q = TC > 0 ? threadIdx.x / (TC > 0 ? TC : 1) : 0;
  const float inv_h = 1.0f / (float)g.H;
  const bool has_h = g.h != nullptr, post = g.post_w != nullptr, has_dr = g.dr != nullptr;
  const int64_t i = 8 * (int64_t)t;
  RowSums<TC> total(red);
  Raw8<HF> ndy, nz;
  Raw8<XF> nr, nd;
  Raw8<true> ng;   // the next gate, as it is stored
  float nrs = 0.0f, npost = 1.0f;
  auto load8_of = [&](auto& to, const void* p, int64_t r) {
    constexpr bool F = sizeof(to) == 32;
    const void* row = row_at<F>(p, r * g.H);
    to = TC == 16 || FULL ? load8<F, FULL>(row, i, g.H) : load8_ahead<F>(row, i, g.H);
  };
  auto load = [&](int64_t r) {
    load8_of(ndy, g.dy, r);
    load8_of(nr, g.r, r);
    if (has_h) load8_of(nz, g.h, r);
    if (has_dr) load8_of(nd, g.dr, r);
    nrs = g.rstd[r];
    if (post) npost = g.post_rstd[r];
  };
  auto load_gate = [&](int64_t gate) {
    const void* p = gate_at(g.gate, g.gate_f32, gate * g.H);
    if (g.gate_f32) ng = TC == 16 || FULL ? load8<true, FULL>(p, i, g.H) : load8_ahead<true>(p, i, g.H);
    else ng.q[0] = (TC == 16 || FULL ? load8<false, FULL>(p, i, g.H) : load8_ahead<false>(p, i, g.H)).q[0];
  };
  auto gate_values = [&](float* f) {
    if (g.gate_f32) {
      if (TC != 16 && !FULL) shift8<true>(ng, i, g.H);
      values8<true>(ng, f);
    } else {
      Raw8<false> b = {ng.q[0]};
      if (TC != 16 && !FULL) shift8<false>(b, i, g.H);
      values8<false>(b, f);
    }
  };
  const int64_t gate_rows = MANY ? g.rows / g.gates : 0;
  constexpr bool kSide = !MANY;   // the rows side by side are one gate's
  const int step = kSide ? G : 1;
  for (int64_t slab = blockIdx.x; slab < sl.count; slab += gridDim.x) {
  const RowRange rr = MANY ? rows_together(g, sl, slab * G + q) : rows_of_slab(g, sl, slab);
  int64_t r = kSide ? rr.first + q : rr.first, gate = rr.gate, gate_end = rr.first + gate_rows;
  if (r < rr.end) load(r);
  float w[8], f[8], pw[8], sw[8] = {}, sa[8] = {}, sp[8] = {};   // f: alpha gate pw, or the gate alone
  param8(g.w, g.w_f32, i, g.H, w);
  if constexpr (MANY) {
    param8(g.post_w, g.w_f32, i, g.H, pw);
    if (r < rr.end) {
      load_gate(gate);
      gate_values(f);
    }
  } else {
    factor8(g, rr.gate, i, f);
  }
  for (; r < rr.end; r += step) {
    float dy[8], n[8], z[8], d[8], e[8];
    if constexpr (TC != 16 && !FULL) {
      shift8<HF>(ndy, i, g.H);
      shift8<XF>(nr, i, g.H);
      if (has_h) shift8<HF>(nz, i, g.H);
      if (has_dr) shift8<XF>(nd, i, g.H);
    }
    values8<HF>(ndy, dy);
    values8<XF>(nr, n);
    if (has_h) values8<HF>(nz, z);
    if (has_dr) values8<XF>(nd, d);
    const float rs = nrs, post_rs = npost;
    if (r + step < rr.end) load(r + step);
    const bool last = MANY && r + 1 == gate_end;
    if (last && r + 1 < rr.end) load_gate(gate + 1);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      n[k] = __fmul_rn(n[k], rs);
      sw[k] = __builtin_fmaf(dy[k], n[k], sw[k]);
      dy[k] = __fmul_rn(dy[k], w[k]);
      e[k] = __fmul_rn(dy[k], n[k]);
    }
    const float c = __fmul_rn(total(sum8(e)), inv_h);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      n[k] = __fmul_rn(rs, __builtin_fmaf(-n[k], c, dy[k]));
      if (has_dr) n[k] = __fadd_rn(n[k], d[k]);   // dx
    }
    if (FULL || i < g.H) store8<XF>(g.dx, r * g.H, i, g.H, n);
    if (has_h) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (post) z[k] = __fmul_rn(z[k], post_rs);
        sa[k] = __builtin_fmaf(n[k], z[k], sa[k]);
        n[k] = __fmul_rn(n[k], MANY ? __fmul_rn(__fmul_rn(g.alpha, f[k]), pw[k]) : f[k]);   // p
        e[k] = __fmul_rn(n[k], z[k]);
      }
      if (post) {
        const float c2 = __fmul_rn(total(sum8(e)), inv_h);
#pragma unroll
        for (int k = 0; k < 8; ++k) n[k] = __fmul_rn(post_rs, __builtin_fmaf(-z[k], c2, n[k]));
      }
      if (FULL || i < g.H) store8<HF>(g.dh, r * g.H, i, g.H, n);
    }
    if (last) {
      put_gate(g, gate, i, f, pw, sa, sp);
      if (r + 1 < rr.end) gate_values(f);
      ++gate;
      gate_end += gate_rows;
    }
  }
  if constexpr (MANY) {
#pragma unroll
    for (int k = 0; k < 8; ++k) sa[k] = sp[k];
  }
  if constexpr (TC > 0) {
    // the rows side by side (a power of two) are added in a tree
    for (int h = G >> 1; h > 0; h >>= 1) {
      const int at = (q & (h - 1)) * TC + t, n4 = h * TC;
      if (q >= h && q < 2 * h) {
        cols[at] = (f4){sw[0], sw[1], sw[2], sw[3]};
        cols[n4 + at] = (f4){sw[4], sw[5], sw[6], sw[7]};
        cols[2 * n4 + at] = (f4){sa[0], sa[1], sa[2], sa[3]};
        cols[3 * n4 + at] = (f4){sa[4], sa[5], sa[6], sa[7]};
      }
      __syncthreads();
      if (q < h) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sw[k] = __fadd_rn(sw[k], cols[(k >> 2) * n4 + at][k & 3]);
          sa[k] = __fadd_rn(sa[k], cols[(2 + (k >> 2)) * n4 + at][k & 3]);
        }
      }
      __syncthreads();
    }
  }
  if (q == 0 && i < g.H) {
    if constexpr (MANY) put_together(g, sl, slab, i, sw, sa);
    else put_sums(g, sl, slab, rr.gate, i, sw, sa);
  }
  }
}

// Rows too long for that, in three launches: each row's sum(g n) / H into c;
// the column sums; dx and dh (which may lie over what is read).
struct LongRow {
  float rs, post_rs, c;
};
template <bool XF, bool HF>
__device__ __forceinline__ void long_row8(const ResidualNormBwdArgs& g, int64_t r, int64_t i, float rs, float* dy,
                                          float* n, float* gw) {
  values8<HF>(load8<HF>(row_at<HF>(g.dy, r * g.H), i, g.H), dy);
  values8<XF>(load8<XF>(row_at<XF>(g.r, r * g.H), i, g.H), n);
  param8(g.w, g.w_f32, i, g.H, gw);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    n[k] = __fmul_rn(n[k], rs);
    gw[k] = __fmul_rn(dy[k], gw[k]);
  }
}
template <bool XF, bool HF>
__device__ __forceinline__ void long_dx8(const ResidualNormBwdArgs& g, int64_t r, int64_t i, const LongRow& a,
                                         const float* n, const float* gw, float* dx, float* z) {
  float d[8];
  if (g.dr != nullptr) values8<XF>(load8<XF>(row_at<XF>(g.dr, r * g.H), i, g.H), d);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    dx[k] = __fmul_rn(a.rs, __builtin_fmaf(-n[k], a.c, gw[k]));
    if (g.dr != nullptr) dx[k] = __fadd_rn(dx[k], d[k]);
  }
  if (g.h == nullptr) return;
  values8<HF>(load8<HF>(row_at<HF>(g.h, r * g.H), i, g.H), z);
  if (g.post_w != nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] = __fmul_rn(z[k], a.post_rs);
  }
}
__device__ __forceinline__ LongRow long_row(const ResidualNormBwdArgs& g, const float* c, int64_t r) {
  return {g.rstd[r], g.post_w != nullptr ? g.post_rstd[r] : 1.0f, c == nullptr ? 0.0f : c[r]};
}

template <bool XF, bool HF>
__global__ __launch_bounds__(1024) void residual_norm_row_long_kernel(ResidualNormBwdArgs g, float* __restrict__ c) {
  __shared__ float red[32];
  const float inv_h = 1.0f / (float)g.H;
  RowSums<0> total(red);
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    LongSum s;
    for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
      float dy[8], n[8], gw[8];
      long_row8<XF, HF>(g, r, i, g.rstd[r], dy, n, gw);
#pragma unroll
      for (int k = 0; k < 8; ++k) n[k] = __fmul_rn(gw[k], n[k]);
      s.add(sum8(n));
    }
    const float v = __fmul_rn(total(s.s), inv_h);
    if (threadIdx.x == 0) c[r] = v;
  }
}

template <bool XF, bool HF, bool MANY>
__global__ __launch_bounds__(256) void residual_norm_columns_long_kernel(ResidualNormBwdArgs g, Slabs sl,
                                                                         const float* __restrict__ c) {
  const int64_t i = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (i >= g.H) return;
  const int64_t gate_rows = g.rows / g.gates;
  for (int64_t slab = blockIdx.y; slab < sl.count; slab += gridDim.y) {
    const RowRange rr = MANY ? rows_together(g, sl, slab) : rows_of_slab(g, sl, slab);
    int64_t gate = rr.gate, gate_end = rr.first + gate_rows;
    float sw[8] = {}, sa[8] = {}, sp[8] = {};
    for (int64_t r = rr.first; r < rr.end; ++r) {
      const LongRow a = long_row(g, c, r);
      float dy[8], n[8], gw[8], dx[8], z[8] = {};
      long_row8<XF, HF>(g, r, i, a.rs, dy, n, gw);
      long_dx8<XF, HF>(g, r, i, a, n, gw, dx, z);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sw[k] = __builtin_fmaf(dy[k], n[k], sw[k]);
        sa[k] = __builtin_fmaf(dx[k], z[k], sa[k]);
      }
      if (MANY && r + 1 == gate_end) {
        float gt[8], pw[8];
        param8(gate_at(g.gate, g.gate_f32, gate * g.H), g.gate_f32, i, g.H, gt);
        param8(g.post_w, g.w_f32, i, g.H, pw);
        put_gate(g, gate++, i, gt, pw, sa, sp);
        gate_end += gate_rows;
      }
    }
    if constexpr (MANY) put_together(g, sl, slab, i, sw, sp);
    else put_sums(g, sl, slab, rr.gate, i, sw, sa);
  }
}

template <bool XF, bool HF>
__global__ __launch_bounds__(1024) void residual_norm_dx_long_kernel(ResidualNormBwdArgs g,
                                                                     const float* __restrict__ c) {
  __shared__ float red[32];
  const float inv_h = 1.0f / (float)g.H;
  const bool has_h = g.h != nullptr, post = g.post_w != nullptr;
  const int64_t gate_rows = g.rows / g.gates;
  RowSums<0> total(red);
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    const LongRow a = long_row(g, c, r);
    auto row8 = [&](int64_t i, float* dx, float* z, float* p) {
      float dy[8], n[8], gw[8], f[8];
      long_row8<XF, HF>(g, r, i, a.rs, dy, n, gw);
      long_dx8<XF, HF>(g, r, i, a, n, gw, dx, z);
      if (!has_h) return;
      factor8(g, r / gate_rows, i, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) p[k] = __fmul_rn(dx[k], f[k]);
    };
    float c2 = 0.0f;
    if (has_h && post) {
      LongSum s;
      for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
        float dx[8], z[8], p[8];
        row8(i, dx, z, p);
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = i + k < g.H ? __fmul_rn(p[k], z[k]) : 0.0f;
        s.add(sum8(p));
      }
      c2 = __fmul_rn(total(s.s), inv_h);
    }
    for (int64_t i = 8 * (int64_t)threadIdx.x; i < g.H; i += 8 * 1024) {
      float dx[8], z[8], p[8];
      row8(i, dx, z, p);
      store8<XF>(g.dx, r * g.H, i, g.H, dx);
      if (!has_h) continue;
      if (post) {
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = __fmul_rn(a.post_rs, __builtin_fmaf(-z[k], c2, p[k]));
      }
      store8<HF>(g.dh, r * g.H, i, g.H, p);
    }
  }
}

// Columns n .. n + 3 of a gate (zeros past the row).
__device__ __forceinline__ void gate4(const ResidualNormBwdArgs& g, int64_t gate, int64_t n, float* f) {
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = n + k < g.H ? param1(g.gate, g.gate_f32, gate * g.H + n + k) : 0.0f;
}

// The results from part, in an order that depends on the sizes alone: y = 0
// dweight, sums over all slabs; 1 dpost_weight, sums over all slabs of the second
// plane times the slab's gate (a single one at the end; sums of gates together
// hold it); 2 + a (with each_gate) dgate a, its slabs' sums.  A workgroup takes
// 4 Q columns, four per thread, and L threads share a column's slabs, each a run of
// them (strided, they would take a gate anew for each slab: 16384x5120 with 8 gates
// 13.4 us, so 5.9).
template <int Q>
__global__ __launch_bounds__(256) void residual_norm_sums_kernel(ResidualNormBwdArgs g, Slabs sl, int each_gate) {
  constexpr int L = 256 / Q, C = 4 * Q, P = 256 / C, R = 4;
  static_assert(L / P == 4, "four rows of red per thread");
  __shared__ float red[L][C + 1], red2[P][C + 1];
  const int q = threadIdx.x % Q, s = threadIdx.x / Q;
  const int64_t n = (int64_t)blockIdx.x * C + 4 * q, per_gate = sl.per_gate;   // slabs are below 2^31
  for (int64_t y = blockIdx.y; y < 2 + (each_gate ? g.gates : 0); y += gridDim.y, __syncthreads()) {
    float* out = y == 0 ? g.dw : y == 1 ? g.dpost : (g.dgate == nullptr ? nullptr : g.dgate + (y - 2) * g.H);
    if (out == nullptr) continue;
    const int64_t first = y < 2 ? 0 : (y - 2) * per_gate, count = y < 2 ? sl.count : per_gate;
    const int64_t Hs = part_columns(g.H);
    const float* v = sl.part + (first * 2 + (y > 0)) * Hs;
    const bool by_gate = y == 1 && g.gate != nullptr && g.gates > 1 && !sl.together;
    float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // (columns past the row's end are read up to its padding, and not used)
    auto add = [&](int64_t p, int64_t end, float* u) {
      auto four = [&](int64_t p) {
        return n < Hs ? *reinterpret_cast<const f4*>(v + p * 2 * Hs + n) : (f4){0.0f, 0.0f, 0.0f, 0.0f};
      };
      for (; p + R <= end; p += R) {
        f4 x[R];
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = four(p + r);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int k = 0; k < 4; ++k) u[k] = __fadd_rn(u[k], x[r][k]);
      }
      for (; p < end; ++p) {
        const f4 x = four(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = __fadd_rn(u[k], x[k]);
      }
    };
    const int64_t share = (count + L - 1) / L, end = (s + 1) * share < count ? (s + 1) * share : count;
    if (by_gate) {
      int64_t p = s * share, gate = p < end ? (uint32_t)p / (uint32_t)per_gate : 0;
      for (; p < end; ++gate) {
        const int64_t to = (gate + 1) * per_gate < end ? (gate + 1) * per_gate : end;
        float u[4] = {0.0f, 0.0f, 0.0f, 0.0f}, f[4];
        gate4(g, gate, n, f);
        add(p, to, u);
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = __builtin_fmaf(u[k], f[k], t[k]);
        p = to;
      }
    } else {
      add(s * share, end, t);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) red[s][4 * q + k] = t[k];
    __syncthreads();
    {
      const int c = threadIdx.x % C, h = threadIdx.x / C;
      red2[h][c] = __fadd_rn(__fadd_rn(red[4 * h][c], red[4 * h + 1][c]), __fadd_rn(red[4 * h + 2][c], red[4 * h + 3][c]));
    }
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * C + threadIdx.x;
    if (threadIdx.x < C && c < g.H) {
      float u = red2[0][threadIdx.x];
#pragma unroll
      for (int h = 1; h < P; ++h) u = __fadd_rn(u, red2[h][threadIdx.x]);
      if (y > 0 && !sl.together) u = __fmul_rn(u, g.alpha);
      if (y == 1 && g.gate != nullptr && g.gates == 1) u = __fmul_rn(u, param1(g.gate, g.gate_f32, c));
      if (y > 1 && g.post_w != nullptr) u = __fmul_rn(u, param1(g.post_w, g.w_f32, c));
      out[c] = u;
    }
  }
}

// rows of up to this many elements go through residual_norm_backward_kernel
constexpr int64_t kBwdRegs = 1024 * 8;

// Threads of a workgroup, rows side by side in it, slabs for each gate: one
// workgroup of eight waves or more per CU, two of four to seven, three of fewer
// (16384x5120 BF16 210 us with 256 slabs, 239 with 384; 16384x2048 97, 92 with 512;
// 12000x1027 60 with 512, 55 with 768), of at least one, two or four rows one after
// another by the number of rows, since every slab's sums are written and read once
// more (256x4096 16.9 with four, 15.0 with two).  A few rows are one slab, whose
// sums need no second launch.  Of twice as many gates as there would be slabs
// (times the rows side by side), some share one:
// a gate for each row of 16384x5120 313 us (1018 with a slab each), of 200000x128
// 106 (6541).
struct BwdShape {
  int threads, side;
  int64_t per_gate, together, count;
};
BwdShape bwd_shape(int64_t rows, int64_t H, int64_t gates) {
  const int64_t units = (H + 7) / 8, gate_rows = rows / gates;
  BwdShape b{0, 1, 1, 0, 0};
  int64_t slabs;
  if (H > kBwdRegs) {
    b.threads = 1024;
    const int64_t room = 2048 / ((H + 2047) / 2048);
    slabs = room < 1 ? 1 : room < 256 ? room : 256;
  } else if (units <= 64) {
    const int tc = units <= 16 ? 16 : 64;
    b.threads = rows >= 256 * 4 * (512 / tc) ? 512 : 256;
    b.side = b.threads / tc;
  } else {
    b.threads = (int)((units + 63) / 64 * 64);
  }
  if (H <= kBwdRegs) slabs = b.threads >= 512 ? 256 : b.threads >= 256 ? 512 : 768;
  if (rows <= (H <= 4096 ? 4 : 2) * b.side && gates == 1) slabs = 1;
  if (slabs > 1 && gates >= 2 * slabs * b.side) {
    b.together = (gates + slabs * b.side - 1) / (slabs * b.side);
    const int64_t walks = (gates + b.together - 1) / b.together;
    b.count = (walks + b.side - 1) / b.side;
    return b;
  }
  b.per_gate = (slabs + gates - 1) / gates;
  const int64_t walk = H > kBwdRegs ? 4 : b.side > 1 || rows <= 64 ? 1 : rows <= 256 ? 2 : 4;
  const int64_t most = (gate_rows + walk * b.side - 1) / (walk * b.side);
  if (b.per_gate > most) b.per_gate = most;
  b.count = gates * b.per_gate;
  return b;
}

template <bool XF, bool HF, int TC, int NT>
hipError_t run_backward_kernel(const ResidualNormBwdArgs& g, const BwdShape& b, const Slabs& sl, hipStream_t stream) {
  const dim3 grid(row_grid(b.count, 1 << 20)), block(b.threads);
  if (b.together)
    hipLaunchKernelGGL((residual_norm_backward_kernel<XF, HF, TC, NT, false, true>), grid, block, 0, stream, g, sl);
  else if (TC == 0 && g.H == (int64_t)b.threads * 8)
    hipLaunchKernelGGL((residual_norm_backward_kernel<XF, HF, TC, NT, TC == 0, false>), grid, block, 0, stream, g, sl);
  else
    hipLaunchKernelGGL((residual_norm_backward_kernel<XF, HF, TC, NT, false, false>), grid, block, 0, stream, g, sl);
  return hipGetLastError();
}

template <bool XF, bool HF>
hipError_t run_backward(const ResidualNormBwdArgs& g, const BwdShape& b, const Slabs& sl, float* c,
                        hipStream_t stream) {
  if (g.H <= 128) return run_backward_kernel<XF, HF, 16, 512>(g, b, sl, stream);
  if (g.H <= 512) return run_backward_kernel<XF, HF, 64, 512>(g, b, sl, stream);
  if (b.threads <= 512) return run_backward_kernel<XF, HF, 0, 512>(g, b, sl, stream);
  if (b.threads <= 768) return run_backward_kernel<XF, HF, 0, 768>(g, b, sl, stream);
  if (g.H <= kBwdRegs) return run_backward_kernel<XF, HF, 0, 1024>(g, b, sl, stream);
  const unsigned rows = row_grid(g.rows, 1 << 20);
  hipLaunchKernelGGL((residual_norm_row_long_kernel<XF, HF>), dim3(rows), dim3(1024), 0, stream, g, c);
  if (g.dw != nullptr || g.dgate != nullptr || g.dpost != nullptr) {
    const dim3 grid((unsigned)((g.H + 2047) / 2048), row_grid(b.count, 65535));
    if (b.together)
      hipLaunchKernelGGL((residual_norm_columns_long_kernel<XF, HF, true>), grid, dim3(256), 0, stream, g, sl, c);
    else
      hipLaunchKernelGGL((residual_norm_columns_long_kernel<XF, HF, false>), grid, dim3(256), 0, stream, g, sl, c);
  }
  hipLaunchKernelGGL((residual_norm_dx_long_kernel<XF, HF>), dim3(rows), dim3(1024), 0, stream, g, c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_residual_norm(const ResidualNormArgs& g, hipStream_t stream) {
  if (g.x_f32) return g.h_f32 ? norm_of_types<true, true>(g, stream) : norm_of_types<true, false>(g, stream);
  return g.h_f32 ? norm_of_types<false, true>(g, stream) : norm_of_types<false, false>(g, stream);
}

int64_t residual_norm_backward_floats(int64_t rows, int64_t H, int64_t gates) {
  if (rows == 0 || H == 0) return 0;
  const int64_t slabs = bwd_shape(rows, H, gates).count;
  return (slabs > 1 ? slabs * 2 * part_columns(H) : 0) + (H > kBwdRegs ? rows : 0);
}

hipError_t launch_residual_norm_backward(const ResidualNormBwdArgs& g, float* ws, hipStream_t stream) {
  Slabs sl{0, 0, 0, 0, ws};   // no rows: sums of no slabs
  bool each_gate = true;
  if (g.rows > 0) {
    const BwdShape b = bwd_shape(g.rows, g.H, g.gates);
    const int64_t slabs = b.count, gate_rows = g.rows / g.gates;
    sl.per_gate = b.per_gate;
    sl.together = b.together;
    sl.count = slabs;
    sl.rows = (gate_rows + b.per_gate - 1) / b.per_gate;
    float* c = ws + (slabs > 1 ? slabs * 2 * part_columns(g.H) : 0);
    hipError_t e;
    if (g.x_f32) e = g.h_f32 ? run_backward<true, true>(g, b, sl, c, stream) : run_backward<true, false>(g, b, sl, c, stream);
    else e = g.h_f32 ? run_backward<false, true>(g, b, sl, c, stream) : run_backward<false, false>(g, b, sl, c, stream);
    if (e != hipSuccess || slabs == 1) return e;
    each_gate = b.per_gate > 1;
  }
  if (g.dw == nullptr && g.dpost == nullptr && (g.dgate == nullptr || !each_gate)) return hipSuccess;
  const unsigned planes = row_grid(2 + (each_gate ? g.gates : 0), 65535);
  auto run = [&](auto quads) {
    constexpr int Q = decltype(quads)::value;
    hipLaunchKernelGGL(residual_norm_sums_kernel<Q>, dim3((unsigned)((g.H + 4 * Q - 1) / (4 * Q)), planes), dim3(256), 0,
                       stream, g, sl, each_gate ? 1 : 0);
  };
  // (few columns in workgroups of 64 would leave most CUs idle)
  if (g.H * planes >= 32768) run(std::integral_constant<int, 16>{});
  else run(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

}  // namespace fp8mot
