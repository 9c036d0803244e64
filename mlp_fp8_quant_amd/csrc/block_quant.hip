// Quantization to FP8 with an FP32 scale for each block of 128 (declared in
// include/fp8mot.h as fp8_quant_block and silu_mul_2in_block).
//
//   s = amax of the block / 448,  q = e4m3(v / s)
//
// with v the elements of x, or g / (1 + exp(-g)) u.  A block is 128 columns of
// a row, 128 rows of a column (the codes then are those of the transposed
// tensor) or a 128 x 128 tile.  Rows of codes end in zeros up to a multiple of
// 16, so that the products take them whatever the size.  Bound by memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_scale.h"
#include "device_common.h"
#include "kernels.h"
#include "rowwise.h"

namespace fp8mot {

namespace {

using namespace rows;
using block::kBlock;

// silu(g) u in FP32: exp(-g) as 2^(hi + lo) with lo the part of g log2(e) that hi
// rounds off (2^lo = 1 + lo ln 2), g times the reciprocal after a Newton step.
// (silu_mul's plain exponential is off by |g| 2^-24, which an FP32 scale would
// show.)  Where the exponential is large or infinite, a division, as the formula
// has it.  With w = 2^-24: the hardware's exponential is within 2 w, 1 + lo ln 2 and
// their product round, d rounds (5 w so far), the refined reciprocal, its product
// with g and that with u round: 8 w and terms of second order, 9 w as the bound.
__device__ __forceinline__ float silu_mul_close(float g, float u) {
  const float c = __builtin_amdgcn_fmed3f(g, -128.0f, 128.0f);   // lo stays finite
  const float hi = __fmul_rn(c, -1.44269504f);
  const float lo = __builtin_fmaf(c, -1.92596303e-8f, __builtin_fmaf(c, -1.44269504f, -hi));
  const float p = __fmul_rn(__builtin_amdgcn_exp2f(hi), __builtin_fmaf(lo, 0.693147181f, 1.0f));
  const float d = __fadd_rn(1.0f, p), r = __builtin_amdgcn_rcpf(d);
  float s = __fmul_rn(g, __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r));
  if (__builtin_expect(!(d < 0x1p64f), 0)) s = g / d;
  return __fmul_rn(s, u);
}

// Blocks of 128 columns.  Sixteen lanes take a block, eight columns each, R
// blocks one after another with all their loads in flight.  FLAT: rows are
// whole blocks, so that block i lies at element 128 i of x and of q and no
// division finds its row.  16384x5120 BF16 53 us, 4.8 TB/s (the same input again and
// again, in part from the caches, 42); SwiGLU 4096x12288 49 to 56 us, 4.5 to 5.2 TB/s.
template <bool F32, bool SILU, bool FLAT, int R>
__global__ __launch_bounds__(256) void quant_rows_kernel(const void* __restrict__ x, const void* __restrict__ u,
                                                         uint8_t* __restrict__ q, float* __restrict__ scales,
                                                         int64_t blocks, int64_t K) {
  const int lane = threadIdx.x & 15;
  const int64_t per_row = (K + kBlock - 1) / kBlock, Kp = (K + 15) / 16 * 16;
  constexpr int ESZ = F32 ? 4 : 2;
  for (int64_t i0 = (int64_t)blockIdx.x * (16 * R); i0 < blocks; i0 += (int64_t)gridDim.x * (16 * R)) {
    Raw8<F32> a[R];
    Raw8<false> b[SILU ? R : 1];
    int64_t row[R], col[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t i = i0 + 16 * j + (threadIdx.x >> 4);
      if constexpr (FLAT) {
        row[j] = 0;
        col[j] = i * kBlock + 8 * lane;
      } else {
        row[j] = blocks <= INT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row;
        col[j] = (i - row[j] * per_row) * kBlock + 8 * lane;
      }
      if (i < blocks) {
        a[j] = load8<F32, FLAT>(static_cast<const uint8_t*>(x) + row[j] * K * ESZ, col[j], K);
        if constexpr (SILU) b[j] = load8<false, FLAT>(static_cast<const uint16_t*>(u) + row[j] * K, col[j], K);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t i = i0 + 16 * j + (threadIdx.x >> 4);
      if (i >= blocks) break;
      float f[8];
      values8<F32>(a[j], f);
      if constexpr (SILU) {
        float v[8];
        values8<false>(b[j], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = silu_mul_close(f[k], v[k]);
      }
      const float s = block::scale_of(block::max16(block::max8(f)));
      block::quotients<8>(f, s);
      if (FLAT || col[j] < Kp)
        *reinterpret_cast<u2a1*>(q + row[j] * Kp + col[j]) =
            (u2a1){e4m3_pack4(f[0], f[1], f[2], f[3]), e4m3_pack4(f[4], f[5], f[6], f[7])};
      if (lane == 0) scales[i] = s;
    }
  }
}

// 128 x 128 tiles of x with one scale each, a workgroup to a tile (25600x5120 BF16
// 72 to 75 us, 5.3 TB/s; transposed 79 to 81): thread t takes
// columns 8 (t % 16) .. + 7 of rows 8 (t / 16) .. + 7.  TRANS: the codes of the
// transposed tensor, turned through 16 KB of LDS (eight codes of one column, rows
// 8 r .. 8 r + 7, lie at chunk r ^ (column / 8) of the column's 128 bytes, which
// spreads both accesses over the banks).
template <bool F32, bool TRANS>
__global__ __launch_bounds__(256) void quant_tile_kernel(const void* __restrict__ x, uint8_t* __restrict__ q,
                                                         float* __restrict__ scales, int64_t M, int64_t K) {
  __shared__ int top[4];
  __shared__ __attribute__((aligned(16))) uint8_t turn[TRANS ? kBlock * kBlock : 16];
  const int cl = threadIdx.x & 15, rl = threadIdx.x >> 4;
  const int64_t kb = (K + kBlock - 1) / kBlock, mb = (M + kBlock - 1) / kBlock;
  for (int64_t tile = blockIdx.x; tile < kb * mb; tile += gridDim.x) {
    const int64_t tm = tile / kb, tk = tile - tm * kb;
    const int64_t m0 = tm * kBlock + 8 * rl, k0 = tk * kBlock + 8 * cl;
    Raw8<F32> raw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (m0 + j < M) raw[j] = load8<F32>(static_cast<const uint8_t*>(x) + (m0 + j) * K * (F32 ? 4 : 2), k0, K);
      else raw[j] = Raw8<F32>{};
    }
    float f[8][8];
    int m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      values8<F32>(raw[j], f[j]);
      m = max(m, block::max8(f[j]));
    }
    m = block::max16(m);
    m = max(max(__builtin_amdgcn_readlane(m, 0), __builtin_amdgcn_readlane(m, 16)),
            max(__builtin_amdgcn_readlane(m, 32), __builtin_amdgcn_readlane(m, 48)));
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
    const float s = block::scale_of(max(max(top[0], top[1]), max(top[2], top[3])));
#pragma unroll
    for (int j = 0; j < 8; ++j) block::quotients<8>(f[j], s);
    if (threadIdx.x == 0) scales[TRANS ? tk * mb + tm : tm * kb + tk] = s;
    if constexpr (!TRANS) {
      const int64_t Kp = (K + 15) / 16 * 16;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (m0 + j < M && k0 < Kp)
          *reinterpret_cast<u2a1*>(q + (m0 + j) * Kp + k0) =
              (u2a1){e4m3_pack4(f[j][0], f[j][1], f[j][2], f[j][3]), e4m3_pack4(f[j][4], f[j][5], f[j][6], f[j][7])};
    } else {
      uint2* const at = reinterpret_cast<uint2*>(turn);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        at[(8 * cl + c) * 16 + (rl ^ cl)] = make_uint2(e4m3_pack4(f[0][c], f[1][c], f[2][c], f[3][c]),
                                                       e4m3_pack4(f[4][c], f[5][c], f[6][c], f[7][c]));
      __syncthreads();
      const int64_t Mp = (M + 15) / 16 * 16, m1 = tm * kBlock + 8 * cl;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int c = 16 * p + rl;   // column of x, row of the codes
        const uint2 v = at[c * 16 + (cl ^ (c >> 3))];
        if (tk * kBlock + c < K && m1 < Mp)
          *reinterpret_cast<u2a1*>(q + (tk * kBlock + c) * Mp + m1) = (u2a1){v.x, v.y};
      }
    }
    __syncthreads();   // LDS is free for the next tile
  }
}

// Blocks of 128 rows of a column, as rows of the transposed tensor.  A workgroup
// takes 128 rows by 8 LC columns: thread t columns 8 (t % LC) .. + 7 of rows
// R (t / LC) .. + R - 1, R = LC / 2.  The columns' maxima are joined through LDS,
// where one thread per column forms the scale and its reciprocal (each thread for
// itself: 25600x5120 103 us, 89 so), and the codes are turned through it: R codes of a
// column, rows R r .. + R - 1, lie at chunk r ^ (TURN * (column / 8)) of its 128 bytes,
// which spreads the writes over the banks.
template <bool F32, int LC>
__global__ __launch_bounds__(256) void quant_columns_kernel(const void* __restrict__ x, uint8_t* __restrict__ q,
                                                            float* __restrict__ scales, int64_t M, int64_t K) {
  constexpr int C = 8 * LC, RL = 256 / LC, R = kBlock / RL, D = R / 4;   // D: dwords of codes per thread and column
  static_assert(R == 4 || R == 8, "");
  constexpr int TURN = LC == 16 ? 1 : 4;   // chunks by which neighbouring lanes' columns are turned
  __shared__ __attribute__((aligned(16))) uint32_t turn[C * kBlock / 4];
  __shared__ float scale[C], inverse[C];
  static_assert(RL * C <= C * kBlock / 4, "the maxima fit the codes' LDS");
  int (*const top)[C] = reinterpret_cast<int (*)[C]>(turn);   // until the scales are known
  const int cl = threadIdx.x % LC, rl = threadIdx.x / LC;
  const int64_t kb = (K + C - 1) / C, mb = (M + kBlock - 1) / kBlock;
  for (int64_t part = blockIdx.x; part < kb * mb; part += gridDim.x) {
    const int64_t tm = part / kb, k1 = (part - tm * kb) * C;
    const int64_t m0 = tm * kBlock + R * rl, k0 = k1 + 8 * cl;
    Raw8<F32> raw[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (m0 + j < M) raw[j] = load8<F32>(static_cast<const uint8_t*>(x) + (m0 + j) * K * (F32 ? 4 : 2), k0, K);
      else raw[j] = Raw8<F32>{};
    }
    float f[R][8];
#pragma unroll
    for (int j = 0; j < R; ++j) values8<F32>(raw[j], f[j]);
    int m[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      m[c] = block::magnitude(f[0][c]);
#pragma unroll
      for (int j = 1; j < R; ++j) m[c] = max(m[c], block::magnitude(f[j][c]));
    }
    *reinterpret_cast<int4*>(&top[rl][8 * cl]) = make_int4(m[0], m[1], m[2], m[3]);
    *reinterpret_cast<int4*>(&top[rl][8 * cl + 4]) = make_int4(m[4], m[5], m[6], m[7]);
    __syncthreads();
    if (threadIdx.x < C) {
      const int c = threadIdx.x;
      int t = top[0][c];
#pragma unroll
      for (int r = 1; r < RL; ++r) t = max(t, top[r][c]);
      const float s = block::scale_of(t);
      scale[c] = s;
      inverse[c] = 1.0f / s;
      if (k1 + c < K) scales[(k1 + c) * mb + tm] = s;
    }
    __syncthreads();
    const int64_t Mp = (M + 15) / 16 * 16;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float s = scale[8 * cl + c], r = inverse[8 * cl + c];
      float v[R];
#pragma unroll
      for (int j = 0; j < R; ++j) v[j] = f[j][c];
      block::quotients<R>(v, s, r);
#pragma unroll
      for (int d = 0; d < D; ++d)
        turn[(8 * cl + c) * 32 + (rl ^ (cl * TURN)) * D + d] =
            e4m3_pack4(v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]);
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < C / 8; ++p) {
      const int c = 8 * p + (threadIdx.x >> 5), w = threadIdx.x & 31;   // column of x, dword of its codes
      const uint32_t v = turn[c * 32 + ((w / D) ^ ((c >> 3) * TURN)) * D + w % D];
      if (k1 + c < K && tm * kBlock + 4 * w < Mp)
        *reinterpret_cast<uint32_t*>(q + (k1 + c) * Mp + tm * kBlock + 4 * w) = v;
    }
    __syncthreads();   // LDS is free for the next part
  }
}

template <bool F32, bool SILU>
hipError_t run_rows(const void* x, const void* u, uint8_t* q, float* scales, int64_t M, int64_t K,
                    hipStream_t stream) {
  constexpr int R = F32 || SILU ? 2 : 4;
  const int64_t blocks = M * ((K + kBlock - 1) / kBlock), groups = (blocks + 16 * R - 1) / (16 * R);
  const dim3 grid((unsigned)(groups < (1 << 22) ? groups : (1 << 22)));
  if (K % kBlock == 0)
    hipLaunchKernelGGL((quant_rows_kernel<F32, SILU, true, R>), grid, dim3(256), 0, stream, x, u, q, scales, blocks, K);
  else
    hipLaunchKernelGGL((quant_rows_kernel<F32, SILU, false, R>), grid, dim3(256), 0, stream, x, u, q, scales, blocks,
                       K);
  return hipGetLastError();
}

template <bool F32>
hipError_t run_quant(const void* x, uint8_t* q, float* scales, int64_t M, int64_t K, int tile, int transpose,
                     hipStream_t stream) {
  if (!tile && !transpose) return run_rows<F32, false>(x, nullptr, q, scales, M, K, stream);
  const int64_t mb = (M + kBlock - 1) / kBlock, squares = mb * ((K + kBlock - 1) / kBlock);
  auto grid = [](int64_t n) { return dim3((unsigned)(n < (1 << 20) ? n : (1 << 20))); };
  if (tile) {
    if (transpose)
      hipLaunchKernelGGL((quant_tile_kernel<F32, true>), grid(squares), dim3(256), 0, stream, x, q, scales, M, K);
    else
      hipLaunchKernelGGL((quant_tile_kernel<F32, false>), grid(squares), dim3(256), 0, stream, x, q, scales, M, K);
  } else if (squares <= 1024) {
    // 64 columns: more workgroups (1531x2053 8.4 us, 11.4 with 128; 25600x5120 96, 89)
    hipLaunchKernelGGL((quant_columns_kernel<F32, 8>), grid(mb * ((K + 63) / 64)), dim3(256), 0, stream, x, q, scales, M,
                       K);
  } else {
    hipLaunchKernelGGL((quant_columns_kernel<F32, 16>), grid(squares), dim3(256), 0, stream, x, q, scales, M, K);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_block(const void* x, int x_f32, uint8_t* q, float* scales, int64_t M, int64_t K, int tile,
                              int transpose, hipStream_t stream) {
  return x_f32 ? run_quant<true>(x, q, scales, M, K, tile, transpose, stream)
               : run_quant<false>(x, q, scales, M, K, tile, transpose, stream);
}

hipError_t launch_silu_mul_block(const uint16_t* g, const uint16_t* u, uint8_t* q, float* scales, int64_t rows,
                                 int64_t K, hipStream_t stream) {
  return run_rows<false, true>(g, u, q, scales, rows, K, stream);
}

}  // namespace fp8mot
