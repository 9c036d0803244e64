// FP8 Linear whose operands have a scale for each block of 128 of K, with bias,
// activation and residual in its epilogue (declared in include/fp8mot.h as
// fp8_linear_block).
//
//   P[m,n,b] = sum_{k in block b} dec(qx[m,k]) dec(qw[n,k])
//   acc[m,n] = sum_b fp32(sx[m,b] sw[n',b]) P[m,n,b]        (one FMA a block)
//   n' = n where W has a scale for each row, n / 128 where for each 128 x 128
//
// and from there as fp8_linear_act.  The codes are decoded exactly to F16 and
// multiplied on the F16 matrix cores, all sums in FP32.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "gemm_parts.h"
#include "kernels.h"
#include "linear_block_plan.h"
#include "linear_epilogue.h"

namespace fp8mot {

namespace {

using tile::decode8;
using tile::f16x8;
using tile::v4f;
using tile::v4i;

// Products of few rows, laid out as fp8_linear_act's: a workgroup computes
// 16 * MB rows of X against 16 * NB rows of W, its NW waves take the 128-K
// stages in turn, each through a ring of two stages of its own in LDS, and the
// waves' sums are added in wave order.  W is the first operand of the 16x16x32
// F16 MFMAs: accumulator register v of lane l is column n = 4 * (l / 16) + v of
// row m = l % 16.  A stage is one block: its products are summed from zero and
// added to the lane's sums by one FMA with the row's scale times the column's.
// A stage brings its scales along: lane i of two copies of four bytes per lane
// those of row i of X and of row i of W (where W's are per tile, the same for
// its 128 rows).  Bound by the weight's bytes and, for few of them, by the launch
// and the first fetch: 1x4096x4096 5.5 us a call, 13x12288x4096 10.5 (4.8 TB/s); 64
// x 64 tiles by the waits of one wave per SIMD, 256x4096x4096 15.6 (0.55 PFLOP/s).
constexpr int kStageK = 128;

template <int MB, int NB, int NW>
__global__ __launch_bounds__(NW * 64, 1) void linear_block_rows_kernel(LinearActArgs g) {
  static_assert(MB <= 4 && NB <= 4, "a copy brings 64 scales");
  constexpr int RB = MB + NB, COPIES = 2 * RB, CODES = RB * 2048, STAGE = CODES + 512;
  constexpr int D = 2;   // stages of a wave's ring
  static_assert(NW * D * STAGE <= 160 * 1024 && NW * MB * NB * 1024 <= NW * D * STAGE, "LDS");
  static_assert(D * (COPIES + 2) < 64, "wait_copies");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * D * STAGE];
  // Epilogue: a wave takes G 16-row blocks of the same 16 columns at once.
  constexpr int PER = MB * NB / NW;
  constexpr int G = PER < 1 ? 1 : (PER < MB ? PER : MB), CHUNKS = MB * NB / G, ROUNDS = (CHUNKS + NW - 1) / NW;
  static_assert(MB % G == 0, "chunks of rows");
  static_assert(ROUNDS <= 2, "operands of the first round and the next");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l15 = lane & 15, kq = lane >> 4;
  const int K = (int)g.K;
  const int stages = (K + kStageK - 1) / kStageK;
  // each XCD takes a run of the tiles in column-major order (see linear_act.hip)
  int tile_n = (int)blockIdx.x, tile_m = (int)blockIdx.y;
  if (MB > 1 && (NB < 4 || (gridDim.x & 7) != 0)) {
    const int down = (int)gridDim.y, tiles = (int)gridDim.x * down, id = tile_m * (int)gridDim.x + tile_n;
    const int tile = (id & 7) * (tiles >> 3) + min(id & 7, tiles & 7) + (id >> 3);
    // tile / down in floats: the quotient, below 2^22, is off by one at most
    tile_n = (int)((float)tile * __builtin_amdgcn_rcpf((float)down));
    const int rest = tile - tile_n * down;
    tile_n = __builtin_amdgcn_readfirstlane(tile_n + (rest >= down ? 1 : 0) - (rest < 0 ? 1 : 0));
    tile_m = tile - tile_n * down;
  }
  const int64_t n0 = (int64_t)tile_n * (16 * NB), m0 = (int64_t)tile_m * (16 * MB);
  uint8_t* const ring = smem + wave * (D * STAGE);

  const bool vec = (g.N & 3) == 0;
  const linear::Epilogue epi = linear::open_outputs(g, m0);
  LinearActArgs ge = g;
  ge.row_scales = 0;   // the sums are scaled already
  linear::Operands<G> op, op2;
  linear::Columns col, col2;
  // chunk q: rows row_of(q), + 16, .. from m0, columns col_of(q) .. + 3
  auto row_of = [&](int q) { return 16 * G * (q / NB) + l15; };
  auto col_of = [&](int q) { return (int)n0 + 16 * (q % NB) + 4 * kq; };
  auto operands = [&](int q, linear::Operands<G>& op, linear::Columns& col) {
    const int row = row_of(q), n = col_of(q), nv = (int)g.N - n;
    if (vec) {
      linear::load_operands<G, true>(ge, epi, m0, row, 16, n, nv, &op);
      col = linear::load_columns<true>(ge, n, nv);
    } else {
      linear::load_operands<G, false>(ge, epi, m0, row, 16, n, nv, &op);
      col = linear::load_columns<false>(ge, n, nv);
    }
  };
  if (wave < CHUNKS) operands(wave, op, col);   // they arrive during the product

  // copy q of a stage fills LDS rows 8q .. 8q + 7 (W's 16 NB rows, then X's):
  // lane l brings row 8q + l/8, physical chunk l % 8
  const v4i wr = tile::make_rsrc_words(g.qw + n0 * K, (g.N - n0) * K);
  const v4i xr = tile::make_rsrc_words(g.qx + m0 * K, (g.M - m0) * K);
  int off[COPIES];
#pragma unroll
  for (int q = 0; q < COPIES; ++q) {
    const int r = 8 * q + (lane >> 3), rr = q < 2 * NB ? r : r - 16 * NB;
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    off[q] = rr < (q < 2 * NB ? g.N - n0 : g.M - m0) ? rr * K + 16 * c : tile::kOOB;
  }
  // scales: rows past M or N read as zeros
  const int64_t w0 = g.row_scales ? n0 : n0 / kStageK, w_rows = g.row_scales ? g.N : (g.N + kStageK - 1) / kStageK;
  const v4i xs = tile::make_rsrc_words(g.sx + m0 * stages, (g.M - m0) * stages * 4);
  const v4i ws = tile::make_rsrc_words(g.sw + w0 * stages, (w_rows - w0) * stages * 4);
  const int xs_off = lane < 16 * MB && lane < g.M - m0 ? lane * stages * 4 : tile::kOOB;
  const int w_row = g.row_scales ? lane : (int)((n0 + lane) / kStageK - w0);
  const int ws_off = lane < 16 * NB && lane < g.N - n0 ? w_row * stages * 4 : tile::kOOB;
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((tile::lds_ptr_t)ring);
  auto issue = [&](int s, int slot) {
    const int k0 = s * kStageK;
    const uint32_t dst = lds0 + slot * STAGE;
    if (k0 + kStageK <= K) {
#pragma unroll
      for (int q = 0; q < COPIES; ++q) tile::copy_to_lds(q < 2 * NB ? wr : xr, dst + q * 1024, off[q], k0);
    } else {   // K ends inside the stage
#pragma unroll
      for (int q = 0; q < COPIES; ++q) {
        const int c = (lane & 7) ^ (((8 * q + (lane >> 3)) >> 1) & 7);
        tile::copy_to_lds(q < 2 * NB ? wr : xr, dst + q * 1024,
                          k0 + 16 * c < K && off[q] != tile::kOOB ? off[q] + k0 : tile::kOOB, 0);
      }
    }
    tile::copy4_to_lds(xs, dst + CODES, xs_off, s * 4);
    tile::copy4_to_lds(ws, dst + CODES + 256, ws_off, s * 4);
  };
  // at most one stage's copies of this wave in flight, or none (vmcnt alone:
  // gfx9 encoding)
  auto wait_copies = [&](bool one) {
    constexpr int n = COPIES + 2;
    if (one) __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | ((n >> 4) << 14));
    else __builtin_amdgcn_s_waitcnt(0x0F70);
  };
  const int mine = wave < stages ? (stages - wave + NW - 1) / NW : 0;   // stages wave, wave + NW, ..
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i < mine) issue(wave + i * NW, i);

  v4f acc[MB][NB];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int c = 0; c < NB; ++c) acc[b][c] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  const int rd0 = l15 * 128 + ((kq ^ (l15 >> 1)) << 4), rd1 = l15 * 128 + (((kq + 4) ^ (l15 >> 1)) << 4);
  int slot = 0;
  for (int i = 0; i < mine; ++i) {
    wait_copies(i + 1 < mine);
    asm volatile("" ::: "memory");
    const uint8_t* st = ring + slot * STAGE;
    v4i f[RB][2];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      f[r][0] = *reinterpret_cast<const v4i*>(st + r * 2048 + rd0);
      f[r][1] = *reinterpret_cast<const v4i*>(st + r * 2048 + rd1);
    }
    float sx[MB];
    v4f sw[NB];
#pragma unroll
    for (int b = 0; b < MB; ++b) sx[b] = reinterpret_cast<const float*>(st + CODES)[16 * b + l15];
#pragma unroll
    for (int c = 0; c < NB; ++c) sw[c] = *reinterpret_cast<const v4f*>(st + CODES + 256 + 64 * c + 16 * kq);
    if (i + D < mine) {
      // the stage has been read before it is refilled
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
      asm volatile("" ::: "memory");
      issue(wave + (i + D) * NW, slot);
    }
    slot = slot + 1 == D ? 0 : slot + 1;
    v4f p[MB][NB];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < NB; ++c) p[b][c] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f16x8 w0[NB], w1[NB];
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        w0[c] = decode8(f[c][h][0], f[c][h][1]);
        w1[c] = decode8(f[c][h][2], f[c][h][3]);
      }
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const f16x8 x0 = decode8(f[NB + b][h][0], f[NB + b][h][1]), x1 = decode8(f[NB + b][h][2], f[NB + b][h][3]);
#pragma unroll
        for (int c = 0; c < NB; ++c) p[b][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0[c], x0, p[b][c], 0, 0, 0);
#pragma unroll
        for (int c = 0; c < NB; ++c) p[b][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1[c], x1, p[b][c], 0, 0, 0);
      }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[b][c][v] = __builtin_fmaf(p[b][c][v], __fmul_rn(sx[b], sw[c][v]), acc[b][c][v]);
  }

  // join: the ring is free once every wave is here (its copies have landed)
  __syncthreads();
  v4f* red = reinterpret_cast<v4f*>(smem);
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int c = 0; c < NB; ++c) red[(wave * (MB * NB) + b * NB + c) * 64 + lane] = acc[b][c];
  if (wave + NW < CHUNKS) operands(wave + NW, op2, col2);
  __syncthreads();
#pragma unroll 1
  for (int q = wave; q < CHUNKS; q += NW) {
    float z[G][4];
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int b = ((q / NB) * G + k) * NB + q % NB;
      v4f s = red[b * 64 + lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        const v4f o = red[(w * (MB * NB) + b) * 64 + lane];
#pragma unroll
        for (int v = 0; v < 4; ++v) s[v] = __fadd_rn(s[v], o[v]);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) z[k][v] = s[v];
    }
    const int row = row_of(q), n = col_of(q), nv = (int)g.N - n;
    auto next = [&] {
      op = op2;
      col = col2;
    };
    if (vec) linear::finish<G, true>(ge, epi, col, row, 16, n, nv, op, z, next);
    else linear::finish<G, false>(ge, epi, col, row, 16, n, nv, op, z, next);
  }
}

template <int MB, int NB, int NW>
hipError_t launch_rows(const LinearActArgs& g, hipStream_t stream) {
  hipLaunchKernelGGL((linear_block_rows_kernel<MB, NB, NW>),
                     dim3((unsigned)((g.N + 16 * NB - 1) / (16 * NB)), (unsigned)((g.M + 16 * MB - 1) / (16 * MB))),
                     dim3(NW * 64), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_block(const LinearActArgs& g, int num_cus, hipStream_t stream) {
  const int tile = linear_block_plan(g.M, g.N, g.K);
  switch (tile) {
    case kRows1x1: return launch_rows<1, 1, 16>(g, stream);
    case kRows1x2: return launch_rows<1, 2, 8>(g, stream);
    case kRows1x4: return launch_rows<1, 4, 4>(g, stream);
    case kRows2x1: return launch_rows<2, 1, 8>(g, stream);
    case kRows2x2: return launch_rows<2, 2, 8>(g, stream);
    case kRows2x4: return launch_rows<2, 4, 4>(g, stream);
    case kRows4x2: return launch_rows<4, 2, 4>(g, stream);
    case kRows4x4: return launch_rows<4, 4, 4>(g, stream);
    case kRows4x4Pair: return launch_rows<4, 4, 2>(g, stream);
    default: return launch_linear_block_tile(g, tile, num_cus, stream);
  }
}

}  // namespace fp8mot
