// FP8 Linear with bias, activation and residual in its epilogue, and that
// epilogue's backward pass (declared in include/fp8mot.h as fp8_linear_act
// and fp8_linear_act_backward).
//
//   acc[m,n] = sum_k dec(qx[m,k]) dec(qw[n,k])          (FP32 accumulation)
//   z        = fma(acc, alpha, bias[n]),     alpha = fp32(s_x s_w)
//   y        = act(z) + residual[m,n]  -> BF16, E4M3(y / s_y) or FP32
//   dz       = dy act'(z),  dbias[n] = sum_m dz[m,n]
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "act.h"
#include "device_common.h"
#include "gemm_parts.h"
#include "kernels.h"
#include "linear_epilogue.h"
#include "rowwise.h"

namespace fp8mot {

namespace {

using tile::decode8;
using tile::f16x8;
using tile::v4f;
using tile::v4i;

// Products of few rows.  A workgroup computes 16 * MB rows of X against 16 * NB
// rows of W; its NW waves take the 128-K stages of K in turn, each through a
// ring of two stages of its own in LDS that the buffer unit fills (rows of 128
// codes, swizzled as in the tiled kernel), so no wave waits for another until
// their sums are added in wave order at the end.  A lane reads 16-byte chunks
// lane / 16 and lane / 16 + 4 of row lane % 16 of each 16-row block and feeds
// bytes 0..7 of a chunk to one 16x16x32 F16 MFMA and bytes 8..15 to the next,
// W as the first operand: accumulator register v of lane l is then column
// n = 4 * (l / 16) + v of row m = l % 16.  Rows past M or N and K past its end
// get offsets past the buffers and land as zeros.
//
// Bound by the bytes of W from memory where rows are few (13x12288x4096 to
// E4M3 with GELU 10.6 us, 4.7 TB/s), then by what a CU takes in of both
// operands from L2, about 50 bytes a clock with copies of whole 128-byte row
// pieces (fragments of 64 bytes straight to registers, half of that: 64x4096
// x4096 16.5 us, 7.9 so), and with two workgroups per CU by decodes and MFMAs
// one after another (512x4096x12288 52 to 56 us, 0.92 to 0.99 PFLOP/s).
constexpr int kStageK = 128;

template <int MB, int NB, int NW>
__global__ __launch_bounds__(NW * 64, 1) void linear_rows_kernel(LinearActArgs g) {
  constexpr int RB = MB + NB, COPIES = 2 * RB, STAGE = RB * 2048;
  constexpr int D = 2;   // stages of a wave's ring
  static_assert(NW * D * STAGE <= 160 * 1024 && NW * MB * NB * 1024 <= NW * D * STAGE, "LDS");
  static_assert(D * COPIES < 64, "wait_copies");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NW * D * STAGE];
  // Epilogue: a wave takes G 16-row blocks of the same 16 columns at once
  // (their operands in flight together), ROUNDS times; one copy of the code,
  // since every launch fetches it cold.  The first round's operands are read
  // during the product, the second's during the join.
  constexpr int PER = MB * NB / NW;
  constexpr int G = PER < 1 ? 1 : (PER < MB ? PER : MB), CHUNKS = MB * NB / G, ROUNDS = (CHUNKS + NW - 1) / NW;
  static_assert(MB % G == 0, "chunks of rows");
  static_assert(ROUNDS <= 2, "operands of the first round and the next");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l15 = lane & 15, kq = lane >> 4;
  const int K = (int)g.K;
  // Workgroups go to the eight XCDs in turn.  Unless that gives an XCD whole
  // columns of tiles at least a cache line of outputs wide, or there is one row
  // of tiles, each XCD takes a run of the tiles in column-major order: its L2
  // then reads few of W's rows and joins the outputs of neighbouring tiles
  // (777x2053x2064 20.0 -> 17.8 us, 128x10000x1024 13.5 -> 12.1, 32x4096x4096
  // 6.7 -> 6.2; but 256x4096x4096 14.7 -> 15.1, one token 4096x4096 5.6 -> 6.1).
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
  const linear::Epilogue epi = linear::open_epilogue(g, m0);
  linear::Operands<G> op, op2;
  linear::Columns col, col2;
  // chunk q: rows row_of(q), + 16, .. from m0, columns col_of(q) .. + 3
  auto row_of = [&](int q) { return 16 * G * (q / NB) + l15; };
  auto col_of = [&](int q) { return (int)n0 + 16 * (q % NB) + 4 * kq; };
  auto operands = [&](int q, linear::Operands<G>& op, linear::Columns& col) {
    const int row = row_of(q), n = col_of(q), nv = (int)g.N - n;
    if (vec) {
      linear::load_operands<G, true>(g, epi, m0, row, 16, n, nv, &op);
      col = linear::load_columns<true>(g, n, nv);
    } else {
      linear::load_operands<G, false>(g, epi, m0, row, 16, n, nv, &op);
      col = linear::load_columns<false>(g, n, nv);
    }
  };
  if (wave < CHUNKS) operands(wave, op, col);   // they arrive during the product

  // copy q of a stage fills LDS rows 8q .. 8q + 7 (W's 16 NB rows, then X's):
  // lane l brings row 8q + l/8, physical chunk l % 8
  const tile::v4i wr = tile::make_rsrc_words(g.qw + n0 * K, (g.N - n0) * K);
  const tile::v4i xr = tile::make_rsrc_words(g.qx + m0 * K, (g.M - m0) * K);
  int off[COPIES];
#pragma unroll
  for (int q = 0; q < COPIES; ++q) {
    const int r = 8 * q + (lane >> 3), rr = q < 2 * NB ? r : r - 16 * NB;
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    off[q] = rr < (q < 2 * NB ? g.N - n0 : g.M - m0) ? rr * K + 16 * c : tile::kOOB;
  }
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
  };
  // at most one stage's copies of this wave in flight, or none (vmcnt alone:
  // gfx9 encoding)
  auto wait_copies = [&](bool one) {
    if (one) __builtin_amdgcn_s_waitcnt(0x0F70 | (COPIES & 15) | ((COPIES >> 4) << 14));
    else __builtin_amdgcn_s_waitcnt(0x0F70);
  };
  const int stages = (K + kStageK - 1) / kStageK;
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
    if (i + D < mine) {
      // the fragments have been read before the stage is refilled
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
      asm volatile("" ::: "memory");
      issue(wave + (i + D) * NW, slot);
    }
    slot = slot + 1 == D ? 0 : slot + 1;
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
        for (int c = 0; c < NB; ++c) acc[b][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0[c], x0, acc[b][c], 0, 0, 0);
#pragma unroll
        for (int c = 0; c < NB; ++c) acc[b][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1[c], x1, acc[b][c], 0, 0, 0);
      }
    }
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
    if (vec) linear::finish<G, true>(g, epi, col, row, 16, n, nv, op, z, next);
    else linear::finish<G, false>(g, epi, col, row, 16, n, nv, op, z, next);
  }
}

template <int MB, int NB, int NW>
hipError_t launch_rows(const LinearActArgs& g, hipStream_t stream) {
  hipLaunchKernelGGL((linear_rows_kernel<MB, NB, NW>),
                     dim3((unsigned)((g.N + 16 * NB - 1) / (16 * NB)), (unsigned)((g.M + 16 * MB - 1) / (16 * MB))),
                     dim3(NW * 64), 0, stream, g);
  return hipGetLastError();
}

// Joins the splits of K: sums part [splits, M, N] in split order and runs the
// epilogue, four consecutive columns per thread.  A workgroup's groups lie
// within kJoinRows rows of each other, which the epilogue addresses from the
// first of them.
constexpr int kJoinRows = 16;

template <bool VEC>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearActArgs g, const float* __restrict__ part,
                                                          int splits) {
  const int N = (int)g.N, per_row = (N + 3) / 4;
  const int64_t m0 = (int64_t)blockIdx.x * kJoinRows;
  const int rows = g.M - m0 < kJoinRows ? (int)(g.M - m0) : kJoinRows;
  const linear::Epilogue e = linear::open_epilogue(g, m0);
  for (int i = (int)blockIdx.y * 256 + (int)threadIdx.x; i < rows * per_row; i += (int)gridDim.y * 256) {
    const int row = i / per_row, n = (i - row * per_row) * 4, nv = N - n;
    linear::Operands<1> op;
    linear::load_operands<1, VEC>(g, e, m0, row, 1, n, nv, &op);
    const linear::Columns col = linear::load_columns<VEC>(g, n, nv);
    float z[1][4] = {{0.0f, 0.0f, 0.0f, 0.0f}}, o[4];
    for (int p = 0; p < splits; ++p) {
      linear::values4(linear::load4<VEC>(linear::rows_of(part + p * g.M * N, m0, g.M, N, 4), 1, row * N + n, nv), 1, o);
#pragma unroll
      for (int c = 0; c < 4; ++c) z[0][c] = p == 0 ? o[c] : __fadd_rn(z[0][c], o[c]);
    }
    linear::finish<1, VEC>(g, e, col, row, 1, n, nv, op, z, [] {});
  }
}

// dz = dy act'(pre) for a slab of rows and 8 LP columns, with the columns'
// sums over the slab (of dz before its rounding to BF16) into part[slab, n].
// Bound by memory.  LP threads side by side hold eight consecutive columns
// each, NT / LP of them share the slab's rows (narrow tensors thus keep all
// lanes busy) and are added through LDS in order; R rows are in flight per
// thread.
template <int LP, int NT>
__global__ __launch_bounds__(NT) void act_backward_kernel(
    const uint16_t* dy, const uint16_t* pre, int act, uint16_t* dz, float* __restrict__ part, int64_t M, int64_t N,
    int64_t slab_rows) {
  constexpr int RL = NT / LP, R = 4;
  __shared__ float red[RL][LP * 8];
  const int cl = threadIdx.x % LP, rl = threadIdx.x / LP;
  const int64_t n = ((int64_t)blockIdx.x * LP + cl) * 8;
  const int64_t r0 = (int64_t)blockIdx.y * slab_rows;
  const int64_t r1 = r0 + slab_rows < M ? r0 + slab_rows : M;
  float s[8] = {};
  if (n < N) {
    for (int64_t r = r0 + rl; r < r1; r += RL * R) {
      rows::Raw8<false> d[R], z[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (r + k * RL < r1) {
          d[k] = rows::load8<false>(dy + (r + k * RL) * N, n, N);
          if (act != kActNone) z[k] = rows::load8<false>(pre + (r + k * RL) * N, n, N);
        }
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (r + k * RL < r1) {
          float v[8], a[8];
          rows::values8<false>(d[k], v);
          if (act != kActNone) {
            rows::values8<false>(z[k], a);
            slope_all<8>(a, act);
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = __fmul_rn(v[c], a[c]);
          }
          if (dz != nullptr) rows::store8_bf16(dz + (r + k * RL) * N, n, N, v);
#pragma unroll
          for (int c = 0; c < 8; ++c) s[c] = __fadd_rn(s[c], v[c]);
        }
      }
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int c = 0; c < 8; ++c) red[rl][cl * 8 + c] = s[c];
  __syncthreads();
  for (int c = threadIdx.x; c < LP * 8; c += NT) {
    float v = red[0][c];
#pragma unroll
    for (int k = 1; k < RL; ++k) v = __fadd_rn(v, red[k][c]);
    const int64_t at = (int64_t)blockIdx.x * (LP * 8) + c;
    if (at < N) part[(int64_t)blockIdx.y * N + at] = v;
  }
}

// How the backward pass of the epilogue covers [M, N].  Up to kActOneSlab rows
// a workgroup of 1024 threads takes 32 columns of all of them and its sums are
// the results: a second launch costs more than the rows (64x4096 4.6 us,
// 5.1 in slabs; but 777x2053 13.0, 8.8 in slabs).  Otherwise 256 threads, up to
// 64 side by side, about eight workgroups per CU, and at least a row per thread
// or (wide rows, whose partial sums cost more) two: 1024x4096 10.3 us, 11.9
// with one, 10.5 with four; 2000x100 5.7 with one, 6.4 with two.
constexpr int64_t kActOneSlab = 128;
struct ActShape {
  int lanes;
  int64_t slabs;
};
ActShape act_shape(int64_t M, int64_t N) {
  if (M <= kActOneSlab) return {4, 1};
  const int lanes = N <= 64 ? 8 : N <= 128 ? 16 : N <= 256 ? 32 : 64;
  const int64_t across = (N + lanes * 8 - 1) / (lanes * 8), side = 256 / lanes;
  int64_t slabs = (256 * 8 + across - 1) / across;
  const int64_t walk = lanes == 64 ? 2 : 1, most = (M + walk * side - 1) / (walk * side);
  if (slabs > most) slabs = most;
  return {lanes, slabs};
}

template <int LP, int NT>
hipError_t run_act_backward(const uint16_t* dy, const uint16_t* pre, int act, uint16_t* dz, float* part, int64_t M,
                            int64_t N, int64_t slabs, hipStream_t stream) {
  hipLaunchKernelGGL((act_backward_kernel<LP, NT>), dim3((unsigned)((N + LP * 8 - 1) / (LP * 8)), (unsigned)slabs),
                     dim3(NT), 0, stream, dy, pre, act, dz, part, M, N, (M + slabs - 1) / slabs);
  return hipGetLastError();
}

}  // namespace

// How a shape runs (MI355X, 256 CUs; us measured with bias and residual).
//
// Few outputs: the smallest tile of 16x16 blocks whose grid gives no CU more
// than one workgroup, since a CU's share of the rows has to pass through its
// own L1 at 40-50 bytes a clock whatever the tile: 1x4096x4096 5.2 with 16x16
// blocks and 16 waves (16x32: 5.6), 64x4096x4096 7.3 with 32x32 (64x32 10.3,
// 32x16 8.2), 256x4096x4096 15.4 with 64x64 (64x32 19.3; 128x128 tiles split
// four ways over K 23.1), 128x12288x4096 22.0 with 64x96 (64x64 in pairs 24.2),
// 500x3000x3008 18.6 (24.8; but 128x12288x512 10.3, in pairs 9.0).  Above that, up to two workgroups per CU (64x64,
// two waves): 512x4096x2048 16.1 (128x128 tiles 23.0), 512x4096x12288 as
// long as 128x128 split in two, 777x2053x2064 20.0 (27.1).
//
// More outputs: the cheapest of the tiles and splits by an estimate of rounds
// of workgroups times (rate * K + what a tile costs besides), plus the second
// launch that joins splits of K.  The rates are fitted to sweeps: 256x256
// tiles 4096x4096x12288 303 (256x128 333, 128x128 337), 128x128 with two K
// groups 2048x2048x8192 67 (256x128 split in two 70) and 1024x4096x4096 40.1
// (256x128 50.7), 256x128 split in three 3000x700x8000 49 (128x128, two K
// groups, unsplit: 60), 128x128 two to a CU 3000x3000x512 30 (256x256 34,
// 256x128 33) and 5000x5000x4096 202 (256x256 216).
LinearPlan linear_plan(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kCus = 256;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int64_t area = up(up(M, 16) * up(N, 16), kCus);   // blocks per CU
  if (M <= 16) return {area <= 1 ? kRows1x1 : area <= 2 ? kRows1x2 : kRows1x4, 1};
  if (area <= 2) return {kRows2x1, 1};
  if (area <= 4) return {kRows2x2, 1};
  if (M <= 32) return {kRows2x4, 1};
  if (area <= 8) return {kRows4x2, 1};
  if (area <= 16) return {kRows4x4, 1};
  if (K >= 1536 && up(M, 64) * up(N, 96) <= kCus) return {kRows4x6, 1};
  if (M <= 64) return {kRows4x4Pair, 1};
  if (area <= 32) return {kRows4x4Pair, 1};
  auto tiles = [&](int bm, int bn) { return up(M, bm) * up(N, bn); };
  const double k0 = (double)K;
  LinearPlan best{kTile256x256, 1};
  double least = (double)up(tiles(256, 256), kCus) * (0.0225 * k0 + 25.0);
  auto offer = [&](LinearPlan p, double us) {
    if (us < least) {
      least = us;
      best = p;
    }
  };
  const double pairs = (double)tiles(128, 128) / (2 * kCus);   // rounds of two workgroups per CU
  if (pairs <= 0.5) offer({kTile128x128, 1}, 0.0075 * k0 + 12.0);
  else offer({kTile128x128, 1}, (pairs <= 1.0 ? 1.0 : 0.5 * (pairs + (double)up(tiles(128, 128), 2 * kCus))) *
                                    (0.0122 * k0 + 12.0));
  const int64_t stages = up(K, 128);
  for (int s = 1; s <= 4 && (s == 1 || stages >= 8 * s); ++s) {
    const double k = (double)(up(stages, s) * 128);
    const double join = s == 1 ? 0.0 : 4.0 + (double)s * (double)M * (double)N * 8.0 / 12e6;
    offer({kTile256x128, s}, (double)up(tiles(256, 128) * s, kCus) * (0.0118 * k + 13.0) + join);
  }
  offer({kTile128x128K2, 1}, (double)up(tiles(128, 128), kCus) * (0.0066 * k0 + 13.0));
  return best;
}

size_t linear_act_workspace(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  const LinearPlan p = linear_plan(M, N, K);
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * sizeof(float) : 0;
}

hipError_t launch_linear_act(const LinearActArgs& g, int accum, float* ws, int num_cus, hipStream_t stream) {
  const LinearPlan p = linear_plan(g.M, g.N, g.K);
  switch (p.tile) {
    case kRows1x1: return launch_rows<1, 1, 16>(g, stream);
    case kRows1x2: return launch_rows<1, 2, 8>(g, stream);
    case kRows1x4: return launch_rows<1, 4, 4>(g, stream);
    case kRows2x1: return launch_rows<2, 1, 8>(g, stream);
    case kRows2x2: return launch_rows<2, 2, 8>(g, stream);
    case kRows2x4: return launch_rows<2, 4, 4>(g, stream);
    case kRows4x2: return launch_rows<4, 2, 4>(g, stream);
    case kRows4x4: return launch_rows<4, 4, 4>(g, stream);
    case kRows4x6: return launch_rows<4, 6, 4>(g, stream);
    case kRows4x4Pair: return launch_rows<4, 4, 2>(g, stream);
    default: break;
  }
  const hipError_t e = launch_linear_tile(g, p, accum, ws, num_cus, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  // rows along x, which takes any number of them
  const int64_t across = (kJoinRows * ((g.N + 3) / 4) + 255) / 256;
  const dim3 grid((unsigned)((g.M + kJoinRows - 1) / kJoinRows), (unsigned)(across < 65535 ? across : 65535));
  if ((g.N & 3) == 0)
    hipLaunchKernelGGL(linear_join_kernel<true>, grid, dim3(256), 0, stream, g, ws, p.splits);
  else
    hipLaunchKernelGGL(linear_join_kernel<false>, grid, dim3(256), 0, stream, g, ws, p.splits);
  return hipGetLastError();
}

// (one slab's sums are the results)
int64_t act_backward_partials(int64_t M, int64_t N) {
  const int64_t slabs = M == 0 || N == 0 ? 0 : act_shape(M, N).slabs;
  return slabs == 1 ? 0 : slabs;
}

hipError_t launch_act_backward(const uint16_t* dy, const uint16_t* pre, int act, uint16_t* dz,
                               float* dbias, int64_t M, int64_t N, float* part, hipStream_t stream) {
  if (M > 0 && N > 0) {
    const ActShape s = act_shape(M, N);
    float* p = dbias != nullptr && s.slabs > 1 ? part : dbias;
    hipError_t e;
    switch (s.lanes) {
      case 4: e = run_act_backward<4, 1024>(dy, pre, act, dz, p, M, N, s.slabs, stream); break;
      case 8: e = run_act_backward<8, 256>(dy, pre, act, dz, p, M, N, s.slabs, stream); break;
      case 16: e = run_act_backward<16, 256>(dy, pre, act, dz, p, M, N, s.slabs, stream); break;
      case 32: e = run_act_backward<32, 256>(dy, pre, act, dz, p, M, N, s.slabs, stream); break;
      default: e = run_act_backward<64, 256>(dy, pre, act, dz, p, M, N, s.slabs, stream); break;
    }
    if (e != hipSuccess || s.slabs == 1) return e;
  }
  if (dbias == nullptr) return hipSuccess;
  return launch_sum_slabs(part, dbias, nullptr, act_backward_partials(M, N), N, N, stream);
}

}  // namespace fp8mot
