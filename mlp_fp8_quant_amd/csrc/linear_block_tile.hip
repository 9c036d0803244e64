// Tiled product of FP8 operands with a scale for each block of 128 of K, and
// fp8_linear_act's epilogue: the kernel behind fp8_linear_block for all but few
// rows.
//
// A workgroup of WM x WN waves, 64 x 32 FN outputs each, computes a BM x BN tile
// from 128-K stages that the buffer unit copies straight into LDS, as in
// linear_act_tile.hip.  A stage is one block: its products are summed from zero
// in accumulators of their own (64 registers beside the 64 of the sums, which is
// what keeps a wave's part at 64 x 64), and the sums take them with one FMA each,
// spread over the MFMAs of the next stage's first step.  W is the first operand:
// register v of lane l of a 32 x 32 block is column n = 8 (v/4) + 4 (l/32) + v%4
// of row m = l % 32, so that a lane needs the scales of two rows of X and, where
// W has one per 128 x 128, one more for all its products; only rows of W with
// scales of their own need 16 for each 32 columns.
//
// Scales come in batches of four stages through LDS, each read for two stages
// before the next batch is on its way into the other of two slots: those of X as
// 16 bytes per row, W's as 16 bytes for the tile's 128 columns or, per row, four
// bytes per lane and stage (column-major, for 16-byte reads).
//
// Many rows are bound by what issues beside the MFMAs and by power: at
// 16384x25600x5120 (3470 to 3670 us, 1.17 to 1.24 PFLOP/s) the matrix cores work in
// 64% of the cycles at 1.67 GHz, and decodes, FMAs and addresses issue in 55%.  A
// wave's part of 64 x 32 decodes half as much again for each MFMA, but two K groups
// of four such waves fill a CU's places where there are few tiles: 512x4096x12288 56
// to 60 us (on the card of the 56, 67 with parts of 64 x 64), 0.86 to 0.92 PFLOP/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "device_common.h"
#include "gemm_parts.h"
#include "kernels.h"
#include "linear_epilogue.h"

namespace fp8mot {

namespace {

using namespace tile;

constexpr int KS = 128;           // K per stage
constexpr int CH = KS / 16;       // 16-byte chunks per LDS row
constexpr int RPI = 1024 / KS;    // LDS rows filled by one wave-wide copy
constexpr int kBand = 8;          // tile rows per band
constexpr int NB = 2;             // stages in LDS
constexpr int kBatch = 4;         // stages whose scales come together

__device__ __forceinline__ int swz(int r, int c) { return c ^ ((r >> 1) & (CH - 1)); }

typedef const __attribute__((address_space(4))) void* kernarg_ptr_t;

constexpr std::true_type yes{};
constexpr std::false_type no{};
constexpr std::integral_constant<int, 0> buf0{};
constexpr std::integral_constant<int, 1> buf1{};
// f with the sequence's numbers as constants
template <class F, int... I>
__device__ __forceinline__ void for_each(std::integer_sequence<int, I...>, F f) {
  f(std::integral_constant<int, I>{}...);
}

struct BlockTileArgs {
  LinearActArgs a;
  int tiles_m, tiles_n;
};

// WROWS: W has a scale for each row.  KFULL: K is a multiple of the stage.  FN:
// blocks of 32 columns of a wave's part.
// KSPL = 2: two groups of WM x WN waves share the tile, taking the even and the
// odd stages, and their sums are added (even + odd) through LDS; KSPL = 1 and
// PERSIST: workgroups walk tiles blockIdx.x, + gridDim.x, .. with the next tile's
// first stages copied in before this tile's epilogue, whose LDS is then apart
// from the stages.
template <int WM, int WN, int FN, int KSPL, bool PERSIST, bool WROWS, bool KFULL>
__global__ __launch_bounds__(WM* WN * 64 * KSPL, 2) void linear_block_tile_kernel(BlockTileArgs t) {
  const int M = (int)t.a.M, N = (int)t.a.N, K = (int)t.a.K;
  constexpr int BM = 64 * WM, BN = 32 * FN * WN, NW = WM * WN, FM = 2;
  static_assert(128 % BN == 0, "one column of W's scale tiles");
  static_assert(!PERSIST || KSPL == 1, "");
  constexpr int A_STAGE = BM * KS, B_STAGE = BN * KS, STAGE = A_STAGE + B_STAGE;
  constexpr int EPI = 4096;   // epilogue bytes per wave
  constexpr int A_LPW = BM / RPI / NW, B_LPW = BN / RPI / NW, LPW = A_LPW + B_LPW;   // copies of a wave
  static_assert(LPW * NW * RPI == BM + BN, "tile rows / waves");
  constexpr int XS = BM * 16, WS = WROWS ? BN * 16 : 256, SLOT = XS + WS;   // scales of a batch
  constexpr int CODES = KSPL * NB * STAGE, LDS = CODES + 2 * SLOT + (PERSIST ? NW * EPI : 0);
  static_assert(LDS <= 160 * 1024, "stages, scales and epilogue fit the 160 KB LDS of a CU");
  static_assert(PERSIST || NW * EPI <= NB * STAGE, "the epilogue fits the stage buffers");
  static_assert(KSPL == 1 || NW * FM * FN * 16 * 64 * 4 <= CODES, "sums fit the stage buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];

  const int tid = threadIdx.x, lane0 = tid & 63;
  const int wave_id = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = KSPL == 1 ? 0 : wave_id / NW;
  const int wave = wave_id - kg * NW;
  const int wm = wave / WN, wn = wave % WN;
  auto a_buf = [&](int b) -> uint8_t* { return smem + kg * NB * STAGE + b * A_STAGE; };
  auto b_buf = [&](int b) -> uint8_t* { return smem + kg * NB * STAGE + NB * A_STAGE + b * B_STAGE; };
  auto lds_of = [&](const uint8_t* p) { return (uint32_t)reinterpret_cast<uintptr_t>((lds_ptr_t)p); };
  const int stages = (K + KS - 1) / KS;
  auto gstage = [&](int i) { return i * KSPL + kg; };
  const int KT = (stages + KSPL - 1) / KSPL;
  const int ntiles = t.tiles_m * t.tiles_n;

  struct Windows {
    v4i a, b, xs, ws;
  };
  auto windows = [&](int m0, int n0) -> Windows {
    const int64_t w0 = WROWS ? n0 : n0 / KS, w_rows = WROWS ? N : (N + KS - 1) / KS;
    return {make_rsrc_words(t.a.qx + (int64_t)m0 * K, (int64_t)(M - m0) * K),
            make_rsrc_words(t.a.qw + (int64_t)n0 * K, (int64_t)(N - n0) * K),
            make_rsrc_words(t.a.sx + (int64_t)m0 * stages, (int64_t)(M - m0) * stages * 4),
            make_rsrc_words(t.a.sw + w0 * stages, (w_rows - w0) * stages * 4)};
  };
  // Copies of a stage: the wave's i-th of A fills LDS rows 8 (wave * A_LPW + i) ..
  // + 7, its others B's rows likewise; lane l brings row l/CH of them, physical
  // chunk l % CH, i.e. logical chunk swz(row, l % CH).  copy_offsets gives the
  // lane's offset in each copy and, as kc, the column of its chunk in even and in
  // odd ones.
  static_assert(A_LPW % 2 == 0 && B_LPW % 2 == 0 && (2 * RPI) % (2 * CH) == 0, "two columns per lane");
  auto copy_offsets = [&](int m0, int n0, int* goff, int* kc) {
    int ln = lane0;
    // opaque, so that no part of this is kept in registers across the epilogue
    if constexpr (PERSIST) asm volatile("" : "+v"(ln));
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
      const bool a = i < A_LPW;
      const int lr = (a ? wave * A_LPW + i : wave * B_LPW + i - A_LPW) * RPI + ln / CH;
      const int c = swz(lr, ln % CH);
      goff[i] = lr < (a ? M - m0 : N - n0) ? lr * K + c * 16 : kOOB;
      if (i < 2) kc[i] = c * 16;
    }
  };
  const uint32_t a_dst = lds_of(a_buf(0) + wave * A_LPW * 1024), b_dst = lds_of(b_buf(0) + wave * B_LPW * 1024);
  // Copy I of this wave for stage s into buffer B.  Unless `inside` (the stage
  // exists), one past the end reads through an empty descriptor: zeros land in
  // LDS.  Unless K is a multiple of the stage, chunks past K's end get an offset
  // past the window.
  auto issue_copy = [&](const Windows& w, const int* goff, const int* kc, auto buffer, int s, auto copy, auto inside) {
    constexpr int I = decltype(copy)::value, B = decltype(buffer)::value;
    const int k0 = s * KS;
    const v4i rs = I < A_LPW ? w.a : w.b;
    const int off = KFULL || kc[I & 1] < K - k0 ? goff[I] : kOOB;
    const bool in = decltype(inside)::value || s < stages;
    copy_to_lds_at<I < A_LPW ? B * A_STAGE + I * 1024 : B * B_STAGE + (I - A_LPW) * 1024>(
        in ? rs : (v4i){0, 0, 0, 0x00020000}, I < A_LPW ? a_dst : b_dst, off, in ? k0 : 0);
  };
  auto issue_copies = [&](const Windows& w, const int* goff, const int* kc, auto buffer, int s, auto inside,
                          auto... copy) { (issue_copy(w, goff, kc, buffer, s, copy, inside), ...); };
  auto issue_stage = [&](const Windows& w, const int* goff, const int* kc, auto buffer, int s) {
    for_each(std::make_integer_sequence<int, LPW>{}, [&](auto... i) { issue_copies(w, goff, kc, buffer, s, no, i...); });
  };
  // Scales of batch h (stages 4h .. 4h + 3) into slot h & 1: 64 rows of X to a
  // copy, and W's.  A row's 16 bytes may run into the next row's, which no stage
  // reads; rows past M or N lie past the window.
  constexpr int X_COPIES = BM / 64, W_COPIES = WROWS ? kBatch * BN / 64 : 1, WAVES = NW * KSPL;
  static_assert(X_COPIES + 1 <= WAVES && (W_COPIES < WAVES || W_COPIES % WAVES == 0), "a wave's copies");
  auto issue_scales = [&](const Windows& w, int h) {
    int ln = lane0;
    if constexpr (PERSIST) asm volatile("" : "+v"(ln));
    const uint32_t dst = lds_of(smem + CODES + (h & 1) * SLOT);
    // one copy per wave: the waves past X's take the tile's scale of W, all of
    // them the same
    const bool x = wave_id < X_COPIES;
    if constexpr (WROWS) {
      if (x) copy_to_lds(w.xs, dst + wave_id * 1024, (wave_id * 64 + ln) * stages * 4, h * 16);
#pragma unroll
      for (int c = 0; c < (W_COPIES + WAVES - 1) / WAVES; ++c) {
        const int d = c * WAVES + wave_id, s = d / (BN / 64), r = d % (BN / 64);
        const int off = h * kBatch + s < stages ? (r * 64 + ln) * stages * 4 : kOOB;
        if (W_COPIES >= WAVES || d < W_COPIES) copy4_to_lds(w.ws, dst + XS + d * 256, off, h * 16 + s * 4);
      }
    } else {
      if (x) copy_to_lds(w.xs, dst + wave_id * 1024, (wave_id * 64 + ln) * stages * 4, h * 16);
      else copy4_to_lds(w.ws, dst + XS, ln < kBatch ? ln * 4 : kOOB, h * 16);
    }
  };

  bool staged = false;
  for (int tile = blockIdx.x, iter = 0; PERSIST ? tile < ntiles : iter < 1; tile += gridDim.x, ++iter) {
  // opaque per tile: addresses and the divisions of tile_of are formed per
  // tile instead of being kept in registers across the epilogue
  int lane = lane0, tiles_m = t.tiles_m, tiles_n = t.tiles_n;
  if constexpr (PERSIST) asm volatile("" : "+v"(lane), "+s"(tiles_m), "+s"(tiles_n));
  int tm, tn;
  tile_of(tile, tiles_m, tiles_n, kBand, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const Windows win = windows(m0, n0);
  int goff[LPW], kc[2];
  copy_offsets(m0, n0, goff, kc);
  v16f acc[FM][FN], p[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = p[i][j][v] = 0.0f;

  // per-lane LDS bases of the chunks a lane reads, one per chunk slot of a
  // stage; blocks and stage buffers are immediate offsets from them
  constexpr int NSTEP = KS / 32;
  int lds_a[NSTEP], lds_b[NSTEP];
  const int half = lane >> 5;
  {
    const int l31 = lane & 31;
    const int ra = wm * 64 + l31, rb = wn * (32 * FN) + l31;
#pragma unroll
    for (int k = 0; k < NSTEP; ++k) {
      lds_a[k] = (int)(a_buf(0) - smem) + ra * KS + (swz(ra, 2 * k + half) << 4);
      lds_b[k] = (int)(b_buf(0) - smem) + rb * KS + (swz(rb, 2 * k + half) << 4);
      asm volatile("" : "+v"(lds_a[k]), "+v"(lds_b[k]));
    }
  }
  // scales of the last finished block: X's two rows, W's tile or (WROWS) where
  // its columns' lie
  const int xs_at = CODES + (wm * 64 + (lane & 31)) * 16;
  const int ws_at = CODES + XS + (WROWS ? (wn * (32 * FN) + 4 * half) * 4 : 0);
  float sx[FM] = {0.0f, 0.0f}, sw = 0.0f;
  int sw_at = ws_at + SLOT;   // zeros at first, for the sums of no block (a scale there could be infinite)
  if (WROWS && tid < BN / 4) *reinterpret_cast<v4f*>(smem + CODES + SLOT + XS + 16 * tid) = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  auto read_scales = [&](int s) {
    const int slot = ((s / kBatch) & 1) * SLOT, k = s % kBatch;
#pragma unroll
    for (int i = 0; i < FM; ++i) sx[i] = *reinterpret_cast<const float*>(smem + xs_at + i * 512 + slot + k * 4);
    if constexpr (WROWS) sw_at = ws_at + slot + k * (BN * 4);
    else sw = *reinterpret_cast<const float*>(smem + ws_at + slot + k * 4);
  };
  // W's scales of columns 32 j + 8 k + 4 half .. + 3 of the last finished block
  auto column_scales = [&](int j, v4f* w) {
    if constexpr (WROWS) {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const v4f*>(smem + sw_at + (32 * j + 8 * k) * 4);
    }
  };
  // c + scale * q: the sums of a 32 x 32 block
  auto promoted = [&](v16f c, const v16f q, float sx, const v4f* w) -> v16f {
    const float s = __fmul_rn(sx, sw);
#pragma unroll
    for (int v = 0; v < 16; ++v) c[v] = __builtin_fmaf(q[v], WROWS ? __fmul_rn(sx, w[v / 4][v % 4]) : s, c[v]);
    return c;
  };
  auto chunk_at = [&](int base, int imm) -> v4i { return *reinterpret_cast<const v4i*>(smem + base + imm); };
  v4i fa[2][FM], fb[2][FN];
  auto rd = [&](int b, int st, int slot) {
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[slot][i] = chunk_at(lds_a[st], b * A_STAGE + i * 32 * KS);
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[slot][j] = chunk_at(lds_b[st], b * B_STAGE + j * 32 * KS);
    __builtin_amdgcn_sched_barrier(0);   // reads ahead of the MFMAs that follow
  };
  // MFMAs of one K-step; the first of a stage takes the last stage's sums first
  // and starts from zero; with copies, those of stage cs into buffer cb go out
  // spread over the block rows
  auto mf = [&](int slot, auto first, auto copies, auto cb, int cs) {
    constexpr bool kFirst = decltype(first)::value, kCopies = decltype(copies)::value;
    f16x8 a0[FM], a1[FM], b0[FN], b1[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const v4i v = fa[slot][i];
      a0[i] = decode8(v[0], v[1]);
      a1[i] = decode8(v[2], v[3]);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const v4i v = fb[slot][j];
      b0[j] = decode8(v[0], v[1]);
      b1[j] = decode8(v[2], v[3]);
    }
    if constexpr (kFirst) {
      // a block's FMAs issue while the matrix core is at the block before
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        v4f w[4];
        column_scales(j, w);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          acc[i][j] = promoted(acc[i][j], p[i][j], sx[i], w);
          asm volatile("" : "+v"(acc[i][j]));   // done here: moved on, the FMAs would keep a second set of p alive
          const v16f zero = {0.0f};
          p[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b0[j], a0[i], zero, 0, 0, 0);
          p[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b1[j], a1[i], p[i][j], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      return;
    }
    auto row = [&](auto i, auto... copy) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        p[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b0[j], a0[i], p[i][j], 0, 0, 0);
        p[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b1[j], a1[i], p[i][j], 0, 0, 0);
      }
      if constexpr (kCopies) issue_copies(win, goff, kc, cb, cs, yes, copy...);
    };
    for_each(std::make_integer_sequence<int, LPW / 2>{}, [&](auto... i) {
      row(std::integral_constant<int, 0>{}, i...);
      row(std::integral_constant<int, 1>{}, std::integral_constant<int, LPW / 2 + i>{}...);
    });
  };

  if (!staged) {
    if (KT > 0) issue_scales(win, 0);
    if (KT > 0) issue_stage(win, goff, kc, buf0, gstage(0));
    if (KT > 1) issue_stage(win, goff, kc, buf1, gstage(1));
  }
  if (KT > 0) {
    // the first stage and the scales before it have landed; where staged the
    // previous epilogue's accesses count too: wait for all (vmcnt alone: gfx9
    // encoding)
    static_assert(LPW < 64, "vmcnt has six bits");
    if (!PERSIST && KT > 1) __builtin_amdgcn_s_waitcnt(0x0F70 | (LPW & 15) | ((LPW >> 4) << 14));
    else __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    rd(0, 0, 0);
  }
  // Per stage: before the MFMAs of a step the next step's fragments are read;
  // at the last step wait for the next stage's copies and this wave's own
  // reads, barrier, read ahead, and refill the freed buffer with stage s + 2.
  // The scales of the next batch go out after the first stage of this one, whose
  // barrier follows the last use of their slot.  inside: stage s + 2 of both
  // groups exists, so that nothing is asked or selected per stage.
  auto stage = [&](auto buffer, int s, auto inside) {
    constexpr bool kInside = decltype(inside)::value;
    constexpr int u = decltype(buffer)::value;
#pragma unroll
    for (int st = 0; st + 1 < NSTEP; ++st) {
      rd(u, st + 1, (st & 1) ^ 1);
      if (st == 1) __builtin_amdgcn_s_setprio(0);
      if (st == 0) mf(st & 1, yes, no, buf0, 0);
      else mf(st & 1, no, no, buf0, 0);
    }
    constexpr int slot = (NSTEP - 1) & 1;
    if (kInside || s + 1 < KT) {
      __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
      __syncthreads();
      if (s * KSPL % kBatch == 0 && s * KSPL + kBatch < stages) issue_scales(win, s * KSPL / kBatch + 1);
      rd(u ^ 1, 0, slot ^ 1);
    }
    __builtin_amdgcn_s_setprio(1);
    read_scales(gstage(s));
    mf(slot, no, inside, buffer, gstage(s + NB));
    if constexpr (!kInside) {
      if (s + NB < KT) issue_stage(win, goff, kc, buffer, gstage(s + NB));
    }
  };
  int s = 0;
  for (; (s + NB + 1) * KSPL + KSPL <= stages; s += NB) {
    stage(buf0, s, yes);
    stage(buf1, s + 1, yes);
  }
  for (; s < KT; s += NB) {
    stage(buf0, s, no);
    if (s + 1 < KT) stage(buf1, s + 1, no);
  }
  // (of an odd number of stages the second group has no last one: its scale would
  // be the next row's, which zeros times an infinity would not survive)
  if (KT > 0 && gstage(KT - 1) < stages) {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      v4f w[4];
      column_scales(j, w);
#pragma unroll
      for (int i = 0; i < FM; ++i) acc[i][j] = promoted(acc[i][j], p[i][j], sx[i], w);
    }
  }
  // no copy into LDS may be on its way when the buffers are refilled or the
  // workgroup ends
  __builtin_amdgcn_s_waitcnt(0x0F70);

  if constexpr (KSPL == 2) {
    __syncthreads();
    v4f* red = reinterpret_cast<v4f*>(smem) + wave * (FM * FN * 4 * 64) + lane;
    if (kg == 1) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            red[((i * FN + j) * 4 + q) * 64] =
                (v4f){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    }
    __syncthreads();
    if (kg == 1) return;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const v4f o = red[((i * FN + j) * 4 + q) * 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] = __fadd_rn(acc[i][j][4 * q + e], o[e]);
        }
  }

  staged = false;
  if (PERSIST && tile + (int)gridDim.x < ntiles) {
    __syncthreads();
    int ntm, ntn;
    tile_of(tile + gridDim.x, tiles_m, tiles_n, kBand, ntm, ntn);
    const Windows nw = windows(ntm * BM, ntn * BN);
    int ngoff[LPW], nkc[2];
    copy_offsets(ntm * BM, ntn * BN, ngoff, nkc);
    if (KT > 0) issue_scales(nw, 0);
    if (KT > 0) issue_stage(nw, ngoff, nkc, buf0, gstage(0));
    if (KT > 1) issue_stage(nw, ngoff, nkc, buf1, gstage(1));
    staged = true;
  }

  // ---- epilogue ----
  // Its arguments are read here, through a pointer that the compiler cannot
  // see through, instead of being kept in scalar registers over the main loop
  // (see linear_act_tile.hip).
  kernarg_ptr_t ka = (kernarg_ptr_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(ka));
  const LinearActArgs& g = ((const BlockTileArgs*)ka)->a;
  // A 32 x 32 block goes through 4 KB of LDS of the wave's own, row m at 128 m,
  // four columns (c = n / 4) at chunk c ^ (m & 7), and comes back as four
  // consecutive columns of four rows per lane.
  if constexpr (!PERSIST && KSPL == 1) __syncthreads();   // every wave has read its last fragments
  // KSPL 2: the wave's own part of the sums' buffer, which it alone has read
  float* epi = reinterpret_cast<float*>(
      smem + (PERSIST ? CODES + 2 * SLOT + wave * EPI : (KSPL == 2 ? wave * (FM * FN * 4096) : wave * EPI)));
  int el = lane0;   // opaque: nothing the epilogue derives from it is formed before
  asm volatile("" : "+v"(el));
  const int er = el >> 3, ec = 4 * (el & 7);
  float* const put = epi + (el & 31) * 32;
  const int turn = el & 7, up = el >> 5;
  const float* const get = epi + er * 32 + 4 * ((el & 7) ^ er);
  const int row_w = wm * 64 + er, nw = n0 + wn * (32 * FN) + ec;   // row from m0
  auto blocks_loop = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    const linear::Epilogue e = linear::open_outputs(g, m0);
    linear::Columns cols[FN];
    linear::Operands<4> op;
    auto operands_of = [&](int b) {
      const int n = nw + 32 * (b % FN);
      linear::load_operands<4, VEC>(g, e, m0, row_w + 32 * (b / FN), 8, n, N - n, &op);
    };
#pragma unroll
    for (int j = 0; j < FN; ++j) cols[j] = linear::load_columns<VEC>(g, nw + 32 * j, N - nw - 32 * j);
    operands_of(0);
#pragma unroll 1
    for (int b = 0; b < FM * FN; ++b) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          if (b == i * FN + j) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<v4f*>(put + 4 * ((2 * q + up) ^ turn)) =
                  (v4f){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          }
      float z[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const v4f s = *reinterpret_cast<const v4f*>(get + 8 * k * 32);
#pragma unroll
        for (int c = 0; c < 4; ++c) z[k][c] = s[c];
      }
      const int row = row_w + 32 * (b / FN), n = nw + 32 * (b % FN);
      linear::Columns col = cols[0];
#pragma unroll
      for (int j = 1; j < FN; ++j)
        if (b % FN == j) col = cols[j];
      linear::finish<4, VEC>(g, e, col, row, 8, n, N - n, op, z, [&] {
        if (b + 1 < FM * FN) operands_of(b + 1);
      });
    }
  };
  if ((N & 3) == 0) blocks_loop(yes);
  else blocks_loop(no);
  }  // tiles
}

template <int WM, int WN, int FN, int KSPL, bool PERSIST, bool WROWS, bool KFULL>
hipError_t launch_kernel(const LinearActArgs& a, int num_cus, hipStream_t stream) {
  BlockTileArgs t{};
  t.a = a;
  t.a.row_scales = 0;   // the epilogue's sums are scaled already
  t.tiles_m = (int)((a.M + 64 * WM - 1) / (64 * WM));
  t.tiles_n = (int)((a.N + 32 * FN * WN - 1) / (32 * FN * WN));
  auto kern = linear_block_tile_kernel<WM, WN, FN, KSPL, PERSIST, WROWS, KFULL>;
  const int64_t tiles = (int64_t)t.tiles_m * t.tiles_n;
  // (one workgroup of a kernel that walks tiles fits a CU)
  const int64_t grid = PERSIST && tiles > num_cus && num_cus >= kNumXcd ? num_cus - num_cus % kNumXcd : tiles;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(WM * WN * 64 * KSPL), 0, stream, t);
  return hipGetLastError();
}

template <int WM, int WN, int FN, int KSPL, bool PERSIST>
hipError_t launch_shape(const LinearActArgs& a, int num_cus, hipStream_t stream) {
  if (a.K % KS == 0)
    return a.row_scales ? launch_kernel<WM, WN, FN, KSPL, PERSIST, true, true>(a, num_cus, stream)
                        : launch_kernel<WM, WN, FN, KSPL, PERSIST, false, true>(a, num_cus, stream);
  return a.row_scales ? launch_kernel<WM, WN, FN, KSPL, PERSIST, true, false>(a, num_cus, stream)
                      : launch_kernel<WM, WN, FN, KSPL, PERSIST, false, false>(a, num_cus, stream);
}

}  // namespace

hipError_t launch_linear_block_tile(const LinearActArgs& g, int tile, int num_cus, hipStream_t stream) {
  switch (tile) {
    case kTile256x128: return launch_shape<4, 2, 2, 1, true>(g, num_cus, stream);
    case kTile128x128: return launch_shape<2, 2, 2, 1, false>(g, num_cus, stream);
    case kTile128x64K2: return launch_shape<2, 2, 1, 2, false>(g, num_cus, stream);
    case kTile128x64: return launch_shape<2, 2, 1, 1, false>(g, num_cus, stream);
    default: return launch_shape<2, 2, 2, 2, false>(g, num_cus, stream);
  }
}

}  // namespace fp8mot
