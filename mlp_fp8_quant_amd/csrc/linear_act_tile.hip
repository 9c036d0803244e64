// Tiled FP8 x FP8 product with bias, activation and residual in its epilogue:
// the kernel behind fp8_linear_act for all but few rows.
//
// The main loop is laid out as in gemm.hip: a workgroup of WM x WN waves
// computes a BM x BN tile from 128-K stages that the buffer unit copies
// straight into LDS (rows of 128 codes, 16-byte chunk c of row r at chunk
// c ^ ((r >> 1) & 7)); the exact engine decodes each fragment to F16 and
// multiplies with v_mfma_f32_32x32x16_f16, the native engine multiplies the
// codes with v_mfma_f32_32x32x64_f8f6f4.  Rows past M or N and K past its end
// read as zeros through the buffers' range checks.
//
// The epilogue takes the accumulators one 32x32 block at a time through 4 KB
// of LDS of the wave's own, from the MFMA's layout (register v of lane l: row
// 8 (v/4) + 4 (l/32) + v%4, column l % 32) to four consecutive columns of
// four rows per lane, and runs a rolled loop over the blocks: one copy of the
// code for every activation and type, accumulators that are only read, the
// next block's residual on its way meanwhile.  (Unrolled over the
// accumulators in place, the activations' branches made the 256x256 kernel
// spill 950 registers: 16384x25600x5120 5.17 ms; 3.1 ms so, 1.38 PFLOP/s.)
// Bound by the matrix cores' clock under load and by the decodes between them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "act.h"
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

__device__ __forceinline__ int swz(int r, int c) { return c ^ ((r >> 1) & (CH - 1)); }

typedef const __attribute__((address_space(4))) void* kernarg_ptr_t;

struct TileArgs {
  LinearActArgs a;
  int tiles_m, tiles_n;
  int split_stages;   // K stages of one split (gridDim.y splits)
  float* part;        // not NULL: raw sums of each split into [splits, M, N]
};

// KFULL: K is a multiple of the stage.  KSPL = 2: two groups of WM x WN waves share the tile, taking the even and
// the odd stages, and their sums are added (even + odd) through LDS.  DEEP:
// as many stages in LDS as fit, up to four, instead of two.
template <int BM, int BN, int WM, int WN, int ENGINE, bool DEEP, int KSPL, bool KFULL>
__global__ __launch_bounds__(WM* WN * 64 * KSPL, 1) void linear_tile_kernel(TileArgs t) {
  const int M = (int)t.a.M, N = (int)t.a.N, K = (int)t.a.K;
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int FM = WTM / 32, FN = WTN / 32;
  constexpr int STAGE = (BM + BN) * KS;
  constexpr int FIT = (160 * 1024) / (KSPL * STAGE);
  constexpr int NB = !DEEP ? 2 : (FIT < 4 ? FIT : 4);
  // The exact engine's workgroups walk tiles blockIdx.x, + gridDim.x, .. with
  // the next tile's first stages copied in before this tile's epilogue, whose
  // LDS is then apart from the stages; the native engine's loop keeps too many
  // registers live for that.
  constexpr bool PERSIST = ENGINE == 0 && KSPL == 1;
  constexpr int EPI = 4096;   // epilogue bytes per wave
  constexpr int A_INS = BM / RPI, INS = (BM + BN) / RPI;
  constexpr int LPW = INS / NW;
  static_assert(LPW * NW == INS, "tile rows / waves");
  constexpr int LDS = KSPL * NB * STAGE + (PERSIST ? NW * EPI : 0);
  static_assert(NB >= 2 && LDS <= 160 * 1024, "stages and epilogue fit the 160 KB LDS of a CU");
  static_assert(PERSIST || NW * EPI <= NB * STAGE, "the epilogue fits the stage buffers");
  static_assert(KSPL == 1 || NW * FM * FN * 16 * 64 * 4 <= KSPL * NB * STAGE, "sums fit the stage buffers");
  static_assert((NB - 1) * LPW < 64, "wait_copies");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];

  const int tid = threadIdx.x, lane0 = tid & 63;
  const int wave_id = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = KSPL == 1 ? 0 : wave_id / NW;
  const int wave = wave_id - kg * NW;
  const int wm = wave / WN, wn = wave % WN;
  constexpr int A_STAGE = BM * KS, B_STAGE = BN * KS;
  auto a_buf = [&](int b) -> uint8_t* { return smem + kg * NB * STAGE + b * A_STAGE; };
  auto b_buf = [&](int b) -> uint8_t* { return smem + kg * NB * STAGE + NB * A_STAGE + b * B_STAGE; };
  // this workgroup's stages of K: [s0, s1)
  const int all_stages = (K + KS - 1) / KS;
  const int s0 = (int)blockIdx.y * t.split_stages;
  const int s1 = min(s0 + t.split_stages, all_stages);
  auto gstage = [&](int i) { return s0 + i * KSPL + kg; };
  const int KT = (s1 - s0 + KSPL - 1) / KSPL;
  const int ntiles = t.tiles_m * t.tiles_n;

  struct Windows {
    v4i a, b;
  };
  auto windows = [&](int m0, int n0) -> Windows {
    return {make_rsrc_words(t.a.qx + (int64_t)m0 * K, (int64_t)(M - m0) * K),
            make_rsrc_words(t.a.qw + (int64_t)n0 * K, (int64_t)(N - n0) * K)};
  };
  // Copy q (= wave * LPW + i) of a stage fills LDS rows q*RPI .. q*RPI+RPI-1
  // (A rows, then B rows); lane l brings row q*RPI + l/CH, physical chunk
  // l % CH, i.e. logical chunk swz(row, l % CH).
  // copy_offsets gives the lane's offset in each copy and, as kc, the column of
  // its chunk in even and in odd ones (rows of consecutive copies lie RPI
  // apart, so the swizzle has no other values).
  static_assert(LPW % 2 == 0 && A_INS % 2 == 0 && (2 * RPI) % (2 * CH) == 0, "two columns per lane");
  auto copy_offsets = [&](int m0, int n0, int* goff, int* kc) {
    int ln = lane0;
    // opaque, so that no part of this is kept in registers across the epilogue
    if constexpr (PERSIST) asm volatile("" : "+v"(ln));
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
      const int q = wave * LPW + i;
      const int lr = (q < A_INS ? q : q - A_INS) * RPI + ln / CH;
      const int c = swz(lr, ln % CH);
      goff[i] = lr < (q < A_INS ? M - m0 : N - n0) ? lr * K + c * 16 : kOOB;
      if (i < 2) kc[i] = c * 16;
    }
  };
  // Copy i of this wave for stage s into buffer b: the stage's column is the
  // wave's scalar offset, and a stage past s1 reads through an empty descriptor
  // (zeros land in LDS).  Unless K is a multiple of the stage (kfull), chunks
  // past K's end get an offset past the window.
  auto issue_copy = [&](const Windows& w, const int* goff, const int* kc, int b, int s, int i, auto kfull) {
    const int k0 = s * KS;
    const int q = wave * LPW + i;
    const v4i rs = q < A_INS ? w.a : w.b;
    const uint32_t dst = (uint32_t)reinterpret_cast<uintptr_t>(
        (lds_ptr_t)(q < A_INS ? a_buf(b) + q * 1024 : b_buf(b) + (q - A_INS) * 1024));
    const int off = decltype(kfull)::value || kc[i & 1] < K - k0 ? goff[i] : kOOB;
    copy_to_lds(s < s1 ? rs : (v4i){0, 0, 0, 0x00020000}, dst, off, s < s1 ? k0 : 0);
  };
  auto issue_stage = [&](const Windows& w, const int* goff, const int* kc, int b, int s, auto kfull) {
#pragma unroll
    for (int i = 0; i < LPW; ++i) issue_copy(w, goff, kc, b, s, i, kfull);
  };

  constexpr std::integral_constant<bool, KFULL> kfull{};
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
  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // per-lane LDS bases of the chunks a lane reads, one per chunk slot of a
  // stage; blocks and stage buffers are immediate offsets from them
  constexpr int NSLOT = 4;
  int lds_a[NSLOT], lds_b[NSLOT];
  {
    const int l31 = lane & 31, half = lane >> 5;
    const int ra = wm * WTM + l31, rb = wn * WTN + l31;
#pragma unroll
    for (int k = 0; k < NSLOT; ++k) {
      const int c = ENGINE == 0 ? 2 * k + half : 4 * (k >> 1) + 2 * half + (k & 1);
      lds_a[k] = (int)(a_buf(0) - smem) + ra * KS + (swz(ra, c) << 4);
      lds_b[k] = (int)(b_buf(0) - smem) + rb * KS + (swz(rb, c) << 4);
      asm volatile("" : "+v"(lds_a[k]), "+v"(lds_b[k]));
    }
  }
  auto chunk_at = [&](int base, int imm) -> v4i { return *reinterpret_cast<const v4i*>(smem + base + imm); };
  // K-steps per stage: exact engine 32 K (one chunk per operand, bytes 0..7
  // and 8..15 to one MFMA each), native engine 64 K (two chunks)
  constexpr int NSTEP = ENGINE == 0 ? KS / 32 : KS / 64;
  typedef typename std::conditional<ENGINE == 0, v4i, v8i>::type frag_t;
  frag_t fa[2][FM], fb[2][FN];
  auto rd = [&](int b, int st, int slot) {
    if constexpr (ENGINE == 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[slot][i] = chunk_at(lds_a[st], b * A_STAGE + i * 32 * KS);
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[slot][j] = chunk_at(lds_b[st], b * B_STAGE + j * 32 * KS);
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[slot][i] = __builtin_shufflevector(chunk_at(lds_a[2 * st], b * A_STAGE + i * 32 * KS),
                                              chunk_at(lds_a[2 * st + 1], b * A_STAGE + i * 32 * KS),
                                              0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[slot][j] = __builtin_shufflevector(chunk_at(lds_b[2 * st], b * B_STAGE + j * 32 * KS),
                                              chunk_at(lds_b[2 * st + 1], b * B_STAGE + j * 32 * KS),
                                              0, 1, 2, 3, 4, 5, 6, 7);
    }
    __builtin_amdgcn_sched_barrier(0);   // reads ahead of the MFMAs that follow
  };
  // MFMAs of one K-step; with copies, those of stage cs into buffer cb go out
  // spread over the block rows
  constexpr int CPR = (LPW + FM - 1) / FM;
  auto mf = [&](int slot, auto copies, int cb, int cs) {
    constexpr bool kCopies = decltype(copies)::value;
    auto send = [&](int i) {
      if constexpr (kCopies) {
#pragma unroll
        for (int c = 0; c < CPR; ++c)
          if (i * CPR + c < LPW) issue_copy(win, goff, kc, cb, cs, i * CPR + c, kfull);
      }
    };
    if constexpr (ENGINE == 0) {
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
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a0[i], b0[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a1[i], b1[j], acc[i][j], 0, 0, 0);
        }
        send(i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[slot][i], fb[slot][j], acc[i][j], 0, 0,
                                                                     0, 0, 0, 0);
        send(i);
      }
    }
  };
  // wait until at most n of this wave's copies are in flight (s_waitcnt
  // vmcnt(n), the other counters left alone: gfx9 encoding)
  auto wait_copies = [&](int n) {
    if (NB > 3 && n >= 3 * LPW) __builtin_amdgcn_s_waitcnt(0x0F70 | ((3 * LPW) & 15) | (((3 * LPW) >> 4) << 14));
    else if (NB > 2 && n >= 2 * LPW) __builtin_amdgcn_s_waitcnt(0x0F70 | ((2 * LPW) & 15) | (((2 * LPW) >> 4) << 14));
    else if (n >= LPW) __builtin_amdgcn_s_waitcnt(0x0F70 | (LPW & 15) | ((LPW >> 4) << 14));
    else __builtin_amdgcn_s_waitcnt(0x0F70);
  };

  if (!staged) {
#pragma unroll
    for (int u = 0; u < NB; ++u)
      if (u < KT) issue_stage(win, goff, kc, u, gstage(u), kfull);
  }
  if (KT > 0) {
    // staged: the previous epilogue's accesses were issued after these copies
    // and count in the same counter, so wait for everything
    if (staged) __builtin_amdgcn_s_waitcnt(0x0F70);
    else wait_copies(LPW * (min(NB, KT) - 1));
    __syncthreads();
    rd(0, 0, 0);
  }
  // Per stage: before the MFMAs of a step the next step's fragments are read;
  // at the last step wait for the next stage's copies and this wave's own
  // reads, barrier, read ahead, and refill the freed buffer with stage s + NB
  // (past the end: zeros into a buffer nobody reads again -- at the last
  // stage, where no barrier has freed this one, the next one).
  for (int kt0 = 0; kt0 < KT; kt0 += NB) {
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const int s = kt0 + u;
      if (s < KT) {
#pragma unroll
        for (int st = 0; st < NSTEP; ++st) {
          const int slot = (u * NSTEP + st) & 1;
          if (st + 1 < NSTEP) {
            rd(u, st + 1, slot ^ 1);
            mf(slot, std::false_type{}, 0, 0);
          } else {
            if (s + 1 < KT) {
              wait_copies(LPW * min(NB - 2, KT - s - 2));
              __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
              __syncthreads();
              rd((u + 1) % NB, 0, slot ^ 1);
            }
            mf(slot, std::true_type{}, s + 1 < KT ? u : (u + 1) % NB, gstage(s + NB));
          }
        }
      }
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
#pragma unroll
    for (int u = 0; u < NB; ++u)
      if (u < KT) issue_stage(nw, ngoff, nkc, u, gstage(u), kfull);
    staged = true;
  }

  // ---- epilogue ----
  // Its arguments are read here, through a pointer that the compiler cannot
  // see through: kept in scalar registers over the main loop they would not
  // fit (159 spilled), and a scalar load pending inside it would turn every
  // LDS wait there into a wait for all LDS reads.
  kernarg_ptr_t ka = (kernarg_ptr_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(ka));
  const LinearActArgs& g = ((const TileArgs*)ka)->a;
  float* const part = ((const TileArgs*)ka)->part;
  // Row r of a block lies at LDS row r ^ ((r >> 2) & 1), so that the two
  // half-waves' writes (rows r and r + 4) go to different bank halves.
  if constexpr (!PERSIST && KSPL == 1) __syncthreads();   // every wave has read its last fragments
  // KSPL 2: the wave's own part of the sums' buffer, which it alone has read
  float* epi = reinterpret_cast<float*>(smem + (PERSIST ? KSPL * NB * STAGE + wave * EPI
                                                       : (KSPL == 2 ? wave * (FM * FN * 4096) : wave * EPI)));
  int el = lane0;   // opaque: nothing the epilogue derives from it is formed before
  asm volatile("" : "+v"(el));
  const int up = el >> 5, er = el >> 3, ec = 4 * (el & 7);
  // row r + 4 up of the block, r = 8 q + e with e < 4, goes to LDS row
  // 8 q + 4 up + (e ^ up): one base for even and one for odd e, the rest an
  // immediate; likewise rows er + 8 k
  float* const put_even = epi + (5 * up) * 32 + (el & 31);
  float* const put_odd = epi + (3 * up) * 32 + (el & 31);
  const float* const get = epi + (er ^ ((er >> 2) & 1)) * 32 + ec;
  const int row_w = wm * WTM + er, nw = n0 + wn * WTN + ec;   // row from m0
  auto blocks_loop = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    const bool raw = part != nullptr;
    const linear::Epilogue e = raw ? linear::Epilogue{} : linear::open_epilogue(g, m0);
    const linear::Rows pr = raw ? linear::rows_of(part + (int64_t)blockIdx.y * M * N, m0, M, N, 4) : linear::Rows{};
    linear::Columns cols[FN];
    linear::Operands<4> op;
    auto operands_of = [&](int b) {
      const int n = nw + 32 * (b % FN);
      linear::load_operands<4, VEC>(g, e, m0, row_w + 32 * (b / FN), 8, n, N - n, &op);
    };
    if (!raw) {
#pragma unroll
      for (int j = 0; j < FN; ++j) cols[j] = linear::load_columns<VEC>(g, nw + 32 * j, N - nw - 32 * j);
    }
    if (!raw) operands_of(0);
#pragma unroll 1
    for (int b = 0; b < FM * FN; ++b) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          if (b == i * FN + j) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              const int r = 8 * (v >> 2) + (v & 3);
              ((v & 1) ? put_odd : put_even)[r * 32] = acc[i][j][v];
            }
          }
      float z[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const v4f s = *reinterpret_cast<const v4f*>(get + 8 * k * 32);
#pragma unroll
        for (int c = 0; c < 4; ++c) z[k][c] = s[c];
      }
      const int row = row_w + 32 * (b / FN), n = nw + 32 * (b % FN);
      if (raw) {
#pragma unroll
        for (int k = 0; k < 4; ++k) linear::store4_f32<VEC>(pr, (row + 8 * k) * N + n, N - n, z[k]);
      } else {
        linear::Columns col = cols[0];
#pragma unroll
        for (int j = 1; j < FN; ++j)
          if (b % FN == j) col = cols[j];
        linear::finish<4, VEC>(g, e, col, row, 8, n, N - n, op, z, [&] {
          if (b + 1 < FM * FN) operands_of(b + 1);
        });
      }
    }
  };
  if ((N & 3) == 0) blocks_loop(std::true_type{});
  else blocks_loop(std::false_type{});
  }  // tiles
}

template <int BM, int BN, int WM, int WN, int ENGINE, bool DEEP, int KSPL, bool KFULL>
hipError_t launch_kernel(TileArgs t, int splits, int num_cus, hipStream_t stream) {
  t.tiles_m = (int)((t.a.M + BM - 1) / BM);
  t.tiles_n = (int)((t.a.N + BN - 1) / BN);
  auto kern = linear_tile_kernel<BM, BN, WM, WN, ENGINE, DEEP, KSPL, KFULL>;
  constexpr int block = WM * WN * 64 * KSPL;
  const int64_t tiles = (int64_t)t.tiles_m * t.tiles_n;
  int64_t grid = tiles;
  if (ENGINE == 0 && KSPL == 1) {   // the kernels that walk several tiles
    static std::atomic<int> occupancy{0};
    int occ = occupancy.load(std::memory_order_relaxed);
    if (occ == 0) {
      if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, block, 0) != hipSuccess || occ < 1) occ = 1;
      occupancy.store(occ, std::memory_order_relaxed);
    }
    const int64_t resident = (int64_t)occ * num_cus;
    if (tiles > resident && resident >= kNumXcd) grid = resident - resident % kNumXcd;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)grid, (unsigned)splits), dim3(block), 0, stream, t);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int ENGINE, bool DEEP, int KSPL>
hipError_t launch_shape(const TileArgs& t, int splits, int num_cus, hipStream_t stream) {
  if (t.a.K % KS == 0)
    return launch_kernel<BM, BN, WM, WN, ENGINE, DEEP, KSPL, true>(t, splits, num_cus, stream);
  return launch_kernel<BM, BN, WM, WN, ENGINE, DEEP, KSPL, false>(t, splits, num_cus, stream);
}

template <int ENGINE>
hipError_t launch_engine(const TileArgs& t, const LinearPlan& p, int num_cus, hipStream_t stream) {
  switch (p.tile) {
    case kTile256x256: return launch_shape<256, 256, 2, 4, ENGINE, false, 1>(t, p.splits, num_cus, stream);
    case kTile256x128: return launch_shape<256, 128, 4, 2, ENGINE, ENGINE == 1, 1>(t, p.splits, num_cus, stream);
    case kTile128x128: return launch_shape<128, 128, 2, 2, ENGINE, false, 1>(t, p.splits, num_cus, stream);
    default: return launch_shape<128, 128, 2, 2, ENGINE, false, 2>(t, p.splits, num_cus, stream);
  }
}

}  // namespace

hipError_t launch_linear_tile(const LinearActArgs& g, const LinearPlan& p, int accum, float* part, int num_cus,
                              hipStream_t stream) {
  TileArgs t{};
  t.a = g;
  const int64_t stages = (g.K + KS - 1) / KS;
  t.split_stages = (int)((stages + p.splits - 1) / p.splits);
  t.part = p.splits > 1 ? part : nullptr;
  if (accum == 1) return launch_engine<1>(t, p, num_cus, stream);
  return launch_engine<0>(t, p, num_cus, stream);
}

}  // namespace fp8mot
