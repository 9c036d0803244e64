// FP8 x FP8 GEMM on gfx950 matrix cores with the per-tensor scale_a * scale_b
// epilogue to BF16, FP8 or FP32.
//
// Pull request "Load static FP8 Cosmos3 Nano/Super checkpoints without
// re-quantizing them", "Description" and commit messages: every projection
// keeps its own FP8 weight and its own weight scale, and each Linear applies
// its own scale in the GEMM epilogue.  The model card's fake-quant setup
// fixes what is computed: y = s_x * s_w * sum_k dec(qx[m,k]) * dec(qw[n,k]).
//
// Two accumulation engines share the tiling:
//
//  ENGINE_F16 (FP8MOT_ACC_EXACT): the FP8 codes are staged through LDS as
//    bytes and decoded exactly to F16 right after each fragment read (the
//    gfx950 packed FP8 -> F16 conversion at scale 1.0: every E4M3 value is an
//    F16 value, NaN stays NaN), then multiplied with v_mfma_f32_32x32x16_f16,
//    whose products are summed to FP32 precision.
//
//  ENGINE_FP8 (FP8MOT_ACC_FP8_MFMA): the codes go to LDS as bytes and are
//    multiplied with v_mfma_f32_32x32x64_f8f6f4 at twice the rate.  On gfx950
//    every FP8 MFMA sums each group of 8 consecutive K products on a grid 13
//    bits below the group's largest product (truncating smaller products
//    toward zero) before adding the group into the FP32 accumulator, so its
//    error can reach ~1e-4 of sum|terms| where a group mixes magnitudes.
//
// Tiling (both engines):
//  * a workgroup computes a BM x BN tile with WM x WN waves, each wave a
//    (BM/WM) x (BN/WN) sub-tile of 32x32 MFMA blocks;
//  * operands are K-contiguous ([M,K] and [N,K]); a stage holds 128 K of the
//    tile's A and B rows (128 LDS bytes per row), two stages live in LDS
//    (three or four in the deep-prefetch variants) and the buffer unit copies
//    them from memory straight into LDS ahead of the MFMAs, one barrier per
//    stage (details below);
//  * the 16-byte chunk c of LDS row r lives at chunk c ^ ((r >> 1) & 7): the
//    LDS serves a 128-bit access 16 lanes at a time across 64 four-byte
//    banks (256 bytes = two rows), and 16 consecutive rows of one logical
//    chunk then cover all 16 distinct 16-byte bank groups;
//  * an MFMA operand fragment is read per lane as whole 16-byte chunks: lane
//    l takes row l % 32 and K positions (l / 32) * w .. + w of the MFMA's K
//    step (w = 8 for F16, 32 for FP8); A and B use the same assignment, so the
//    dot product does not depend on the instruction's internal K order;
//  * accumulator register v of lane l holds row 8*(v/4) + 4*(l/32) + v%4,
//    column l % 32 of its 32x32 block;
//  * tiles are ordered so that the workgroups dealt to one XCD (blocks go to
//    the 8 XCDs round-robin) walk a band of neighbouring tiles and share A and
//    B rows in that XCD's L2;
//  * the epilogue scales the accumulators, converts them (BF16, or SwiGLU to
//    FP8 in the fused gate/up kernel), transposes 4x4 blocks inside lane
//    quads so each lane owns consecutive columns of one row, and stores them
//    straight to memory.
//
// On MI355X the matrix cores slow down with the data they multiply (random
// codes draw more power than zeros, and the clock drops), so kernel times
// depend on the operands; the kernels keep every instruction that is not an
// MFMA to a minimum.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <atomic>
#include <type_traits>

#include "device_common.h"
#include "kernels.h"

namespace fp8mot {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kNumXcd = 8;      // MI355X: 8 XCDs
constexpr int kGroupM = 8;      // tile rows per band

// Workgroup id -> (tile_m, tile_n).
__device__ __forceinline__ void tile_of(int bid, int tiles_m, int tiles_n,
                                        int& tm, int& tn) {
  const int nb = tiles_m * tiles_n;
  // undo the round-robin XCD dealing: blocks of one XCD become contiguous
  const int xcd = bid % kNumXcd, idx = bid / kNumXcd;
  const int q = nb / kNumXcd, r = nb % kNumXcd;
  const int t = (xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q) + idx;
  // banded order: kGroupM tile rows advance together along N
  const int per_band = kGroupM * tiles_n;
  const int band = t / per_band;
  const int first_m = band * kGroupM;
  const int rows = min(tiles_m - first_m, kGroupM);
  const int in_band = t - band * per_band;
  tm = first_m + in_band % rows;
  tn = in_band / rows;
}

// Two E4M3 codes (the low or high half of a dword) -> two F16 values with the gfx950
// packed conversion at scale 1.0.  Every finite E4M3 value is exactly an F16
// value (max 448, smallest subnormal 2^-9 is an F16 normal) and the NaN codes
// become an F16 NaN; all 256 codes were checked on the hardware.
template <bool HIGH>
__device__ __forceinline__ int e4m3x2_to_f16x2(uint32_t x) {
  return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, 1.0f, HIGH));
}

// Buffer resource over [base, base + bytes): loads beyond it return 0 and
// stores beyond it are dropped, which is how every bound below is enforced
// without a branch.  The third-dword value is the standard gfx9 raw-buffer
// configuration.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base,
                                                           int64_t bytes) {
  const int n = bytes > 0x7FFFFFF0LL ? 0x7FFFFFF0 : (int)bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n,
                                           0x00020000);
}

constexpr int kOOB = 0x7FFFFFF0;  // a byte offset past every buffer

// The same raw-buffer descriptor as four dwords (base address, stride 0,
// size in bytes, the configuration dword) for the inline-assembly copy below.
__device__ __forceinline__ v4i make_rsrc_words(const void* base, int64_t bytes) {
  const int n = bytes > 0x7FFFFFF0LL ? 0x7FFFFFF0 : (int)bytes;
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return (v4i){(int)(uint32_t)a, (int)(uint32_t)((a >> 32) & 0xFFFF), n, 0x00020000};
}

// One wave-wide 16-byte-per-lane copy from a buffer straight into LDS
// (buffer_load_dwordx4 ... lds): lane i's bytes land at lds_addr + 16 * i,
// out-of-range lanes write zeros.  Written as assembly so that the compiler,
// which cannot tell which stage buffer a copy writes, does not make every
// LDS read wait for every copy; the kernel waits for its copies itself
// (s_waitcnt vmcnt) before the barrier that publishes a stage.  M0 holds the
// LDS address; one wait state separates its write from the copy.  The
// memory address is the descriptor's base + soff (one value for the wave)
// + voff (per lane).
__device__ __forceinline__ void copy_to_lds(v4i rsrc, uint32_t lds_addr, int voff, int soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
      : "memory", "m0");
}

typedef unsigned v2u __attribute__((ext_vector_type(2)));

// Lane t of a quad holds byte e = row e of column t; afterwards it holds
// byte e = column e of row t (a 4x4 byte transpose across the quad).
__device__ __forceinline__ uint32_t quad_transpose_bytes(uint32_t x, int t) {
  // exchange 16-bit halves with lane t ^ 2, then bytes with lane t ^ 1
  const uint32_t p = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true);   // quad_perm [2,3,0,1]
  const uint32_t z = __builtin_amdgcn_perm(p, x, t < 2 ? 0x05040100u : 0x03020706u);
  const uint32_t r = (uint32_t)__builtin_amdgcn_mov_dpp((int)z, 0xB1, 0xF, 0xF, true);   // quad_perm [1,0,3,2]
  return __builtin_amdgcn_perm(r, z, (t & 1) ? 0x03070105u : 0x06020400u);
}

// Lane t of a quad holds four 16-bit values of column t, rows 0..3, as
// a = row0 | row1 << 16 and b = row2 | row3 << 16; afterwards d0, d1 hold
// row t, columns 0..3 (d0 = col0 | col1 << 16, d1 = col2 | col3 << 16).
__device__ __forceinline__ void quad_transpose_halves(uint32_t a, uint32_t b, int t,
                                                      uint32_t& d0, uint32_t& d1) {
  // lanes 0, 1 keep rows 0-1 and take those of columns t + 2; lanes 2, 3
  // keep rows 2-3 and take those of columns t - 2
  const uint32_t send = t < 2 ? b : a;
  const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)send, 0x4E, 0xF, 0xF, true);
  const uint32_t u = t < 2 ? a : got;    // rows ra, ra+1 of column t & 1
  const uint32_t v = t < 2 ? got : b;    // rows ra, ra+1 of column (t & 1) + 2
  // even lanes keep row ra and send row ra+1; odd lanes the reverse
  const uint32_t s2 = (t & 1) ? __builtin_amdgcn_perm(v, u, 0x05040100u)    // u.lo | v.lo << 16
                              : __builtin_amdgcn_perm(v, u, 0x07060302u);   // u.hi | v.hi << 16
  const uint32_t r2 = (uint32_t)__builtin_amdgcn_mov_dpp((int)s2, 0xB1, 0xF, 0xF, true);
  if (t & 1) {
    d0 = __builtin_amdgcn_perm(u, r2, 0x07060100u);   // r2.lo | u.hi << 16
    d1 = __builtin_amdgcn_perm(v, r2, 0x07060302u);   // r2.hi | v.hi << 16
  } else {
    d0 = __builtin_amdgcn_perm(r2, u, 0x05040100u);   // u.lo | r2.lo << 16
    d1 = __builtin_amdgcn_perm(r2, v, 0x07060100u);   // v.lo | r2.hi << 16
  }
}

// Operand staging: a stage covers KS = 128 of K.  Its LDS rows hold the 128
// FP8 codes of one A or B row, and NB stages live in LDS at once (two, or
// with DEEP as many as fit, up to four): the NB A stages first, then the NB
// B stages, so that a fragment read is a per-lane base plus an offset that
// fits the LDS instruction's immediate.  The
// global -> LDS copy is done by the buffer unit itself (buffer_load_dwordx4
// with the LDS flag): one wave-wide instruction fills 1 KB of a stage (8
// rows) -- lane i's 16 bytes land at byte 16*i -- with no registers in
// between and no wait in the wave.  Loads that fall outside a buffer resource
// write zeros, which pads ragged M, N and K.  The copies of stage s + NB go
// out as soon as every wave has finished reading stage s, spread between the
// MFMAs of that step.  Measured on MI355X: whole 128-byte row segments per
// copy move L2-resident data ~1.8x faster than 64-byte ones (the L2 serves a
// request per segment), which outweighs the deeper prefetch that 64-K stages
// allow in the same LDS; staging through registers and ds_write was no
// faster.
constexpr int KS = 128;           // K per stage
constexpr int CH = KS / 16;       // 16-byte chunks per LDS row
constexpr int RW = 256 / KS;      // LDS rows per 256-byte bank window
constexpr int RPI = 1024 / KS;    // LDS rows filled by one wave-wide copy

// Physical chunk of logical chunk c in LDS row r.  The LDS serves a 128-bit
// access 16 lanes at a time across 64 four-byte banks (256 bytes = RW rows);
// the 16 lanes of a fragment read touch 16 consecutive rows at one logical
// chunk, and the XOR with the row's window index spreads them over all 16
// distinct 16-byte bank groups.
__device__ __forceinline__ int swz(int r, int c) { return c ^ ((r / RW) & (CH - 1)); }

struct GemmArgs {
  const uint8_t* A;   // [M, K]
  const uint8_t* B;   // [N, K]   (fused: the gate weight)
  const uint8_t* B2;  // fused: the up weight [N, K]
  void* C;            // [M, N]   (fused: the FP8 SwiGLU output)
  int M, N, K;
  const float* sx;    // (OUT 3, 4: per-row scales [M])
  const float* sw;    // (fused: gate weight scale; OUT 3, 4: per-channel scales [N])
  const float* sw2;   // fused: up weight scale
  const float* sy;    // FP8 output scale (fused: the down projection's input scale)
  int tiles_m, tiles_n;
  int ldc;            // row stride of C in elements (>= N; N for a contiguous C)
  // Grouped launch (groups > 1): up to three projections of the same A, each
  // with its own B, C, weight scale and N (contiguous C), in one grid; the
  // tile columns of group p follow those of groups 0 .. p-1.
  int groups;
  const uint8_t* gB[3];
  void* gC[3];
  const float* gsw[3];
  int gN[3];
  int gtiles_n[3];
};

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// OUT: 0 BF16, 1 FP8, 2 FP32 with per-tensor scales; 3 BF16, 4 FP32 with a
// scale per row of A and per row of B (per-token / per-channel).  FUSED: gate and up GEMMs of a gated MLP in one
// tile (BN = 256 = 128 gate rows + 128 up rows of the same output columns)
// whose epilogue applies SwiGLU and writes FP8, bit for bit what the separate
// BF16 GEMMs followed by silu_mul_2in_fp8 produce.  KSPL = 2: two groups of
// WM x WN waves share the tile, group 0 taking the even 128-K stages and
// group 1 the odd ones, each with its own stages in LDS; at the end group 1
// hands its sums to group 0 through LDS, which adds them (even + odd) and
// runs the epilogue.  That doubles the waves per CU (and the bytes in flight)
// when there are too few tiles to give every CU more than one.
template <int BM, int BN, int WM, int WN, int OUT, int ENGINE, bool FUSED, bool DEEP = false,
          int KSPL = 1>
__global__ __launch_bounds__(WM* WN * 64 * KSPL, 1) void gemm_kernel(GemmArgs g) {
  const int M = g.M, K = g.K;
  constexpr int NW = WM * WN;                   // waves per K group
  constexpr int WTM = BM / WM, WTN = BN / WN;   // wave tile
  constexpr int FM = WTM / 32, FN = WTN / 32;   // 32x32 blocks per wave
  constexpr int STAGE = (BM + BN) * KS;
  // stages resident in LDS per K group: two, or with DEEP as many as the
  // 160 KB hold, up to four (two for 256x256 tiles, three for 256x128, four
  // for 128x128; three for 128x64 with the K split's two groups)
  constexpr int NB = !DEEP ? 2 : (160 * 1024) / (KSPL * STAGE) < 4 ? (160 * 1024) / (KSPL * STAGE) : 4;
  constexpr int A_INS = BM / RPI, INS = (BM + BN) / RPI;   // wave-wide copies per stage
  constexpr int LPW = INS / NW;                            // ... per wave
  static_assert(LPW * NW == INS, "tile rows / waves");
  static_assert(!FUSED || (BN == 256 && FN % 2 == 0), "fused tiles pair gate/up blocks");
  static_assert(KSPL == 1 || (KSPL == 2 && !FUSED), "K split: plain tiles");
  static_assert(KSPL * NB * STAGE <= 160 * 1024, "stages fit the 160 KB LDS of a CU");
  static_assert(KSPL == 1 || NW * FM * FN * 16 * 64 * 4 <= KSPL * NB * STAGE,
                "the K groups' sums fit the stage buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[KSPL * NB * STAGE];

  const int tid = threadIdx.x, lane0 = tid & 63;
  const int wave_id = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = KSPL == 1 ? 0 : wave_id / NW;    // K group
  const int wave = wave_id - kg * NW;             // wave within its K group
  const int wm = wave / WN, wn = wave % WN;
  // LDS of K group kg: its NB A stages, then its NB B stages, so that every
  // fragment read is a per-lane base plus an offset that fits the LDS
  // instruction's 16-bit immediate
  constexpr int A_STAGE = BM * KS, B_STAGE = BN * KS;
  auto a_buf = [&](int b) -> uint8_t* { return smem + kg * NB * STAGE + b * A_STAGE; };
  auto b_buf = [&](int b) -> uint8_t* { return smem + kg * NB * STAGE + NB * A_STAGE + b * B_STAGE; };
  // K group kg's local stage t is the tile's stage t * KSPL + kg
  auto gstage = [&](int t) { return t * KSPL + kg; };
  // A tile's place in the grid: its output rows from m0 and columns from n0
  // (fused: 128 of each of G and U), and -- in a grouped launch, which walks
  // the groups' tile columns -- its projection's B, C, weight scale and N.
  struct TileInfo {
    int m0, n0, N, ldc;
    const uint8_t* B;
    void* C;
    const float* sw;
  };
  auto tile_info = [&](int tile) -> TileInfo {
    int tm, tn;
    tile_of(tile, g.tiles_m, g.tiles_n, tm, tn);
    TileInfo t{0, 0, g.N, g.ldc, g.B, g.C, g.sw};
    if (g.groups > 1) {
      int p = 0;
      while (p + 1 < g.groups && tn >= g.gtiles_n[p]) {
        tn -= g.gtiles_n[p];
        ++p;
      }
      t.B = g.gB[p];
      t.C = g.gC[p];
      t.sw = g.gsw[p];
      t.N = g.gN[p];
      t.ldc = t.N;
    }
    t.m0 = tm * BM;
    t.n0 = tn * (FUSED ? BN / 2 : BN);
    return t;
  };
  // Operand windows of a tile (buffer resources starting at its first A and
  // B rows): rows past M (N) lie outside them and read as zeros.
  struct Windows {
    v4i a, b, b2;
  };
  auto windows = [&](const TileInfo& t) -> Windows {
    Windows w;
    w.a = make_rsrc_words(g.A + (int64_t)t.m0 * K, (int64_t)(M - t.m0) * K);
    w.b = make_rsrc_words(t.B + (int64_t)t.n0 * K, (int64_t)(t.N - t.n0) * K);
    w.b2 = FUSED ? make_rsrc_words(g.B2 + (int64_t)t.n0 * K, (int64_t)(t.N - t.n0) * K) : w.b;
    return w;
  };

  // Copy q (= wave * LPW + i) of a stage fills LDS rows q*RPI .. q*RPI+RPI-1
  // (A rows, then B rows); lane l brings row q*RPI + l/CH, physical chunk
  // l % CH, i.e. logical chunk swz(row, l % CH) of the row's 64 K.  Fused:
  // B's LDS rows come in 32-row blocks alternating gate / up, so that a
  // wave's 32x32 blocks j (gate) and j + 1 (up) cover the same columns.
  // Rows past M (N) get an offset past every window.
  auto copy_offsets = [&](const TileInfo& t, int* goff, int* gkc) {
#pragma unroll
    for (int i = 0; i < LPW; ++i) {
      const int q = wave * LPW + i;
      const int lr = (q < A_INS ? q : q - A_INS) * RPI + lane0 / CH;   // row in the A or B region
      const int c = swz(lr, lane0 % CH);
      int grow, lim;
      if (q < A_INS) {
        grow = lr;
        lim = M - t.m0;
      } else {
        grow = FUSED ? (lr >> 6) * 32 + (lr & 31) : lr;
        lim = t.N - t.n0;
      }
      goff[i] = grow < lim ? grow * K + c * 16 : kOOB;
      gkc[i] = c * 16;
    }
  };
  // Copy i of this wave for stage s into buffer b.  When K is a multiple of
  // the stage (KFULL), every stage lies wholly inside K or wholly past it and
  // a copy needs no per-lane arithmetic: the lane's offset within the first
  // stage goes in as is and the stage's column offset k0 as the wave's scalar
  // offset, so a row inside the window reads row * K + k0 + chunk, inside the
  // window, and a row past it keeps kOOB, past every window however the
  // range check treats the scalar offset (kOOB + k0 stays below 2^32); a
  // stage past the end of K reads through an empty descriptor, so nothing is
  // read and zeros land in LDS.  Otherwise each chunk is checked against K.
  auto issue_copy = [&](const Windows& w, const int* goff, const int* gkc, int b, int s, int i,
                        auto kfull) {
    const int k0 = s * KS;
    const int q = wave * LPW + i;
    const v4i rs = q < A_INS ? w.a : ((FUSED && (((q - A_INS) * RPI) & 32)) ? w.b2 : w.b);
    const uint32_t dst = (uint32_t)reinterpret_cast<uintptr_t>(
        (lds_ptr_t)(q < A_INS ? a_buf(b) + q * 1024 : b_buf(b) + (q - A_INS) * 1024));
    if constexpr (decltype(kfull)::value) {
      copy_to_lds(k0 < K ? rs : (v4i){0, 0, 0, 0x00020000}, dst, goff[i], k0);
    } else {
      const int off = (goff[i] != kOOB && k0 + gkc[i] < K) ? goff[i] + k0 : kOOB;
      copy_to_lds(rs, dst, off, 0);
    }
  };
  auto issue_stage = [&](const Windows& w, const int* goff, const int* gkc, int b, int s,
                         auto kfull) {
#pragma unroll
    for (int i = 0; i < LPW; ++i) issue_copy(w, goff, gkc, b, s, i, kfull);
  };
  // local stages per K group (group 1 of an odd count runs one past the end
  // of K, on zeros, so that both groups meet the same barriers)
  const int KT = ((K + KS - 1) / KS + KSPL - 1) / KSPL;
  const int ntiles = g.tiles_m * g.tiles_n;

  // Persistent loop: a workgroup takes tiles blockIdx.x, + gridDim.x, ...
  // (gridDim.x is a multiple of the 8 XCDs, so every tile it takes belongs
  // to its own XCD's band).  The first NB stages of the next tile are copied
  // into LDS after this tile's main loop and before its epilogue, which then
  // runs while they are on their way.  A launch with one tile per workgroup
  // runs the loop once (K-split launches always do).
  // Exact-engine tiles only: the FP8 engine's loop keeps more registers live
  // and would spill in a tile loop, so its workgroups take one tile each.
  constexpr bool PERSIST = ENGINE == 0 && KSPL == 1;
  // The tile loop, compiled twice: for K a multiple of the stage (copies
  // without per-lane arithmetic) and for any other K.  The choice is made
  // once, here: a branch inside the loop would make the register allocator
  // spill.
  auto tiles_loop = [&](auto kfull) {
  bool staged = false;
  for (int tile = blockIdx.x, iter = 0; PERSIST ? tile < ntiles : iter < 1;
       tile += gridDim.x, ++iter) {
  // the lane index, opaque to the compiler for each tile: the per-lane LDS
  // fragment addresses and epilogue indices derived from it are formed per
  // tile instead of being hoisted out of this loop and kept live across the
  // epilogue, which needs those registers
  int lane = lane0;
  if constexpr (PERSIST) asm volatile("" : "+v"(lane));
  const TileInfo ti = tile_info(tile);
  const Windows win = windows(ti);
  int goff[LPW], gkc[LPW];
  copy_offsets(ti, goff, gkc);
  const int m0 = ti.m0, n0 = ti.n0, N = ti.N, ldc = ti.ldc;
  const float* gsw = ti.sw;
  void* gCp = ti.C;
  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // Per-lane LDS bases of the chunks a lane reads, one per chunk slot k of a
  // stage (F16 engine: step k reads logical chunk 2k + lane/32; FP8 engine:
  // step k/2 reads chunks 4(k/2) + 2(lane/32) and the next one), for the
  // lane's row in its wave's first A and B block of stage 0.  A row's
  // swizzle depends only on the row's bits 1..3, which blocks 32 rows apart
  // share, so block i of A (j of B) in stage b is base + b * A_STAGE +
  // i * 32 * KS (+ b * B_STAGE + j * 32 * KS): an immediate offset.  Opaque
  // to the compiler, so that it keeps these sums instead of re-forming them.
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
  auto chunk_at = [&](int base, int imm) -> v4i {
    return *reinterpret_cast<const v4i*>(smem + base + imm);
  };
  // K-steps per stage.  FP8 engine: one step of 64 K, a lane reading two
  // chunks (32 codes) per operand.  F16 engine: two steps of 32 K, a lane
  // reading one chunk (16 codes) per operand, converting it to two F16
  // operands and issuing two 32x32x16 MFMAs -- bytes 0..7 of every lane's
  // chunk feed the first, bytes 8..15 the second, for A and B alike.
  constexpr int NSTEP = ENGINE == 0 ? KS / 32 : KS / 64;
  // operand fragments (raw codes), double-buffered: K-step t of the whole
  // loop uses slot t & 1
  typedef typename std::conditional<ENGINE == 0, v4i, v8i>::type frag_t;
  frag_t fa[2][FM], fb[2][FN];
  auto rd = [&](int b, int st, int slot) {   // fragments of step st of the stage in buffer b
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
    // keep the reads ahead of the MFMAs that follow, so that their latency
    // is covered by this step's matrix work
    __builtin_amdgcn_sched_barrier(0);
  };
  // MFMAs of one K-step.  With copies, the copies of stage cs into buffer cb
  // are issued one after each 32-row block of A (the rest after the last),
  // so that the address unit is fed steadily instead of every wave queueing
  // its copies at once.
  constexpr int CPR = (LPW + FM - 1) / FM;   // copies issued after each block row
  auto mf = [&](int slot, auto copies, int cb, int cs) {
    constexpr bool kCopies = decltype(copies)::value;
    if constexpr (ENGINE == 0) {
      f16x8 a0[FM], a1[FM], b0[FN], b1[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const v4i v = fa[slot][i];
        a0[i] = __builtin_bit_cast(f16x8, (v4i){e4m3x2_to_f16x2<false>(v[0]), e4m3x2_to_f16x2<true>(v[0]),
                                                e4m3x2_to_f16x2<false>(v[1]), e4m3x2_to_f16x2<true>(v[1])});
        a1[i] = __builtin_bit_cast(f16x8, (v4i){e4m3x2_to_f16x2<false>(v[2]), e4m3x2_to_f16x2<true>(v[2]),
                                                e4m3x2_to_f16x2<false>(v[3]), e4m3x2_to_f16x2<true>(v[3])});
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const v4i v = fb[slot][j];
        b0[j] = __builtin_bit_cast(f16x8, (v4i){e4m3x2_to_f16x2<false>(v[0]), e4m3x2_to_f16x2<true>(v[0]),
                                                e4m3x2_to_f16x2<false>(v[1]), e4m3x2_to_f16x2<true>(v[1])});
        b1[j] = __builtin_bit_cast(f16x8, (v4i){e4m3x2_to_f16x2<false>(v[2]), e4m3x2_to_f16x2<true>(v[2]),
                                                e4m3x2_to_f16x2<false>(v[3]), e4m3x2_to_f16x2<true>(v[3])});
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a0[i], b0[j], acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(a1[i], b1[j], acc[i][j], 0, 0, 0);
        }
        if constexpr (kCopies) {
#pragma unroll
          for (int c = 0; c < CPR; ++c)
            if (i * CPR + c < LPW) issue_copy(win, goff, gkc, cb, cs, i * CPR + c, kfull);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fa[slot][i], fb[slot][j], acc[i][j], 0, 0, 0, 0, 0, 0);
        if constexpr (kCopies) {
#pragma unroll
          for (int c = 0; c < CPR; ++c)
            if (i * CPR + c < LPW) issue_copy(win, goff, gkc, cb, cs, i * CPR + c, kfull);
        }
      }
    }

  };
  // wait until at most n of this wave's stage copies are still in flight
  // (s_waitcnt vmcnt(n), expcnt and lgkmcnt left alone: gfx9 encoding)
  auto wait_copies = [&](int n) {
    if (NB > 4 && n >= 4 * LPW) __builtin_amdgcn_s_waitcnt(0x0F70 | ((4 * LPW) & 15) | (((4 * LPW) >> 4) << 14));
    else if (NB > 3 && n >= 3 * LPW) __builtin_amdgcn_s_waitcnt(0x0F70 | ((3 * LPW) & 15) | (((3 * LPW) >> 4) << 14));
    else if (NB > 2 && n >= 2 * LPW) __builtin_amdgcn_s_waitcnt(0x0F70 | ((2 * LPW) & 15) | (((2 * LPW) >> 4) << 14));
    else if (n >= LPW) __builtin_amdgcn_s_waitcnt(0x0F70 | (LPW & 15) | ((LPW >> 4) << 14));
    else __builtin_amdgcn_s_waitcnt(0x0F70);
  };
  static_assert(NB >= 2 && NB <= 5 && (NB - 1) * LPW < 64, "wait_copies covers up to four stages in flight");

  // Pipeline, per stage s (buffer s % NB), K-steps t = 0 .. NSTEP-1:
  //  * before the MFMAs of step t, the fragments of the next step are read
  //    into the other register slot;
  //  * at the last step, the next stage must be ready: wait for this wave's
  //    copies of stage s + 1 and for its own fragment reads of stage s,
  //    barrier (every wave's copies of s + 1 have landed and nobody reads
  //    stage s any more), issue the copies of stage s + NB into the buffer
  //    just freed, then read the first fragments of stage s + 1.
  // The MFMAs of a step are issued after these reads, so the barrier wait
  // overlaps the matrix pipe still working through the previous step.
  // have the epilogue's kernel arguments in registers before the loop, so no
  // scalar load is still pending inside it (that would turn every LDS wait
  // there into a wait for all LDS reads)
  asm volatile("" ::"s"(g.sx), "s"(gsw), "s"(g.sw2), "s"(g.sy), "s"(gCp));
  if (!staged) {
#pragma unroll
    for (int u = 0; u < NB; ++u)
      if (u < KT) issue_stage(win, goff, gkc, u, gstage(u), kfull);
  }
  if (KT > 0) {
    // staged: the previous epilogue's stores were issued after these copies
    // and count in the same counter, so wait for everything
    if (staged) __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
    else wait_copies(LPW * (min(NB, KT) - 1));
    __syncthreads();
    rd(0, 0, 0);
  }
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
            // The copies of stage s + NB go into the buffer just freed.  Past
            // the end of K they touch no memory and write zeros, into a
            // buffer nobody reads again -- at the last stage, where no
            // barrier has freed this buffer, into the next one instead (the
            // wait after the loop drains them before any buffer is refilled).
            mf(slot, std::true_type{}, s + 1 < KT ? u : (u + 1) % NB, gstage(s + NB));
          }
        }
      }
    }
  }
  // no copy into LDS may still be on its way when the workgroup ends or
  // the buffers are refilled
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)

  if constexpr (KSPL == 2) {
    // Group 1's sums go through LDS to the wave of group 0 that holds the same
    // blocks: 16-byte pieces, lane-major (conflict-free), over the stage
    // buffers, which nobody reads or fills any more after this barrier.
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

  // The next tile's first stages: every wave has read this tile's last
  // fragments (its MFMAs are issued), so after one barrier the buffers are free.
  staged = false;
  if (PERSIST && tile + (int)gridDim.x < ntiles) {
    __syncthreads();
    const TileInfo nt = tile_info(tile + gridDim.x);
    const Windows nw = windows(nt);
    int ngoff[LPW], ngkc[LPW];
    copy_offsets(nt, ngoff, ngkc);
#pragma unroll
    for (int u = 0; u < NB; ++u)
      if (u < KT) issue_stage(nw, ngoff, ngkc, u, gstage(u), kfull);
    staged = true;
  }

  // ---- epilogue: y = fp32(acc * alpha), then the output format ----
  // Accumulator register v of 32x32 block (i, j) holds row
  // i*32 + 8*(v/4) + 4*(lane/32) + v%4, column j*32 + lane%32: the four
  // registers v = 4q .. 4q+3 are four consecutive rows of one column, and the
  // four lanes of a quad hold four consecutive columns.  A 4x4 transpose
  // inside the quad (two DPP exchanges) turns that into one row-piece of four
  // consecutive columns per lane, stored straight to global memory.
  // Per-row scales (OUT 3, 4): alpha[m, n] = fp32(s_x[m] * s_w[n]), formed
  // per output exactly as the per-tensor alpha is; the four consecutive rows
  // of a register group take one 16-byte load of s_x, each column one s_w.
  constexpr bool ROWWISE = OUT >= 3;
  const float alpha = ROWWISE ? 0.0f : __fmul_rn(*g.sx, *gsw);
  const __amdgpu_buffer_rsrc_t rsx = make_rsrc(g.sx + (ROWWISE ? m0 : 0), ROWWISE ? (int64_t)(M - m0) * 4 : 0);
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(gsw + (ROWWISE ? n0 : 0), ROWWISE ? (int64_t)(N - n0) * 4 : 0);
  auto row_scales4 = [&](int row) -> v4i {   // s_x of tile rows row .. row + 3 (row % 4 == 0)
    return __builtin_amdgcn_raw_buffer_load_b128(rsx, row * 4, 0, 0);
  };
  float swc[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j)
    swc[j] = ROWWISE ? __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                           rsw, (wn * WTN + (lane & 31) + j * 32) * 4, 0, 0))
                     : 0.0f;
  void* __restrict__ C = gCp;
  constexpr int ESZ = (OUT == 0 || OUT == 3) ? 2 : (OUT == 1 ? 1 : 4);
  const __amdgpu_buffer_rsrc_t rc_rs =
      make_rsrc(static_cast<uint8_t*>(C) + ((int64_t)m0 * ldc) * ESZ, (int64_t)(M - m0) * ldc * ESZ);
  const int col_l = wn * WTN + (lane & 31);          // + j*32
  const int row_l = wm * WTM + (lane >> 5) * 4;       // + i*32 + 8*(v/4) + v%4
  const int qt = lane & 3;                            // lane's place in its quad

  if constexpr (FUSED) {
    // G and U of one output element sit in blocks j (gate) and j + 1 (up) of
    // the same lane and register: round each to BF16 exactly as the BF16
    // epilogue does, apply SwiGLU exactly as silu_mul_2in_fp8 does, encode
    // four rows at a time, transpose the bytes in the quad and store one
    // dword (a row's four consecutive columns) per lane.
    const float alpha_u = __fmul_rn(*g.sx, *g.sw2);
    const float rs = 1.0f / *g.sy;
    const __amdgpu_buffer_rsrc_t rq_rs =
        make_rsrc(static_cast<uint8_t*>(C) + (int64_t)m0 * ldc, (int64_t)(M - m0) * ldc);
    const int col_q = n0 + (wn * WTN) / 2 + ((lane & 31) & ~3);   // + p*32
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int p = 0; p < FN / 2; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int v = 4 * q + e;
            const uint32_t gu = bf16x2_rne(__fmul_rn(acc[i][2 * p][v], alpha),
                                           __fmul_rn(acc[i][2 * p + 1][v], alpha_u));
            h[e] = __fmul_rn(silu_mul(__uint_as_float(gu << 16), __uint_as_float(gu & 0xFFFF0000u)), rs);
          }
          const uint32_t w = quad_transpose_bytes(e4m3_pack4(h[0], h[1], h[2], h[3]), qt);
          const int row = row_l + i * 32 + q * 8 + qt;       // row within tile
          const int col = col_q + p * 32;
          const int off = (m0 + row < M && col < N) ? row * ldc + col : kOOB;
          __builtin_amdgcn_raw_buffer_store_b32(w, rq_rs, off, 0, 0);
        }
  } else if constexpr (OUT == 0 || OUT == 3) {
    // BF16: four rows of a column -> two packed dwords, transposed in the
    // quad so that each lane stores four consecutive columns of one row
    // (8 bytes).  Rows whose width is not a multiple of 4 take 2-byte stores.
    const bool vec_ok = (N % 4) == 0 && (ldc % 4) == 0;
    const int col_q = n0 + wn * WTN + ((lane & 31) & ~3);   // + j*32
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v4i sxr = {0, 0, 0, 0};
        if constexpr (ROWWISE) sxr = row_scales4(row_l + i * 32 + q * 8);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          float al[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            al[e] = ROWWISE ? __fmul_rn(__int_as_float(sxr[e]), swc[j]) : alpha;
          const uint32_t a = bf16x2_rne(__fmul_rn(acc[i][j][4 * q + 0], al[0]), __fmul_rn(acc[i][j][4 * q + 1], al[1]));
          const uint32_t b = bf16x2_rne(__fmul_rn(acc[i][j][4 * q + 2], al[2]), __fmul_rn(acc[i][j][4 * q + 3], al[3]));
          uint32_t d0, d1;
          quad_transpose_halves(a, b, qt, d0, d1);
          const int row = row_l + i * 32 + q * 8 + qt;
          const int col = col_q + j * 32;
          if (vec_ok) {
            const int off = (m0 + row < M && col < N) ? (row * ldc + col) * 2 : kOOB;
            __builtin_amdgcn_raw_buffer_store_b64((v2u){d0, d1}, rc_rs, off, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int off = (m0 + row < M && col + e < N) ? (row * ldc + col + e) * 2 : kOOB;
              const uint32_t d = e < 2 ? d0 : d1;
              __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(d >> ((e & 1) * 16)), rc_rs, off, 0, 0);
            }
          }
        }
      }
  } else if constexpr (OUT == 1) {
    // FP8: the four rows of a column are encoded into one dword, transposed
    // in the quad so that each lane stores four consecutive columns of one
    // row (4 bytes).  Rows whose width is not a multiple of 4 take byte
    // stores.
    const float sy = *g.sy;
    const bool vec_ok = (N % 4) == 0 && (ldc % 4) == 0;
    const int col_q = n0 + wn * WTN + ((lane & 31) & ~3);   // + j*32
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          float h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = __fmul_rn(acc[i][j][4 * q + e], alpha) / sy;   // IEEE division
          const uint32_t w = quad_transpose_bytes(e4m3_pack4(h[0], h[1], h[2], h[3]), qt);
          const int row = row_l + i * 32 + q * 8 + qt;
          const int col = col_q + j * 32;
          if (vec_ok) {
            const int off = (m0 + row < M && col < N) ? row * ldc + col : kOOB;
            __builtin_amdgcn_raw_buffer_store_b32(w, rc_rs, off, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int off = (m0 + row < M && col + e < N) ? row * ldc + col + e : kOOB;
              __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(w >> (8 * e)), rc_rs, off, 0, 0);
            }
          }
        }
  } else {
    // FP32 (per-tensor or per-row scales): one dword per element
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v4i sxr = {0, 0, 0, 0};
        if constexpr (ROWWISE) sxr = row_scales4(row_l + i * 32 + q * 8);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int col = col_l + j * 32;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int v = 4 * q + e;
            const int row = row_l + i * 32 + q * 8 + e;
            const bool ok = (m0 + row < M) && (n0 + col < N);
            const int off = ok ? (row * ldc + n0 + col) * ESZ : kOOB;
            const float al = ROWWISE ? __fmul_rn(__int_as_float(sxr[e]), swc[j]) : alpha;
            const float y = __fmul_rn(acc[i][j][v], al);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y), rc_rs, off, 0, 0);
          }
        }
      }
  }
  }  // tile loop
  };
  if (K % KS == 0)
    tiles_loop(std::true_type{});
  else
    tiles_loop(std::false_type{});
}

// Launches one GEMM kernel: one workgroup per tile, or -- for the exact
// engine when there are more tiles than the GPU holds at once -- as many
// workgroups as are resident (the kernel's occupancy per CU times the CUs, a
// multiple of the 8 XCDs), each walking its tiles with the next tile's first
// stages prefetched during the current one's epilogue.  K-split and
// FP8-engine launches keep one tile per workgroup.
template <int BM, int BN, int WM, int WN, int OUT, int ENGINE, bool FUSED, bool DEEP, int KSPL>
hipError_t launch_kernel(const GemmArgs& a, int num_cus, hipStream_t stream) {
  auto kern = gemm_kernel<BM, BN, WM, WN, OUT, ENGINE, FUSED, DEEP, KSPL>;
  constexpr int block = WM * WN * 64 * KSPL;
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  int64_t grid = tiles;
  if (ENGINE == 0 && KSPL == 1) {   // the kernels that walk several tiles
    static std::atomic<int> occupancy{0};
    int occ = occupancy.load(std::memory_order_relaxed);
    if (occ == 0) {
      if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, block, 0) != hipSuccess || occ < 1)
        occ = 1;
      occupancy.store(occ, std::memory_order_relaxed);
    }
    const int64_t resident = (int64_t)occ * num_cus;
    if (tiles > resident && resident >= kNumXcd) grid = resident - resident % kNumXcd;
  }
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(block), 0, stream, a);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int ENGINE, bool DEEP, int KSPL>
hipError_t launch_tiled(GemmArgs a, int out_kind, int num_cus, hipStream_t stream) {
  switch (out_kind) {
    case 0: return launch_kernel<BM, BN, WM, WN, 0, ENGINE, false, DEEP, KSPL>(a, num_cus, stream);
    case 1: return launch_kernel<BM, BN, WM, WN, 1, ENGINE, false, DEEP, KSPL>(a, num_cus, stream);
    case 3: return launch_kernel<BM, BN, WM, WN, 3, ENGINE, false, DEEP, KSPL>(a, num_cus, stream);
    case 4: return launch_kernel<BM, BN, WM, WN, 4, ENGINE, false, DEEP, KSPL>(a, num_cus, stream);
    default: return launch_kernel<BM, BN, WM, WN, 2, ENGINE, false, DEEP, KSPL>(a, num_cus, stream);
  }
}

// Tile counts of a launch with BM x BN tiles (a grouped launch adds up the
// groups' tile columns).
template <int BM, int BN>
void set_tiles(GemmArgs& a) {
  a.tiles_m = (a.M + BM - 1) / BM;
  if (a.groups > 1) {
    a.tiles_n = 0;
    for (int p = 0; p < a.groups; ++p) {
      a.gtiles_n[p] = (a.gN[p] + BN - 1) / BN;
      a.tiles_n += a.gtiles_n[p];
    }
  } else {
    a.tiles_n = (a.N + BN - 1) / BN;
  }
}

template <int BM, int WM, int WN, int ENGINE>
hipError_t launch_fused(GemmArgs a, int num_cus, hipStream_t stream) {
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + 127) / 128;
  return launch_kernel<BM, 256, WM, WN, 0, ENGINE, true, false, 1>(a, num_cus, stream);
}

int64_t tiles_of(int64_t M, int64_t N, int bm, int bn) {
  return ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
}

int forced_env(const char* name) {
  const char* e = getenv(name);
  return e ? atoi(e) : -1;
}

// Tile configuration per shape (MI355X, 256 CUs): the largest tile that
// still gives about one workgroup per CU.  Measured on the workload shapes:
// 256x256 tiles with 8 waves (two per SIMD) are fastest once there are
// ~0.7 tiles per CU; below that 256x128 (8 waves), then 128x128 and 128x64
// (4 waves; 512x4096x4096: 33.9 -> 25.8 us, 512x4096x12288: 72.7 -> 55.6 us
// with 128x64) keep the CUs busy.  Where 256x256 tiles are used, 192x256
// tiles (8 waves of 96x64, one workgroup per CU as well) replace them when
// they need no more rounds of one workgroup per CU: per FLOP they run 3-4%
// slower (whole rounds on both, 12288x4096x4096: 299 against 309-311 us), so
// they pay only where they fill a round that 256x256 tiles leave partly empty
// (split Q/K/V, 3072 x 3*4096 x 4096: 576 tiles of 256x256 are 2.25 per CU,
// 768 of 192x256 exactly 3; 274 -> 232 us, and 185.6 -> 163.9 us for 1536
// rows).  Needing one round more, they came out within -3% .. +1.5%
// (4608x12288x4096, 6144x12288x4096: a partial last round costs less than a
// full one), so 256x256 stays there.  FP8MOT_GEMM_CFG=<1|5|3|6|7> forces one
// configuration (tuning; 6 is 128x64, 7 is 192x256).
int pick_cfg(int64_t tiles_256x256, int64_t tiles_192x256, int64_t tiles_256x128,
             int64_t tiles_128x128, int num_cus) {
  static const int forced = forced_env("FP8MOT_GEMM_CFG");
  if (forced >= 0) return forced == 1 || forced == 5 || forced == 6 || forced == 7 ? forced : 3;
  const int64_t want = (int64_t)num_cus * 7 / 10;
  if (tiles_256x256 >= want) {
    const int64_t r256 = (tiles_256x256 + num_cus - 1) / num_cus;
    const int64_t r192 = (tiles_192x256 + num_cus - 1) / num_cus;
    return r192 <= r256 ? 7 : 1;
  }
  if (tiles_256x128 >= want) return 5;
  return tiles_128x128 >= want ? 3 : 6;
}

// Deep prefetch (three or four stages in LDS) pays for the FP8 engine, whose
// loop is short enough to wait on the copies; the F16 engine is bound by its
// own issue (decode + MFMA) and keeps two stages.  A 128x128 tile with four
// stages fills the CU's LDS, so it is used only when there is at most one
// tile per CU -- otherwise two-stage tiles run two to a CU.  A 128-row tile
// that has a CU to itself splits K over two wave groups instead (see
// gemm_splits_k).
template <int BM, int BN, int WM, int WN, int ENGINE>
hipError_t launch_cfg(GemmArgs a, int out_kind, int num_cus, hipStream_t stream, bool split) {
  set_tiles<BM, BN>(a);
  // (the FP8 engine never splits 128x64 tiles, and only the FP8 engine takes
  // deep prefetch without a split: the other combinations are not built)
  if constexpr (BM == 128 && !(ENGINE == 1 && BN == 64)) {
    // 128x64 tiles leave room for three stages per K group (measured on the
    // und tower's 512x4096x12288 down projection, whose copies the two-stage
    // loop waits on)
    if (split) return launch_tiled<BM, BN, WM, WN, ENGINE, BN == 64, 2>(a, out_kind, num_cus, stream);
  }
  if constexpr (ENGINE == 1) {
    if (BM + BN > 256 || (int64_t)a.tiles_m * a.tiles_n <= num_cus)
      return launch_tiled<BM, BN, WM, WN, ENGINE, true, 1>(a, out_kind, num_cus, stream);
  }
  return launch_tiled<BM, BN, WM, WN, ENGINE, false, 1>(a, out_kind, num_cus, stream);
}

template <int ENGINE>
hipError_t launch_engine(GemmArgs a, int out_kind, int num_cus, hipStream_t stream) {
  auto tiles = [&](int bm, int bn) {
    int64_t tn = 0;
    if (a.groups > 1) {
      for (int p = 0; p < a.groups; ++p) tn += (a.gN[p] + bn - 1) / bn;
    } else {
      tn = (a.N + bn - 1) / bn;
    }
    return (int64_t)((a.M + bm - 1) / bm) * tn;
  };
  const int cfg = pick_cfg(tiles(256, 256), tiles(192, 256), tiles(256, 128), tiles(128, 128), num_cus);
  const bool split = a.groups == 1 && gemm_splits_k(a.M, a.N, a.K, num_cus, ENGINE);
  switch (cfg) {
    case 1: return launch_cfg<256, 256, 2, 4, ENGINE>(a, out_kind, num_cus, stream, false);
    case 7: return launch_cfg<192, 256, 2, 4, ENGINE>(a, out_kind, num_cus, stream, false);
    case 5: return launch_cfg<256, 128, 4, 2, ENGINE>(a, out_kind, num_cus, stream, false);
    case 6: return launch_cfg<128, 64, 2, 2, ENGINE>(a, out_kind, num_cus, stream, split);
    default: return launch_cfg<128, 128, 2, 2, ENGINE>(a, out_kind, num_cus, stream, split);
  }
}

}  // namespace

bool gemm_splits_k(int64_t M, int64_t N, int64_t K, int num_cus, int accum) {
  static const int forced = forced_env("FP8MOT_GEMM_SPLIT");   // 0: never, 1: any K (tuning)
  if (forced == 0 || K <= KS) return false;
  const int cfg = pick_cfg(tiles_of(M, N, 256, 256), tiles_of(M, N, 192, 256),
                           tiles_of(M, N, 256, 128), tiles_of(M, N, 128, 128), num_cus);
  // 128x64 tiles split K for the exact engine only: the FP8 engine's four
  // 24 KB stages in LDS serve it better there (512x4096x12288: 48.1 us split,
  // 41.1 us with four stages), while at 128x128 the split wins for both
  // engines (2048x2048x8192 FP8 engine: 42.0 against 46.5 us).
  if (cfg != 3 && !(cfg == 6 && accum != 1)) return false;   // 1: FP8 engine
  if (tiles_of(M, N, 128, cfg == 3 ? 128 : 64) > num_cus) return false;
  return K > N || forced == 1;
}

hipError_t launch_gemm(const uint8_t* qa, const uint8_t* qb, void* y,
                       int64_t M, int64_t N, int64_t K, const float* sx,
                       const float* sw, int out_kind, const float* sy,
                       int accum, int num_cus, hipStream_t stream, int64_t ldc) {
  GemmArgs a{};
  a.A = qa; a.B = qb; a.C = y;
  a.M = (int)M; a.N = (int)N; a.K = (int)K;
  a.sx = sx; a.sw = sw; a.sy = sy;
  a.ldc = (int)(ldc > 0 ? ldc : N);
  a.groups = 1;
  if (accum == 1) return launch_engine<1>(a, out_kind, num_cus, stream);
  return launch_engine<0>(a, out_kind, num_cus, stream);
}

hipError_t launch_gemm_grouped(const uint8_t* qa, int groups, const uint8_t* const* qb,
                               void* const* y, const int64_t* N, int64_t M, int64_t K,
                               const float* sx, const float* const* sw, int accum,
                               int num_cus, hipStream_t stream) {
  GemmArgs a{};
  a.A = qa;
  a.M = (int)M; a.K = (int)K;
  a.sx = sx;
  a.groups = groups;
  for (int p = 0; p < groups; ++p) {
    a.gB[p] = qb[p];
    a.gC[p] = y[p];
    a.gsw[p] = sw[p];
    a.gN[p] = (int)N[p];
  }
  a.B = qb[0]; a.C = y[0]; a.sw = sw[0]; a.N = (int)N[0]; a.ldc = (int)N[0];
  if (accum == 1) return launch_engine<1>(a, 0, num_cus, stream);
  return launch_engine<0>(a, 0, num_cus, stream);
}

hipError_t launch_gemm_swiglu(const uint8_t* qx, const uint8_t* wg, const uint8_t* wu,
                              uint8_t* qh, int64_t M, int64_t I, int64_t H,
                              const float* sx, const float* sg, const float* su,
                              const float* sh, int accum, int num_cus, hipStream_t stream) {
  GemmArgs a{};
  a.A = qx; a.B = wg; a.B2 = wu; a.C = qh;
  a.M = (int)M; a.N = (int)I; a.K = (int)H;
  a.sx = sx; a.sw = sg; a.sw2 = su; a.sy = sh;
  a.ldc = (int)I;
  a.groups = 1;
  if (accum == 1) return launch_fused<256, 2, 4, 1>(a, num_cus, stream);
  return launch_fused<256, 2, 4, 0>(a, num_cus, stream);
}

}  // namespace fp8mot

