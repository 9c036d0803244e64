// Device pieces of the Linear epilogue's FP8 x FP8 products (gfx950): tile
// order, exact decode, operand windows and copies into LDS.  gemm.hip, whose
// recorded counters are tied to its own text, holds the same pieces itself: a
// change to one belongs in the other too.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8mot {
namespace tile {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kNumXcd = 8;         // MI355X: 8 XCDs
constexpr int kOOB = 0x7FFFFFF0;   // a byte offset past every buffer window

// Workgroup id -> (tile_m, tile_n): blocks go to the 8 XCDs round-robin, so
// each XCD gets a contiguous run of tiles, walked in bands of `band` tile rows
// that share A and B rows in that XCD's L2.
__device__ __forceinline__ void tile_of(int bid, int tiles_m, int tiles_n, int band, int& tm, int& tn) {
  const int nb = tiles_m * tiles_n;
  const int xcd = bid % kNumXcd, idx = bid / kNumXcd;
  const int q = nb / kNumXcd, r = nb % kNumXcd;
  const int t = (xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q) + idx;
  const int per_band = band * tiles_n;
  const int b = t / per_band;
  const int first_m = b * band;
  const int rows = min(tiles_m - first_m, band);
  const int in_band = t - b * per_band;
  tm = first_m + in_band % rows;
  tn = in_band / rows;
}

// Eight E4M3 codes (two dwords) -> eight F16 values with the gfx950 packed
// conversion at scale 1.0: every E4M3 value is exactly an F16 value (max 448,
// smallest subnormal 2^-9 is an F16 normal) and the NaN codes become a NaN.
__device__ __forceinline__ f16x8 decode8(int lo, int hi) {
  return __builtin_bit_cast(
      f16x8, (v4i){__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)lo, 1.0f, false)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)lo, 1.0f, true)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)hi, 1.0f, false)),
                   __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)hi, 1.0f, true))});
}

// Buffer resource over [base, base + bytes): loads beyond it return 0 and
// stores beyond it are dropped.  The third-dword value is the standard gfx9
// raw-buffer configuration.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const int n = bytes > 0x7FFFFFF0LL ? 0x7FFFFFF0 : (bytes > 0 ? (int)bytes : 0);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, n, 0x00020000);
}

// The same descriptor as four dwords for the inline-assembly copy below.
__device__ __forceinline__ v4i make_rsrc_words(const void* base, int64_t bytes) {
  const int n = bytes > 0x7FFFFFF0LL ? 0x7FFFFFF0 : (int)bytes;
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return (v4i){(int)(uint32_t)a, (int)(uint32_t)((a >> 32) & 0xFFFF), n, 0x00020000};
}

// One wave-wide 16-byte-per-lane copy from a buffer straight into LDS: lane
// i's bytes land at lds_addr + 16 * i, out-of-range lanes write zeros.  As
// assembly, so that the compiler does not make every LDS read wait for every
// copy; the kernel waits for its copies itself before the barrier that
// publishes a stage.  M0 holds the LDS address; one wait state separates its
// write from the copy.
__device__ __forceinline__ void copy_to_lds(v4i rsrc, uint32_t lds_addr, int voff, int soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
      : "memory", "m0");
}

}  // namespace tile
}  // namespace fp8mot
