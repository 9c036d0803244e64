/*
 * fp8mot.h -- C ABI of libfp8mot: the static per-tensor FP8 (OCP E4M3FN)
 * W8A8 Linear stack of a Mixture-of-Transformers decoder tower, on AMD
 * MI355X (gfx950).
 *
 * Sources (the passages each call follows are cited at the call):
 *  [MC]  model card "Cosmos3-Nano-Policy-DROID, FP8 + RTN + moving-average
 *        activation observer": header paragraph and section "Scheme".
 *  [PR]  pull request "Load static FP8 Cosmos3 Nano/Super checkpoints without
 *        re-quantizing them" (TensorRT-LLM 17476): sections "Description",
 *        "What changed", "Supported surface, and what is refused", and the
 *        commit messages.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - All tensor pointers are DEVICE pointers on the current HIP device,
 *    owned by the caller; the library allocates nothing and keeps no
 *    per-call state (the one exception is the fixed scratch array behind
 *    gated_mlp_fp8_noalloc, see there).  Tensors are dense and contiguous (row-major); a
 *    strided tensor must be rejected by the caller before it gets here
 *    ([PR] first commit message: strided inputs are refused, not copied).
 *  - BF16 tensors are passed as uint16_t bit patterns, FP8 tensors as uint8_t
 *    E4M3FN codes (bias 7, no infinities, 0x7F/0xFF are NaN, max 448).
 *  - Every scale is a `const float*` DEVICE pointer to one FP32 scalar.  The
 *    library never reads a scale on the host: a host read would synchronize
 *    the device on the hot path ([PR] "What changed": the shared-scale
 *    invariant is validated once when the weights are loaded, and no scale
 *    is read during the forward pass).  A NULL scale asks for
 *    dynamic quantization, which the static path refuses
 *    (FP8MOT_ERR_UNSUPPORTED; [PR] "What changed": dynamic quantization is
 *    rejected explicitly).
 *  - Scales must be finite and > 0; that is validated once at load with
 *    fp8_check_shared_scale / by the caller, not per call.
 *  - Calls are asynchronous on `stream`.  The return code covers argument
 *    validation and kernel launch, not kernel completion.  Nothing is
 *    launched when a call returns an error.
 *  - Base pointers of tensors must be 16-byte aligned (128-bit loads and
 *    stores); otherwise FP8MOT_ERR_MISALIGNED -- a refusal, not a slow path
 *    ([PR] "Supported surface, and what is refused": an unsupported case is
 *    refused outright rather than served by a silent fallback).
 *  - Sizes are int64_t element counts.  Negative sizes are
 *    FP8MOT_ERR_INVALID_ARG; an empty tensor (a zero size) is a valid no-op
 *    and then data pointers may be NULL.
 *  - GEMM size limits (fp8_linear and every call built on it): M, N, K at
 *    most INT32_MAX; 256 * K below 0x7FFFF000 (K <= 8,388,576); 256 output
 *    rows below 0x7FFFF000 bytes (row length ldc = N, or the ldc argument,
 *    times 1, 2 or 4 bytes for FP8, BF16, FP32 output); at most INT32_MAX
 *    tiles of 128 x 64.  The kernels address one tile's rows with 32-bit
 *    offsets; larger sizes are FP8MOT_ERR_INVALID_ARG, never wrapped.
 *  - Only gfx950 devices are supported; any other device gives
 *    FP8MOT_ERR_UNSUPPORTED.
 *  - The library is reentrant: calls on different streams may overlap.
 */
#ifndef FP8MOT_H
#define FP8MOT_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FP8MOT_OK = 0,
  FP8MOT_ERR_INVALID_ARG = 1,    /* NULL pointer, negative or too large size, K % 16 != 0, bad enum, non-finite c */
  FP8MOT_ERR_MISALIGNED = 2,     /* a tensor base pointer is not 16-byte aligned */
  FP8MOT_ERR_SCALE_MISMATCH = 3, /* a shared-quantization group's input scales differ */
  FP8MOT_ERR_UNSUPPORTED = 4,    /* NULL scale (dynamic quantization) or non-gfx950 device */
  FP8MOT_ERR_HIP = 5,            /* a HIP runtime call or a kernel launch failed */
  FP8MOT_ERR_WORKSPACE = 6,      /* workspace NULL, misaligned or smaller than required */
  FP8MOT_ERR_TOO_LARGE = 7       /* sizes exceed the allocation-free entry point's scratch */
} fp8mot_status;

/* Bytes of device scratch behind gated_mlp_fp8_noalloc (one copy per device,
 * held by the library until the process ends). */
#define FP8MOT_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* Output kind of fp8_linear. */
typedef enum {
  FP8MOT_OUT_BF16 = 0, /* y = bf16_rne(acc * (s_x * s_w)), uint16_t [M, N] */
  FP8MOT_OUT_FP8 = 1,  /* y = e4m3(acc * (s_x * s_w) / s_y), uint8_t [M, N] */
  FP8MOT_OUT_F32 = 2,  /* y = acc * (s_x * s_w) before any output rounding, float [M, N] */
  FP8MOT_OUT_FP8_BLOCK = 3 /* fp8_residual_norm alone: codes with an FP32 scale for each
                              128 columns of a row, as fp8_quant_block gives them */
} fp8mot_out;

/* Accumulation engine of the FP8 GEMMs (fp8_linear and the composites).
 *
 * FP8MOT_ACC_EXACT: the FP8 codes are decoded exactly to F16 in the kernel
 *   and multiplied on the F16 matrix cores; products are accumulated to FP32
 *   precision (|y - alpha*S| stays far inside 1e-5 * alpha * sum|terms|).
 *   Peak is the F16 MFMA rate (2.5 PFLOP/s dense on MI355X).
 * FP8MOT_ACC_FP8_MFMA: the native FP8 matrix-core instruction at twice that
 *   rate.  On gfx950 the FP8 MFMA sums each group of 8 consecutive K products
 *   on a grid 13 bits below the group's largest product (smaller products are
 *   truncated toward zero) before adding the group to the FP32 accumulator;
 *   the per-output error is bounded by alpha * sum over groups of
 *   7 * 2^(e_max(group) - 13) and reaches ~1e-4 of sum|terms| on adversarial
 *   inputs (about 5e-5 on Gaussian activations and weights).
 * The two engines give different (each deterministic) results. */
typedef enum {
  FP8MOT_ACC_EXACT = 0,
  FP8MOT_ACC_FP8_MFMA = 1
} fp8mot_acc;

/* Element type of the float tensors that come in two: the bias and residual
 * of fp8_linear_act and the layer norm's inputs. */
typedef enum {
  FP8MOT_ELEM_BF16 = 0, /* uint16_t bit patterns */
  FP8MOT_ELEM_F32 = 1   /* float */
} fp8mot_elem;

/* Activation of fp8_linear_act, evaluated in FP32.  At z = -Inf gelu,
 * gelu_tanh and silu give the NaN of -Inf * 0; a NaN stays a NaN.  gelu's
 * Phi(-a) is within (1.25 a^2 + 14) 2^-24 of its own size while it is a normal
 * FP32 number (a < 12.9); the sigma of the other two is within about |x| 2^-23
 * of its size at an argument x < 0. */
typedef enum {
  FP8MOT_ACT_NONE = 0,      /* z */
  FP8MOT_ACT_RELU = 1,      /* max(z, 0) */
  FP8MOT_ACT_GELU = 2,      /* z * Phi(z), Phi the normal distribution function */
  FP8MOT_ACT_GELU_TANH = 3, /* z * (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
  FP8MOT_ACT_SILU = 4       /* z / (1 + exp(-z)) */
} fp8mot_act;

/* Observer mode of fp8_observe. */
typedef enum {
  FP8MOT_OBS_MAX = 0,       /* running max of the per-call amax */
  FP8MOT_OBS_MOVING_AVG = 1 /* moving average of the per-call amax */
} fp8mot_obs;

/* Observer state, 16 bytes in device memory.  An all-zero state is a fresh
 * observer (the caller zero-fills it once).  `m` is the observed value,
 * `count` the number of calls folded in; `pending` (the call's running amax)
 * and `arrived` (the call's workgroups that have added theirs) are the
 * library's own reduction slots and are back at zero after each call.  Calls
 * on one state must not overlap (use one stream, or one state per stream). */
typedef struct {
  float m;
  int32_t count;
  uint32_t pending;
  uint32_t arrived;
} fp8mot_observer_state;

/* ------------------------------------------------------------------ */
/* Library                                                             */
/* ------------------------------------------------------------------ */

/* Checks that `device` is a gfx950 GPU and caches that result.  Optional:
 * every call checks the current device itself.  Returns FP8MOT_OK,
 * FP8MOT_ERR_UNSUPPORTED (other architecture) or FP8MOT_ERR_HIP. */
int fp8mot_init(int device);

/* Static message for a status code (never NULL). */
const char* fp8mot_status_string(int status);

/* Number of activation-quantization launches made by this process so far
 * (fp8_quant_static, and the one inside each composite).  A test hook for
 * the single-quantization property: a composite call adds exactly 1. */
uint64_t fp8mot_debug_quant_launches(void);

/* Measurement aid, not a step of the path: the read/write ceiling of the
 * HBM-bound kernels' byte mix.  Reads a[0..n) (and b[0..n) when b is not
 * NULL) as 16-bit words and writes out[0..n) = the low byte of a[i] (or of
 * a[i] ^ b[i]): 2 bytes read + 1 written per element like fp8_quant_static,
 * or 4 + 1 like silu_mul_2in_fp8, with their access pattern and grid and no
 * arithmetic.  a, b: [n] 16-byte aligned; out: [n] 16-byte aligned.
 * Refusals as fp8_quant_static (no scale). */
int fp8mot_rw_ceiling(const uint16_t* a, const uint16_t* b, uint8_t* out, int64_t n,
                      hipStream_t stream);

/* Measurement aid, not a step of the path: the rate the matrix cores sustain
 * on given FP8 data with nothing else in the loop (no copies, LDS, decodes or
 * epilogue).  MI355X's clock, and with it the MFMA rate, falls under its
 * power limit by an amount that depends on how much the operand bits toggle,
 * so the GEMM kernels are measured against this rather than the published
 * dense peaks alone.  Every wave takes four A fragments from a[0..na) and
 * four B fragments from b[0..nb) (E4M3 codes, each lane its own, indices
 * wrapped), then issues 8 * iters MFMAs on four accumulators:
 * accum = FP8MOT_ACC_EXACT: v_mfma_f32_32x32x16_f16 on the codes decoded
 * exactly to F16 (2*32*32*16 FLOP each); FP8MOT_ACC_FP8_MFMA: the native
 * v_mfma_scale_f32_32x32x64_f8f6f4 (2*32*32*64 FLOP each).  Grid: one
 * 512-thread workgroup per CU.  sink: one device float, written only if the
 * products sum to a sentinel that finite data never reaches.  *flops (host)
 * receives the launch's FLOP count.  Refusals: a NULL pointer, na or nb < 64,
 * iters < 1 or another accum -> FP8MOT_ERR_INVALID_ARG, before any device
 * access. */
int fp8mot_mfma_ceiling(const uint8_t* a, int64_t na, const uint8_t* b, int64_t nb,
                        int64_t iters, int accum, float* sink, double* flops,
                        hipStream_t stream);

/* Conversion of fp8mot_convert_f32. */
typedef enum {
  FP8MOT_CONV_E4M3_PACKED = 0, /* packed gfx950 conversion after a NaN-propagating clamp to
                                  +-448, NaN bytes set to 0x7F: the quantize and SwiGLU
                                  kernels' bodies and the GEMMs' FP8 output */
  FP8MOT_CONV_E4M3_INT = 1,    /* integer round-to-nearest-even on the bit pattern: the
                                  elementwise kernels' tails */
  FP8MOT_CONV_BF16 = 2         /* packed gfx950 BF16 conversion: the GEMM epilogues */
} fp8mot_conv;

/* Verification aid, not a step of the path: the FP32 -> E4M3 and FP32 ->
 * BF16 conversions of the path's kernels, applied to any FP32 input, so that
 * they can be checked on every FP32 bit pattern against the encoding rules
 * ([MC] "Scheme": E4M3 with round to nearest even; the library saturates to
 * +-448, maps NaN to 0x7F and keeps the sign of zero; BF16 round to nearest
 * even, NaN stays NaN).
 *   kind FP8MOT_CONV_E4M3_PACKED or FP8MOT_CONV_E4M3_INT:
 *     out: uint8_t [n], out[i] = the E4M3 code of x[i];
 *   kind FP8MOT_CONV_BF16:
 *     out: uint16_t [n], out[i] = the BF16 bits of x[i].
 * x: float [n], 16-byte aligned; out 16-byte aligned.  n must be a multiple
 * of 4 (the kernels convert four values at a time); n == 0 is a no-op.
 * Refusals: n < 0, n % 4 != 0, another kind, or (n > 0) a NULL pointer ->
 * FP8MOT_ERR_INVALID_ARG; a misaligned pointer -> FP8MOT_ERR_MISALIGNED. */
int fp8mot_convert_f32(const float* x, void* out, int64_t n, int kind, hipStream_t stream);

/* ------------------------------------------------------------------ */
/* Steps of the hot path                                               */
/* ------------------------------------------------------------------ */

/* Static activation quantization ([MC] "Scheme": FP8 E4M3 activations with
 * one static per-tensor scale; [PR] "What changed": the shared activation is
 * quantized once and the FP8 tensor is handed to every projection).
 *   q[i] = e4m3(fp32(x[i]) / *d_scale)
 * with one correctly rounded FP32 division and round-to-nearest-even E4M3
 * encoding that saturates to +-448 (NaN -> 0x7F, the sign of zero kept).
 * x: BF16 [n], q: E4M3 [n] (flat; any rank). */
int fp8_quant_static(const uint16_t* x, uint8_t* q, int64_t n,
                     const float* d_scale, hipStream_t stream);

/* FP8 Linear, one projection with its own weight and weight scale
 * ([PR] "Description": each projection keeps s_i * qW_i, no re-quantization
 * onto max(s); commit messages: each Linear applies its own scale in the
 * GEMM epilogue).
 *   acc[m,n] = sum_k e4m3_value(qx[m,k]) * e4m3_value(qw[n,k])  (FP32 accumulation)
 *   alpha    = fp32(*d_sx * *d_sw)
 *   y[m,n]   = per `out_kind` (see fp8mot_out), acc * alpha first.
 * qx: E4M3 [M, K] row-major; qw: E4M3 [N, K] row-major (out x in, K
 * contiguous); y: [M, N] row-major, contiguous (leading dimension N).
 * K must be a multiple of 16.  d_sy is used only for FP8MOT_OUT_FP8 (NULL
 * there is FP8MOT_ERR_UNSUPPORTED) and ignored otherwise.  K == 0 writes
 * zeros.  `accum` selects the engine (fp8mot_acc).  Order of the FP32 sum:
 * along K, except for a GEMM with K > N whose 128-row output tiles (128x128,
 * or 128x64 when even those are too few) give no CU more than one, where the
 * 128-K blocks at even and at odd
 * positions are summed separately and the two sums added at the end (both
 * orders are FP32 accumulation of the same exact products).  The order
 * depends on (M, N, K) only, so equal shapes give equal bits. */
int fp8_linear(const uint8_t* qx, const uint8_t* qw, void* y, int64_t M,
               int64_t N, int64_t K, const float* d_sx, const float* d_sw,
               int out_kind, const float* d_sy, int accum, hipStream_t stream);

/* Two-input SwiGLU with direct FP8 emission ([PR] "What changed" and the
 * first commit message: SiLU(G) * U from two separate tensors, quantized for
 * the FP8 down projection; flat indexing, rank-agnostic).
 *   q[i] = e4m3(silu(g[i]) * u[i] / *d_s_out),  silu(g) = g / (1 + exp(-g))
 * evaluated in FP32.  g, u: BF16 [n]; q: E4M3 [n]. */
int silu_mul_2in_fp8(const uint16_t* g, const uint16_t* u, uint8_t* q,
                     int64_t n, const float* d_s_out, hipStream_t stream);

/* The same with the swiglu_alpha / swiglu_beta variant ([PR] commit message
 * on swiglu_alpha / swiglu_beta: alpha is a gain inside the sigmoid, beta an
 * offset on up):
 *   q[i] = e4m3(g[i] * sigmoid(alpha * g[i]) * (u[i] + beta) / *d_s_out)
 * in FP32.  A zero beta leaves u untouched, so (alpha, beta) = (1, 0) gives
 * exactly the codes of silu_mul_2in_fp8.  Non-finite alpha or beta is
 * FP8MOT_ERR_INVALID_ARG; other arguments as silu_mul_2in_fp8. */
int silu_mul_2in_fp8_ab(const uint16_t* g, const uint16_t* u, uint8_t* q,
                        int64_t n, const float* d_s_out, float alpha, float beta,
                        hipStream_t stream);

/* One-input SwiGLU with gate and up adjacent in one tensor ([PR] commit
 * message: silu_and_mul needs gate and up adjacent; the two-input form exists
 * because separate projections have no such tensor).  x: BF16 [rows, 2*inter]
 * whose row r holds the inter gate values, then the inter up values;
 * q: E4M3 [rows, inter]:
 *   q[r, c] = e4m3(g * sigmoid(alpha g) * (u + beta) / *d_s_out),
 *   g = x[r, c], u = x[r, inter + c],
 * bit for bit what silu_mul_2in_fp8_ab gives on the two halves.  x and q
 * 16-byte aligned (FP8MOT_ERR_MISALIGNED); rows, inter >= 0; any inter (a
 * multiple of 16 takes the vector path). */
int silu_mul_fp8(const uint16_t* x, uint8_t* q, int64_t rows, int64_t inter,
                 const float* d_s_out, float alpha, float beta, hipStream_t stream);

/* ------------------------------------------------------------------ */
/* Per-row FP8 (per-channel weights, per-token activations)            */
/* ------------------------------------------------------------------ */

/* Per-row dynamic quantization ([MC] section 3.2: the per-channel weight /
 * per-token activation builds; the runtime FP8 path quantizes weights per
 * output channel at load and activations per token at run time).  For each
 * row r of x (BF16 [rows, K]):
 *   d_scales[r] = fp32(max_k |x[r,k]|) / 448      (FP32 division)
 *   q[r,k]      = e4m3(fp32(x[r,k]) / d_scales[r]) (IEEE FP32 division)
 * A zero row gets scale 0 and keeps its signed zeros; a row holding a NaN
 * gets a NaN scale and NaN codes.  Used for per-token activations (rows =
 * tokens) and, at load time, per-channel weights (rows = output channels).
 * K must be a multiple of 16 (FP8MOT_ERR_INVALID_ARG); x, q 16-byte aligned
 * (FP8MOT_ERR_MISALIGNED); d_scales: FP32 [rows], caller-owned device memory.
 * rows == 0 does nothing; K == 0 writes scale 0 for every row (an empty row
 * is a zero row) and then x and q may be NULL. */
int fp8_quant_per_row(const uint16_t* x, uint8_t* q, float* d_scales,
                      int64_t rows, int64_t K, hipStream_t stream);

/* FP8 GEMM with per-row scales on both operands:
 *   y[m,n] = fp32( acc[m,n] * fp32(d_sx[m] * d_sw[n]) ),
 *   acc[m,n] = sum_k dec(qx[m,k]) * dec(qw[n,k])   (engine per `accum`)
 * d_sx: FP32 [M] (per token), d_sw: FP32 [N] (per output channel), both
 * device memory, 16-byte aligned.  out_kind: FP8MOT_OUT_BF16 or
 * FP8MOT_OUT_F32 (FP8 output is FP8MOT_ERR_UNSUPPORTED).  Other arguments and
 * refusals as fp8_linear. */
int fp8_linear_rowwise(const uint8_t* qx, const uint8_t* qw, void* y, int64_t M,
                       int64_t N, int64_t K, const float* d_sx, const float* d_sw,
                       int out_kind, int accum, hipStream_t stream);

/* ------------------------------------------------------------------ */
/* FP8 with a scale for each block of 128                              */
/* ------------------------------------------------------------------ */

/* Dynamic quantization with an FP32 scale for each block of 128, finer than
 * fp8_quant_per_row's: an outlier costs precision in its block alone.
 *   scale = fp32(amax of the block) / 448,  q = e4m3(fp32(x) / scale)
 * (IEEE FP32 divisions) for blocks of x [M, K] (of x_elem, fp8mot_elem) that are
 *   tile 0: 128 columns of a row (the last one K's remainder)
 *   tile 1: 128 x 128 tiles (the last ones the remainders)
 * and with transpose 1 the same of x^T, whose codes and scales are written
 * as those of a [K, M] tensor:
 *   transpose 0: q [M, ld(K)], scales [M, nb(K)], or with tile [nb(M), nb(K)]
 *   transpose 1: q [K, ld(M)], scales [K, nb(M)], or with tile [nb(K), nb(M)]
 * with nb(n) = ceil(n / 128) and ld(n) = n rounded up to a multiple of 16, the
 * codes from n on being those of zeros: rows of codes of any length are
 * operands of fp8_linear_block.  Activations and gradients have blocks of a
 * row, weights tiles; a product's backward pass takes the transposed forms:
 *   dx = dy w     fp8_linear_block of dy's rows and w's transposed tiles
 *   dw = dy^T x   fp8_linear_block of dy's and x's transposed rows, FP32 out
 * A zero block gets scale 0 and keeps its signed zeros; one that holds a NaN
 * gets a NaN scale and NaN codes (its padding too), one with an infinity an
 * infinite scale, zeros and, for the infinity, a NaN code.
 * M up to INT32_MAX and K up to 2^26; x, q 16-byte aligned.  q and scales lie
 * apart from x and from each other.  M == 0 or K == 0 does nothing. */
int fp8_quant_block(const void* x, int x_elem, uint8_t* q, float* d_scales, int64_t M,
                    int64_t K, int tile, int transpose, hipStream_t stream);

/* silu_mul_2in_fp8 with a scale for each 128 columns of a row, taken from the
 * values themselves instead of calibrated:
 *   v = g / (1 + exp(-g)) * u            (FP32, within 9 * 2^-24 of its value;
 *                                         zero where exp(-g) overflows)
 *   q, scales = fp8_quant_block of v [M, K]  (tile 0, transpose 0)
 * g, u: BF16 [M, K], 16-byte aligned like q [M, ld(K)]; limits as there. */
int silu_mul_2in_block(const uint16_t* g, const uint16_t* u, uint8_t* q, float* d_scales,
                       int64_t M, int64_t K, hipStream_t stream);

/* FP8 Linear of operands that have a scale for each block of 128 of K, with
 * fp8_linear_act's epilogue:
 *   P[m,n,b] = sum_{k in block b} e4m3_value(qx[m,k]) * e4m3_value(qw[n,k])
 *   acc[m,n] = sum_b fp32(d_sx[m,b] * d_sw[n',b]) * P[m,n,b]
 *   z = acc + bias[n],  v = act(z) + residual[m,n],  y per out_kind
 * d_sx: FP32 [M, nb(K)]; d_sw: with w_rows 0 FP32 [nb(N), nb(K)] and n' = n / 128
 * (weights), with w_rows 1 FP32 [N, nb(K)] and n' = n (a weight's gradient,
 * whose operands are both quantized along the rows summed over).  The sums are
 * FP32 on the exact engine (codes decoded to F16, see FP8MOT_ACC_EXACT): each
 * block's products are summed by themselves and added by one FMA, along K in
 * turns or strided over the waves of a workgroup; the order depends on
 * (M, N, K) only.  The scales may differ widely, between blocks too; a product
 * of two scales below FP32's range is 0, above it infinite.
 * bias, act, residual, pre, out_kind (BF16, FP8 at d_sy, FP32), d_sy and the
 * overlaps that are allowed: as fp8_linear_act (y may be the residual: a
 * weight's gradient is added to in place).  No workspace.  K == 0 gives
 * act(bias) + residual.  K must be a multiple of 16 (pad codes with zeros, as
 * fp8_quant_block does); M, N, K as in fp8_linear; qx, qw, y, bias, residual,
 * pre 16-byte aligned. */
int fp8_linear_block(const uint8_t* qx, const uint8_t* qw, void* y, int64_t M, int64_t N,
                     int64_t K, const float* d_sx, const float* d_sw, int w_rows,
                     const void* bias, int bias_elem, int act, const void* residual,
                     int residual_elem, uint16_t* pre, int out_kind, const float* d_sy,
                     hipStream_t stream);

/* ------------------------------------------------------------------ */
/* Linear epilogue: bias, activation, residual                         */
/* ------------------------------------------------------------------ */

/* Bytes of workspace fp8_linear_act needs: 0 for most shapes, FP32 partial
 * sums where K is split over workgroups (more than about two million outputs,
 * rows and columns counted in whole sixteens, whose tiles leave CUs idle, and
 * K of about 2000 or more).  Depends on (M, N, K) only: tiles and splits are
 * chosen for 256 CUs, whatever the device has.  Returns 0 for sizes that
 * fp8_linear_act refuses. */
size_t fp8_linear_act_workspace(int64_t M, int64_t N, int64_t K);

/* FP8 Linear with bias, activation and residual in its epilogue:
 *   acc[m,n] = sum_k e4m3_value(qx[m,k]) * e4m3_value(qw[n,k])
 *   z        = fma(acc, alpha, bias[n]),     alpha = fp32(s_x * s_w)
 *   v        = act(z) + residual[m,n]
 *   y[m,n]   = bf16_rne(v) | e4m3(v * r) | v    per out_kind
 * each step one FP32 operation, r = fp32(1 / *d_sy), which has to be finite;
 * NULL bias or residual leaves its addition out.  The bias of a projection, the activation of an ungated MLP and the
 * residual stream's addition after o and down are what a decoder layer does
 * to a projection's output; here no pass over [M, N] is spent on them.
 *  - row_scales 0: d_sx, d_sw one scale each, as fp8_linear; row_scales 1:
 *    d_sx [M] and d_sw [N], alpha[m,n] = fp32(d_sx[m] * d_sw[n]), as
 *    fp8_linear_rowwise.
 *  - bias: [N] of bias_elem (fp8mot_elem); residual: [M, N] of residual_elem.
 *  - pre: NULL, or BF16 [M, N] that receives bf16_rne(z), which the backward
 *    pass needs.
 *  - y may be the residual itself where the element types agree (the sum is
 *    then added in place); any other overlap of y or pre with an input or
 *    with each other is refused.
 *  - accum as fp8_linear.  Calls of few rows (M <= 64) or few outputs (about
 *    two million and less) are bound by bytes, not by the matrix cores, and
 *    always sum as FP8MOT_ACC_EXACT does.
 *  - ws: 16-byte aligned device workspace of at least
 *    fp8_linear_act_workspace(M, N, K) bytes (may be NULL where that is 0).
 *    Calls that may run at the same time need workspaces of their own; one
 *    that lies over another tensor of the call is refused.
 * K == 0 gives act(bias) + residual.  The order of the FP32 sum depends on
 * (M, N, K, accum) only; it is not fp8_linear's.  qx, qw, y, bias, residual,
 * pre 16-byte aligned; row scales too.  M, N, K as in fp8_linear. */
int fp8_linear_act(const uint8_t* qx, const uint8_t* qw, void* y, int64_t M, int64_t N,
                   int64_t K, const float* d_sx, const float* d_sw, int row_scales,
                   const void* bias, int bias_elem, int act, const void* residual,
                   int residual_elem, uint16_t* pre, int out_kind, const float* d_sy,
                   int accum, void* ws, size_t ws_bytes, hipStream_t stream);

/* Bytes of workspace fp8_linear_act_backward needs for dbias (column sums
 * over slabs of rows; 0 where one slab is all).  Returns 0 for sizes that
 * fp8_linear_act_backward refuses. */
size_t fp8_linear_act_backward_workspace(int64_t M, int64_t N);

/* Backward pass of fp8_linear_act's epilogue: for the gradient dy of y,
 *   dz[m,n]  = bf16_rne(dy * act'(pre)),   dbias[n] = sum_m dy * act'(pre)
 * (the residual's gradient is dy itself).  The sum takes the FP32 products,
 * before their rounding to BF16, in an order that depends on (M, N) only.
 * dz goes on to the input's gradient through the frozen weight:
 * fp8_quant_per_row and fp8_linear_rowwise on the transposed codes.
 * dy, pre, dz: BF16 [M, N]; dbias: FP32 [N]; all 16-byte aligned.  dz or
 * dbias may be NULL (not computed), and with FP8MOT_ACT_NONE pre too.  dz may
 * be dy or pre itself; any other overlap is refused.  relu's slope at 0 is 0;
 * gelu's and silu's at an infinite argument are the NaN of Inf * 0.  M == 0
 * writes dbias = 0.
 * M up to INT32_MAX, N up to 2^26.
 * ws: 16-byte aligned, at least fp8_linear_act_backward_workspace(M, N)
 * bytes, apart from every tensor of the call; unused where dbias is NULL. */
int fp8_linear_act_backward(const uint16_t* dy, const uint16_t* pre, int act, uint16_t* dz,
                            float* dbias, int64_t M, int64_t N, void* ws, size_t ws_bytes,
                            hipStream_t stream);

/* ------------------------------------------------------------------ */
/* Layer norm                                                          */
/* ------------------------------------------------------------------ */

/* Layer norm of each row of x, with direct FP8 emission for the projections
 * that read it (one quantized tensor for a group that shares its input scale,
 * as silu_mul_2in_fp8 emits the down projection's input):
 *   mean = sum_i x[i] / H,   var = sum_i (x[i] - mean)^2 / H
 *   rstd = 1 / sqrt(var + eps)             (where |mean| > 4 / rstd, both are
 *          corrected by the mean of the differences x[i] - mean)
 *   v    = fma((x[i] - mean) * rstd, weight[i], bias[i])       (FP32)
 *   y[i] = bf16_rne(v) | e4m3(v * r) | v    per out_kind, r = fp32(1 / *d_sy)
 * x: [rows, H] of x_elem (fp8mot_elem); weight, bias: [H] of wb_elem, either
 * may be NULL (ones, zeros); y: [rows, H]; mean, rstd: FP32 [rows] for the
 * backward pass, or NULL.  eps finite and >= 0.  y may be x itself where the
 * element types agree; any other overlap is refused.  H up to 2^26, rows up to
 * INT32_MAX;
 * x, y, weight, bias 16-byte aligned.  1 / *d_sy has to be finite.  A row that
 * holds a NaN or an infinity, or whose sums leave FP32's range, becomes NaN
 * (or what 1 / sqrt(Inf) = 0 makes of it, where the squares alone overflow). */
int fp8_layer_norm(const void* x, int x_elem, const void* weight, const void* bias,
                   int wb_elem, void* y, int out_kind, const float* d_sy, float* mean,
                   float* rstd, int64_t rows, int64_t H, float eps, hipStream_t stream);

/* Bytes of workspace fp8_layer_norm_backward needs for dweight and dbias
 * (column sums over slabs of rows; 0 where one slab is all).  Returns 0 for
 * sizes that fp8_layer_norm_backward refuses. */
size_t fp8_layer_norm_backward_workspace(int64_t rows, int64_t H);

/* Backward pass of fp8_layer_norm, for the gradient dy of y (an FP8 y passes
 * its gradient straight through):
 *   xh = (x - mean) * rstd,   g = dy * weight
 *   dx = rstd * (g - sum_i g / H - xh * sum_i(g * xh) / H) + dres
 *   dweight[i] = sum_rows dy * xh,   dbias[i] = sum_rows dy
 * mean, rstd: what fp8_layer_norm wrote.  dres: NULL, or the gradient that
 * reaches x past the norm (the residual stream's), added before dx is
 * rounded.  dy: of dy_elem; x, dres, dx: of x_elem; weight: [H] of w_elem or
 * NULL (ones); dweight, dbias: FP32 [H], either may be NULL (not computed).
 * dx may be dy or dres itself where the element types agree, or x; any other
 * overlap of an output is refused.  rows == 0 writes dweight = dbias = 0.  Sizes as fp8_layer_norm.
 * The sums over rows take an order that depends on (rows, H) only.  All
 * tensors 16-byte aligned but mean and rstd.  ws: 16-byte aligned, at least
 * fp8_layer_norm_backward_workspace(rows, H) bytes, apart from every tensor of
 * the call; unused where dweight and dbias are NULL. */
int fp8_layer_norm_backward(const void* dy, int dy_elem, const void* x, int x_elem,
                            const void* weight, int w_elem, const float* mean,
                            const float* rstd, const void* dres, void* dx, float* dweight,
                            float* dbias, int64_t rows, int64_t H, void* ws, size_t ws_bytes,
                            hipStream_t stream);

/* ------------------------------------------------------------------ */
/* Norms before and after a block, its gate and residual scale         */
/* ------------------------------------------------------------------ */

/* What stands between two blocks of a decoder layer, in one pass: the norm
 * after the block's last projection, the block's gate, the residual addition
 * with its scale, and the norm before the next block with direct FP8 emission
 * for the projections that read it (root mean square norms):
 *   post_rstd = 1 / sqrt(sum_i hidden[i]^2 / H + eps)
 *   z    = hidden[i] * post_rstd                   (hidden[i] without post_weight)
 *   f    = (alpha * gate[i]) * post_weight[i]      (alpha times what there is)
 *   r[i] = fma(z, f, x[i])                         the residual stream, x's type
 *   rstd = 1 / sqrt(sum_i r[i]^2 / H + eps)
 *   w    = r[i] * rstd * weight[i]
 *   y[i] = bf16_rne(w) | e4m3(w / *d_sy) (times fp32(1 / *d_sy)) | w, or with
 *          FP8MOT_OUT_FP8_BLOCK codes [rows, ld(H)] and d_scales [rows, nb(H)]
 *          as fp8_quant_block gives them of w
 * each step one FP32 operation; rstd and w are taken from r before its rounding
 * to x's type.  f is formed before hidden comes in: where alpha * gate leaves
 * FP32's range f is infinite or 0, also where the whole product would be in it.
 *  - x, r: [rows, H] of x_elem; hidden: [rows, H] of h_elem, or NULL for the
 *    norm alone (r, gate and post_weight then have to be NULL: y of x).
 *  - gate: NULL, or [gates, H] of gate_elem, each row the gate of rows / gates
 *    rows one after another (one for all, one for each sample of a batch of
 *    equal lengths, one for each row); gates, up to INT32_MAX, has to divide
 *    rows.
 *  - post_weight, weight: [H] of w_elem; weight NULL: ones.  alpha finite.
 *  - rstd, post_rstd: FP32 [rows] for the backward pass, or NULL.
 *  - r may be x itself (the stream is then updated in place), and y x without
 *    hidden, where the element types agree; any other overlap of an output is refused.
 * eps finite and >= 0; H up to 2^26, rows up to INT32_MAX; tensors 16-byte
 * aligned but d_scales, rstd and post_rstd.  A row of zeros with eps 0 is NaN
 * (0 * Inf); a NaN or an infinity, or squares beyond FP32's range, make of
 * their row what the formulas do. */
int fp8_residual_norm(const void* x, int x_elem, const void* hidden, int h_elem,
                      const void* gate, int gate_elem, int64_t gates,
                      const void* post_weight, const void* weight, int w_elem, void* r,
                      void* y, int out_kind, const float* d_sy, float* d_scales, float* rstd,
                      float* post_rstd, int64_t rows, int64_t H, float alpha, float eps,
                      hipStream_t stream);

/* Bytes of workspace fp8_residual_norm_backward needs (column sums over slabs
 * of rows; gates 1 without a gate).  Returns 0 for sizes that it refuses. */
size_t fp8_residual_norm_backward_workspace(int64_t rows, int64_t H, int64_t gates);

/* Backward pass of fp8_residual_norm, for the gradients dy of y (an FP8 y
 * passes its gradient straight through) and dr, what reaches r past the norm:
 *   n = r * rstd,  g = dy * weight,  z = hidden * post_rstd (hidden without post_weight)
 *   dx = rstd * (g - n * sum_i(g * n) / H) + dr
 *   p  = dx * ((alpha * gate) * post_weight)
 *   dhidden = post_rstd * (p - z * sum_i(p * z) / H)  (p without post_weight)
 *   dweight = sum_rows dy * n,   dpost_weight = sum_rows alpha * gate * dx * z
 *   dgate   = alpha * post_weight * the sum of dx * z over the gate's rows
 * in FP32, dx not yet rounded where it is used again; of the last two, factors
 * that rows share multiply those rows' sum.  r, rstd, post_rstd:
 * what fp8_residual_norm wrote (r as stored).  dy, hidden, dhidden: of h_elem;
 * r, dr, dx: of r_elem.  Without hidden gate, post_weight, dhidden, dgate and
 * dpost_weight have to be NULL; dr NULL: no such gradient.  dweight,
 * dpost_weight FP32 [H], dgate FP32 [gates, H]: each may be NULL (not
 * computed), and without gate or post_weight has to be.  dx may be dy, r or dr
 * itself and dhidden dy or hidden, where the element types agree; any other
 * overlap of an output is refused.  rows == 0 writes zeros to the parameters'
 * gradients.  The sums over rows take an order that depends on (rows, H,
 * gates) only.  Sizes and alignment as there; ws: 16-byte aligned, at least
 * fp8_residual_norm_backward_workspace(rows, H, gates) bytes, apart from every
 * tensor of the call. */
int fp8_residual_norm_backward(const void* dy, const void* r, int r_elem, const void* hidden,
                               int h_elem, const void* gate, int gate_elem, int64_t gates,
                               const void* post_weight, const void* weight, int w_elem,
                               const float* rstd, const float* post_rstd, const void* dr,
                               void* dx, void* dhidden, float* dgate, float* dpost_weight,
                               float* dweight, int64_t rows, int64_t H, float alpha, void* ws,
                               size_t ws_bytes, hipStream_t stream);

/* ------------------------------------------------------------------ */
/* Fused-topology comparison (what the split path avoids)              */
/* ------------------------------------------------------------------ */

/* fp8_linear writing into a row-strided output: row m of y starts ldc
 * elements after row m - 1 (ldc >= N), so two projections can write the
 * column slices [:, 0:N) and [:, N:2N) of one [M, 2N] buffer ([PR] "What
 * changed": writing both GEMMs into column slices of one buffer went wrong
 * in the original stack because the GEMM assumed the leading dimension was
 * N).  Elements of y outside [0, M) x [0, N) are not written.  ldc < N is
 * FP8MOT_ERR_INVALID_ARG; other arguments as fp8_linear. */
int fp8_linear_ldc(const uint8_t* qx, const uint8_t* qw, void* y, int64_t M,
                   int64_t N, int64_t K, int64_t ldc, const float* d_sx,
                   const float* d_sw, int out_kind, const float* d_sy, int accum,
                   hipStream_t stream);

/* The failure mode of a fused group that keeps one scale ([PR]
 * "Description": each member re-quantized as FP8-round((s_i * qW_i) /
 * max(s))), for the fused-topology comparison only:
 *   out[k] = e4m3(fp32(fp32(*d_s_member * dec(qw[k])) / max(d_s_group[0..g-1])))
 * qw, out: E4M3 [n], 16-byte aligned; d_s_member: FP32 scalar, d_s_group:
 * FP32 [group_size] (1..64), device memory.  NULL scales are
 * FP8MOT_ERR_UNSUPPORTED. */
int fp8_requantize_onto_max(const uint8_t* qw, uint8_t* out, int64_t n,
                            const float* d_s_member, const float* d_s_group,
                            int group_size, hipStream_t stream);

/* ------------------------------------------------------------------ */
/* Composites (one shared quantization, contiguous outputs, no sync)   */
/* ------------------------------------------------------------------ */

/* Bytes of workspace gated_mlp_fp8 needs: qX [M,H] + qH [M,I], each region
 * 256-byte aligned.  Returns 0 for negative sizes. */
size_t gated_mlp_fp8_workspace(int64_t M, int64_t H, int64_t I);

/* Gated MLP with split gate/up ([PR] "What changed": GatedMLP with
 * split_gate_up quantizes the shared activation once and hands both
 * projections the FP8 tensor; SiLU(G)*U emits FP8 at the down input scale).
 *   qX = quant(x; sx); G = linear(qX, wg; sx, sg); U = linear(qX, wu; sx, su)
 *   qH = silu_mul_2in(G, U; sh); y = linear(qH, wd; sh, sd)  (BF16 out)
 * Bitwise equal to those five calls when I >= H (the gate and up GEMMs and
 * the SwiGLU run as one kernel whose epilogue rounds G and U to BF16 and
 * applies the SwiGLU exactly as the separate calls do; G and U are never
 * written).  With H > I and few tiles the separate gate/up fp8_linear calls
 * sum K in two halves (see fp8_linear) while this kernel sums along K, so
 * an SwiGLU code can then differ by one step.
 * x: [M, H]; wg, wu: [I, H]; wd: [H, I];
 * y: [M, H].  H and I multiples of 16.  ws: device workspace of at least
 * gated_mlp_fp8_workspace(M, H, I) bytes, 256-byte aligned.  `accum`
 * selects the GEMM engine (fp8mot_acc) of all three GEMMs.  I == 0 (empty
 * weights, whose pointers may be NULL) writes y = 0, the down projection of
 * an empty sum; M == 0 or H == 0 writes nothing. */
int gated_mlp_fp8(const uint16_t* x, int64_t M, int64_t H, int64_t I,
                  const float* d_sx, const uint8_t* wg, const float* d_sg,
                  const uint8_t* wu, const float* d_su, const float* d_sh,
                  const uint8_t* wd, const float* d_sd, uint16_t* y, void* ws,
                  size_t ws_bytes, int accum, hipStream_t stream);

/* gated_mlp_fp8 for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same launches and bitwise the same y, with qX and qH kept in a scratch
 * array the library holds per device (FP8MOT_NOALLOC_SCRATCH_BYTES, a
 * file-scope device array whose address is looked up once per device)
 * instead of a caller workspace.  The call allocates nothing.
 * Limit: gated_mlp_fp8_workspace(M, H, I) <= FP8MOT_NOALLOC_SCRATCH_BYTES
 * (64 MiB: M * (H + I) up to about 64M codes, e.g. M = 4096, H = 4096,
 * I = 12288), else FP8MOT_ERR_TOO_LARGE and nothing is launched.
 * Every call on one device shares that device's scratch: calls that overlap
 * on one GPU (different streams, or different threads without ordering) race
 * on it and must be serialized by the caller.  Nothing in the scratch needs
 * to start at zero (each call overwrites the qX and qH it reads).  Other
 * arguments, refusals and the engine choice as gated_mlp_fp8. */
int gated_mlp_fp8_noalloc(const uint16_t* x, int64_t M, int64_t H, int64_t I,
                          const float* d_sx, const uint8_t* wg, const float* d_sg,
                          const uint8_t* wu, const float* d_su, const float* d_sh,
                          const uint8_t* wd, const float* d_sd, uint16_t* y, int accum,
                          hipStream_t stream);

/* The gate/up half of the gated MLP from an already quantized activation
 * ([PR] "What changed": one quantized activation handed to both
 * projections; the two-input SwiGLU emits FP8 for the down projection):
 *   qh = silu_mul_2in_fp8(linear(qx, wg; sx, sg), linear(qx, wu; sx, su); sh)
 * (bitwise when I >= H, as for gated_mlp_fp8), computed by one kernel that
 * shares each qx tile between the two GEMMs and never writes G or U.  qx: E4M3 [M, H]; wg, wu: E4M3 [I, H];
 * qh: E4M3 [M, I].  H and I multiples of 16.  `accum` per fp8mot_acc. */
int fp8_gate_up_swiglu(const uint8_t* qx, const uint8_t* wg, const float* d_sx,
                       const float* d_sg, const uint8_t* wu, const float* d_su,
                       const float* d_sh, uint8_t* qh, int64_t M, int64_t I,
                       int64_t H, int accum, hipStream_t stream);

/* Bytes of workspace qkv_fp8 needs: qX [M, H], 256-byte aligned. */
size_t qkv_fp8_workspace(int64_t M, int64_t H);

/* Split Q/K/V with one shared activation quantization ([PR] "What changed":
 * Attention with share_qkv_input_quant; "It is also faster": split
 * projections give contiguous outputs).
 *   qX = quant(x; sx); yq = linear(qX, wq; sx, sq); yk = ...; yv = ...
 * x: [M, H]; wq: [Nq, H]; wk: [Nk, H]; wv: [Nv, H]; yq: [M, Nq], yk: [M, Nk],
 * yv: [M, Nv], three separate contiguous BF16 tensors.  H multiple of 16.
 * The three GEMMs run as one grouped launch, or as three launches when
 * fp8_linear would split K for one of them; either way bitwise what three
 * fp8_linear calls give.  A member with N == 0 is skipped and its pointers may be NULL.
 * H == 0 quantizes nothing (x, the weights and ws may be NULL) and writes each
 * projection's epilogue of an empty sum, zero; M == 0 writes nothing.
 * Cross-attention, where k/v read a different tensor than q, must not use
 * this call: quantize each input separately and use fp8_linear.  `accum`
 * selects the GEMM engine (fp8mot_acc). */
int qkv_fp8(const uint16_t* x, int64_t M, int64_t H, const float* d_sx,
            const uint8_t* wq, int64_t Nq, const float* d_sq,
            const uint8_t* wk, int64_t Nk, const float* d_sk,
            const uint8_t* wv, int64_t Nv, const float* d_sv, uint16_t* yq,
            uint16_t* yk, uint16_t* yv, void* ws, size_t ws_bytes, int accum,
            hipStream_t stream);

/* ------------------------------------------------------------------ */
/* Calibration                                                         */
/* ------------------------------------------------------------------ */

/* Folds one calibration call into an observer ([MC] header and "Scheme":
 * static input scales from the global max of the activations, or from a
 * moving average of the per-call maxima with constant 0.01).
 *   a = max |x[i]|   (NaN if any x[i] is NaN)
 *   first call: m = a
 *   FP8MOT_OBS_MAX:        m = max(m, a)            (NaN propagates)
 *   FP8MOT_OBS_MOVING_AVG: m = m + c * (a - m)      (three FP32 roundings, no FMA)
 * x: BF16 [n], n >= 1 (an empty call has no maximum to fold, so n == 0 is
 * FP8MOT_ERR_INVALID_ARG, the one exception to the empty-tensor rule above).
 * d_state: device fp8mot_observer_state (zero-filled
 * before the first call; 16-byte aligned).  `c` is used by the moving
 * average only and must be finite.  Calls on one state must be
 * stream-ordered. */
int fp8_observe(const uint16_t* x, int64_t n, void* d_state, int mode,
                float c, hipStream_t stream);

/* Same as fp8_observe with a = max |silu(g[i]) * u[i]| (FP32 evaluation as in
 * silu_mul_2in_fp8): calibrates the down projection's input scale from the
 * gate/up outputs without materializing the product. */
int fp8_observe_swiglu(const uint16_t* g, const uint16_t* u, int64_t n,
                       void* d_state, int mode, float c, hipStream_t stream);

/* *d_scale = fp32(state.m / 448): the static per-tensor scale. */
int fp8_scale_from_state(const void* d_state, float* d_scale,
                         hipStream_t stream);

/* Load-time check of a shared-quantization group ([PR] "What changed": the
 * projections sharing one quantized activation must carry the same
 * calibrated input_scale; validated when the weights are loaded, not in the
 * forward pass).
 * h_scales: HOST array of n >= 1 scales.  FP8MOT_OK iff all are finite,
 * > 0 and bitwise equal; FP8MOT_ERR_SCALE_MISMATCH if they differ;
 * FP8MOT_ERR_INVALID_ARG for NULL, n < 1, or a non-finite or non-positive
 * scale.  Pure host code: usable without a GPU. */
int fp8_check_shared_scale(const float* h_scales, int n);

#ifdef __cplusplus
}
#endif

#endif /* FP8MOT_H */
