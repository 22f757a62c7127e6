/*
 * libspin — the online hot path of SpinQuant (arXiv 2405.16406) on AMD
 * Instinct MI355X (gfx950): Hadamard rotations applied online, symmetric INT4
 * quantization of activations / KV vectors, INT4 x INT4 GEMM, the offline
 * fold of a rotation into a weight, and a paged quantized KV cache with its
 * attention, drafted trees and eviction.
 *
 * Where each operation comes from (page "SpinQuant, Reproduced"):
 *   - Q1, Q5 "Method 1/2": a pre-norm transformer is invariant to an
 *     orthogonal change of basis of its hidden state; R1 (residual) and R2
 *     (head-wise, value path) are folded into weights; R3 (KV path) and R4
 *     (before down_proj) cannot be folded and run online as Hadamards.
 *   - abstract (all pages): weights, activations and KV cache are 4-bit.
 * The pages fix no interface, granularity, rounding or storage; the choices
 * below (per-token / per-channel / per-(token, head) absmax / 7 scales,
 * round-half-even, clamp to +-7, nibble packing) are this library's reading.
 *
 * Conventions shared by every call
 *   - Tensor pointers are DEVICE pointers to row-major, contiguous memory,
 *     allocated and freed by the caller; the library never allocates, frees
 *     or keeps them.  Every tensor pointer must be 16-byte aligned (4 bytes
 *     suffice for the tables and lists of spin_kv_move).
 *   - What a call writes lies apart from what it reads and from what else it
 *     writes, unless the call says that the two may be the same.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Calls validate their arguments on the host, enqueue kernels on `stream`
 *     and return without synchronising; device faults surface at the caller's
 *     next synchronisation.
 *   - Validation failures return a non-zero spin_status and enqueue nothing,
 *     so no output is written.  SPIN_ERR_HIP means the HIP runtime rejected a
 *     launch; outputs are then undefined.
 *   - Empty problems (M, N, T or H equal to 0) are valid and enqueue nothing.
 *   - The library holds no state; calls are re-entrant and thread-safe.
 *   - INT4 codes are two's-complement nibbles in [-7, 7] (-8 never occurs);
 *     byte j of a packed row holds code 2j in bits 0..3 and code 2j+1 in bits
 *     4..7.
 *   - Hadamard orders ("had_n"): 1 (no rotation), 2^k for 1 <= k <= 14, and
 *     12 * 2^k for 0 <= k <= 10.  H_{2^k} is Sylvester's matrix in natural
 *     order, H[i][j] = (-1)^popcount(i & j).  H_12 is Paley's first
 *     construction over GF(11): with chi the quadratic character mod 11,
 *     Q[a][b] = chi(b - a) and H_12 = I + [[0, 1^T], [-1, Q]] (row/column 0
 *     the border).  H_{12 * 2^k} = H_12 (x) H_{2^k}, element index a*2^k + b.
 *     The rotation applied is the row-vector product y = x . H_n / sqrt(n),
 *     block-diagonally along a row longer than n.
 */
#ifndef LIBSPIN_H
#define LIBSPIN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status and dtype travel as plain ints: every int a caller passes is a
   valid argument (an unknown dtype is rejected with SPIN_ERR_UNSUPPORTED,
   spin_status_string names an unknown status), which an enum type would not
   allow in C++. */
typedef int spin_status;
enum {
    SPIN_OK = 0,
    SPIN_ERR_NULL = 1,          /* a required pointer is NULL                      */
    SPIN_ERR_BAD_SHAPE = 2,     /* a size is negative, not a required multiple, or too large */
    SPIN_ERR_MISALIGNED = 3,    /* a tensor pointer is not 16-byte aligned         */
    SPIN_ERR_UNSUPPORTED = 4,   /* unsupported Hadamard order, dtype or flag value */
    SPIN_ERR_HIP = 5            /* the HIP runtime reported an error               */
};

typedef int spin_dtype;
enum { SPIN_F32 = 0, SPIN_F16 = 1 };

/* Largest row length spin_fwht_quant accepts. */
#define SPIN_FWHT_MAX_K 32768
/* Most rows one spin_fwht_quant (and _f6, _gemm) call takes, and most
   (token, head) vectors one spin_kv_quant call takes: each kernel launch has
   fewer than 2^32 work-items in its one grid dimension, and these kernels
   give a row 256 of them (rounded up to 256 rows where rows are placed per
   XCD), a workgroup of 256 to 32 KV vectors. */
#define SPIN_FWHT_MAX_M ((1 << 24) - 256)
#define SPIN_KV_MAX_VECTORS (((1LL << 24) - 1) * 32)
/* Largest K spin_w4a4_gemm accepts: 49 * K * 256 must stay below 2^31
   (the kernel accumulates codes scaled by 16 on each side in int32). */
#define SPIN_GEMM_MAX_K 171136

/*
 * spin_fold_rotation — offline fold of a rotation into a weight, then
 * per-output-channel INT4 (page "SpinQuant, Reproduced", Q5: R1/R2 are merged
 * into adjacent weights and are free at runtime; R4's inverse is merged into
 * down_proj).
 *
 *   W       [K][N] float32   input features x output features
 *   R       [r_block][r_block] float32, or NULL for the library Hadamard
 *           H_{r_block} / sqrt(r_block) (r_block must then be a Hadamard order)
 *   W_rot   [K][N] float32   OUTPUT: W' = blockdiag(R, ..., R)^T W  (required;
 *           it is both the result and the buffer the quantizer reads)
 *   Wq      [N][K/2] uint8   OUTPUT: codes of column n of W', packed
 *   w_scale [N] float32      OUTPUT: fl32(max_k |W'[k][n]| / 7)
 * Codes are clamp(rne(fl32(W'[k][n] / w_scale[n])), -7, 7); a column of zeros
 * gets scale 0 and zero codes.
 * Requirements: K > 0, K % 64 == 0, K % r_block == 0, N >= 0, r_block >= 1.
 * W' accumulates in float32; it is within 1e-5 (relative, per column) of the
 * float64 product.
 */
spin_status spin_fold_rotation(const float* W, int K, int N, const float* R, int r_block,
                               float* W_rot, uint8_t* Wq, float* w_scale, void* stream);

/*
 * spin_fwht_quant — online Hadamard + per-token INT4 of activations (page
 * "SpinQuant, Reproduced", Q5: R4 before down_proj is applied online as a
 * Hadamard over the MLP width; abstract: 4-bit activations).
 *
 *   X        [M][K] float32 (x_dtype SPIN_F32) or float16 (SPIN_F16)
 *   had_n    Hadamard order (see above); 1 = quantize only; K % had_n == 0
 *   Xq       [M][K/2] uint8   OUTPUT: packed codes of y
 *   x_scale  [M] float32      OUTPUT: s = fl32(max_k |y[m][k]| / 7)
 *   X_rot    [M][K] float32 or NULL   OUTPUT: exactly the float32 values y
 *            that were quantized
 * y = x . blockdiag(H_n / sqrt(n)) computed in float32 (within 1e-5 relative
 * per row of the exact product); codes are clamp(rne(fl32(y / s)), -7, 7)
 * with the IEEE float32 quotient, bit-exact; a zero row gets s = 0 and zero
 * codes.  Requirements: 0 <= M <= SPIN_FWHT_MAX_M, 0 < K <= SPIN_FWHT_MAX_K,
 * K % 32 == 0.
 */
spin_status spin_fwht_quant(const void* X, spin_dtype x_dtype, int M, int K, int had_n,
                            uint8_t* Xq, float* x_scale, float* X_rot, void* stream);

/*
 * spin_w4a4_gemm — INT4 x INT4 product with per-token and per-channel scales
 * (abstract: W4A4).
 *
 *   Xq       [M][K/2] uint8   packed activation codes (from spin_fwht_quant)
 *   x_scale  [M] float32
 *   Wq       [N][K/2] uint8   packed weight codes, output-channel-major
 *                             (from spin_fold_rotation)
 *   w_scale  [N] float32
 *   Y        [M][N] float32   OUTPUT: fl32(fl32(float(acc) * x_scale[m]) * w_scale[n])
 *   acc_out  [M][N] int32 or NULL   OUTPUT: acc[m][n] = sum_k qx[m][k] * qw[n][k]
 * The integer product is exact (int32 accumulation, bit-exact) for codes in
 * [-7, 7], the range the library produces; any nibble is accepted, and with
 * -8 codes the bound on K that keeps the sum exact is 64/49 times smaller.
 * Requirements: M, N >= 0, K > 0, K % 64 == 0, K <= SPIN_GEMM_MAX_K.
 */
spin_status spin_w4a4_gemm(const uint8_t* Xq, const float* x_scale, const uint8_t* Wq,
                           const float* w_scale, int M, int N, int K, float* Y,
                           int32_t* acc_out, void* stream);

/* Kernel families for spin_w4a4_gemm_ex. */
#define SPIN_GEMM_AUTO 0   /* the choice spin_w4a4_gemm makes */
#define SPIN_GEMM_INT8 1   /* codes widened to int8, int8 matrix cores, int32 accumulation */
#define SPIN_GEMM_FP6 2    /* codes as FP6 E2M3 (u = q + 8, exact), FP6 matrix cores */
#define SPIN_GEMM_FP6_SPLITK 3   /* the FP6 tiles with K split into slices; see below */
/* K range of the FP6 kernel: its float32 accumulator of products u_a * u_b <= 225
   is exact while 225 K < 2^24 (K < 74566; the bound stops at the power of two
   below), and its pipeline needs two steps of 128 codes. */
#define SPIN_GEMM_FP6_MIN_K 256
#define SPIN_GEMM_FP6_MAX_K 65536

/*
 * spin_w4a4_gemm_ex — spin_w4a4_gemm with the kernel family named: the same
 * arguments, outputs and guarantees (every family gives the same bits), for
 * callers that tune the choice for their shapes.  `kernel` is SPIN_GEMM_AUTO,
 * SPIN_GEMM_INT8, SPIN_GEMM_FP6 or SPIN_GEMM_FP6_SPLITK.
 * SPIN_GEMM_FP6_SPLITK (taken by AUTO for 129 or more rows whose 256 x 256
 * tiles leave half the compute units idle, when it predicts a gain) is three
 * launches on `stream`: Y is zeroed, the FP6 tiles of every K slice add their
 * exact int32 partial products into Y read as int32 (atomically), and a last
 * pass turns Y into the dequantized float32 outputs in place (and writes
 * acc_out).  The slice count is chosen from the shape (1 when slicing does not
 * pay).  The integer sum is exact and the epilogue the same, so the bits equal
 * the other families'; between the launches Y holds integers.
 * Errors: SPIN_ERR_UNSUPPORTED for another `kernel` value; with
 * SPIN_GEMM_FP6 or SPIN_GEMM_FP6_SPLITK, SPIN_ERR_BAD_SHAPE unless K % 128 == 0
 * and SPIN_GEMM_FP6_MIN_K <= K <= SPIN_GEMM_FP6_MAX_K; otherwise as
 * spin_w4a4_gemm.
 */
spin_status spin_w4a4_gemm_ex(const uint8_t* Xq, const float* x_scale, const uint8_t* Wq,
                              const float* w_scale, int M, int N, int K, float* Y,
                              int32_t* acc_out, int kernel, void* stream);

/*
 * The FP6 operand layout of activation codes, written by spin_fwht_quant_f6
 * and read by spin_w4a4_gemm_f6 and spin_w4a4_gemm_f6f6 (this library's
 * format, also written by spin_codes_f6; the pages fix no
 * storage): the INT4 codes q of an [M][K] activation matrix, each held as the
 * 6-bit field of u = q + 8 (bits 0..3 = u, bits 4..5 = 0: the FP6 E2M3 value
 * u / 8), ordered for the gfx950 matrix cores.  Row r, code k lies in the
 * 1536-byte region (r / 32) * (K / 64) + k / 64, at byte
 * ((k % 64) / 32) * 768 + (r % 32) * 24 + ((k % 32) / 16) * 12 of it, in field
 * sigma(k % 16) of those 12 bytes read as a 96-bit little-endian number (field
 * p at bits 6p .. 6p + 5), sigma = 0 1 12 2 3 14 4 5 11 6 7 13 8 9 15 10.
 * Rows are rounded up to a multiple of 32; the rows past M are padding that
 * spin_fwht_quant_f6 does not write and that no result depends on (they hold
 * whatever the buffer held).  K % 64 == 0.  1.5 bytes per code.
 */
#define SPIN_F6_BYTES(M, K) ((size_t)(((M) + 31) / 32) * ((size_t)(K) / 64) * 1536)

/* Longest row spin_fwht_quant_f6 quantizes without a rotation (had_n == 1). */
#define SPIN_FWHT_F6_QUANT_MAX_K 16384

/*
 * spin_fwht_quant_f6 — spin_fwht_quant (per-token INT4, after the R4 Hadamard
 * or with no rotation, page "SpinQuant, Reproduced", Q5) with the codes
 * written in the FP6 operand layout above, for spin_w4a4_gemm_f6 and
 * spin_w4a4_gemm_f6f6.
 *
 *   X        [M][K] float16 with K == had_n == 12288 (the down projection's
 *            input, R4 online), or float16 / float32 with had_n == 1 (inputs
 *            whose rotation is folded upstream: qkv_proj, o_proj, gate/up)
 *   Xf6      SPIN_F6_BYTES(M, K) bytes   OUTPUT: the codes spin_fwht_quant
 *            computes for the same arguments, in the FP6 operand layout
 *   x_sum    [M] int32     OUTPUT: sum_k q[m][k]
 *   x_scale  [M] float32   OUTPUT: as spin_fwht_quant
 * Requirements: 0 <= M <= SPIN_FWHT_MAX_M; had_n == 12288: x_dtype ==
 * SPIN_F16, K == 12288; had_n == 1: K % 128 == 0, SPIN_GEMM_FP6_MIN_K <= K <=
 * SPIN_FWHT_F6_QUANT_MAX_K.
 * Errors: SPIN_ERR_NULL, SPIN_ERR_UNSUPPORTED for another had_n or dtype,
 * SPIN_ERR_BAD_SHAPE, SPIN_ERR_MISALIGNED (16-byte alignment).
 */
spin_status spin_fwht_quant_f6(const void* X, spin_dtype x_dtype, int M, int K, int had_n, uint8_t* Xf6,
                               int32_t* x_sum, float* x_scale, void* stream);

/*
 * spin_w4a4_gemm_f6 — spin_w4a4_gemm with the activation codes in the FP6
 * operand layout (abstract: W4A4): Y and acc_out are the same bits
 * spin_w4a4_gemm gives for those codes.
 *
 *   Xf6      SPIN_F6_BYTES(M, K) bytes (from spin_fwht_quant_f6)
 *   x_sum    [M] int32, sum_k q[m][k]   x_scale [M] float32
 *   Wq, w_scale, Y, acc_out   as for spin_w4a4_gemm
 * Requirements: M, N >= 0, K % 128 == 0,
 * SPIN_GEMM_FP6_MIN_K <= K <= SPIN_GEMM_FP6_MAX_K.
 */
spin_status spin_w4a4_gemm_f6(const uint8_t* Xf6, const int32_t* x_sum, const float* x_scale,
                              const uint8_t* Wq, const float* w_scale, int M, int N, int K, float* Y,
                              int32_t* acc_out, void* stream);

/*
 * spin_codes_f6 — packed INT4 codes [N][K/2] (spin_fold_rotation's Wq, or
 * the activation codes of spin_fwht_quant) rewritten in the FP6 operand
 * layout above (row n of the codes as row r of the layout), with the code
 * sum of every row, for spin_w4a4_gemm_f6f6.  Weights are static, so theirs
 * is done once, offline (abstract: W4A4), and the conversion of the weight
 * codes into the matrix cores' operand format leaves the hot path.  Any
 * nibble is accepted (-8 becomes the field of u = 0).
 *
 *   Wq     [N][K/2] uint8    packed codes
 *   Wf6    SPIN_F6_BYTES(N, K) bytes   OUTPUT (padding rows past N unwritten)
 *   w_sum  [N] int32         OUTPUT: sum_k q[n][k]
 * Requirements: N >= 0, K > 0, K % 64 == 0, K <= SPIN_GEMM_MAX_K.
 * Errors: SPIN_ERR_NULL for a null pointer, SPIN_ERR_BAD_SHAPE, and
 * SPIN_ERR_MISALIGNED unless every pointer is 16-byte aligned; N == 0 enqueues
 * nothing.
 */
spin_status spin_codes_f6(const uint8_t* Wq, int N, int K, uint8_t* Wf6, int32_t* w_sum, void* stream);

/*
 * spin_w4a4_gemm_f6f6 — spin_w4a4_gemm with both operands in the FP6 operand
 * layout (activations from spin_fwht_quant_f6, weights from spin_codes_f6):
 * Y and acc_out are the same bits spin_w4a4_gemm gives for those codes.
 *
 *   Xf6, x_sum, x_scale   as for spin_w4a4_gemm_f6
 *   Wf6      SPIN_F6_BYTES(N, K) bytes, w_sum [N] int32 (the weight codes
 *            from spin_codes_f6)
 *   w_scale, Y, acc_out   as for spin_w4a4_gemm
 * Requirements: M, N >= 0, K % 128 == 0,
 * SPIN_GEMM_FP6_MIN_K <= K <= SPIN_GEMM_FP6_MAX_K.
 * Errors: SPIN_ERR_NULL, SPIN_ERR_BAD_SHAPE, SPIN_ERR_MISALIGNED (16-byte
 * alignment of every pointer) as for spin_w4a4_gemm_f6; M == 0 or N == 0
 * enqueues nothing.
 */
spin_status spin_w4a4_gemm_f6f6(const uint8_t* Xf6, const int32_t* x_sum, const float* x_scale,
                                const uint8_t* Wf6, const int32_t* w_sum, const float* w_scale, int M, int N,
                                int K, float* Y, int32_t* acc_out, void* stream);

/* 32-bit words of the workspace spin_fwht_quant_gemm takes. */
#define SPIN_FWHT_QUANT_GEMM_WORKSPACE_WORDS 1025

/*
 * spin_fwht_quant_gemm — the down projection's input rotation R4 and its
 * W4A4 product in one launch: spin_fwht_quant followed by spin_w4a4_gemm
 * (page "SpinQuant, Reproduced", Q5: R4 is an online Hadamard right before
 * down_proj; abstract: W4A4).
 *
 *   X          [M][K] float16, K == had_n == 12288 (the MLP width; H_12 (x) H_1024)
 *   Wq, w_scale, N   the folded INT4 weights as for spin_w4a4_gemm
 *   Xq, x_scale      OUTPUT: the codes and scales spin_fwht_quant writes
 *   Y, acc_out       OUTPUT: as spin_w4a4_gemm writes them from those codes
 *   workspace  SPIN_FWHT_QUANT_GEMM_WORKSPACE_WORDS uint32 of device memory,
 *              all zero before the first call; each call leaves it zero.
 * Every output equals, bit for bit, what the two separate calls write.
 * Requirements: x_dtype == SPIN_F16, K == had_n == 12288 (other shapes: the
 * two calls), M, N >= 0; acc_out may be NULL.  Calls that share a workspace
 * must not overlap (calls on one stream do not); the kernel is launched
 * cooperatively (all its workgroups resident at once).
 * Errors: SPIN_ERR_UNSUPPORTED for another dtype or order, SPIN_ERR_BAD_SHAPE,
 * SPIN_ERR_NULL, SPIN_ERR_MISALIGNED as for the two calls; SPIN_ERR_HIP if
 * the device cannot run the cooperative launch.  The wait of a GEMM tile for
 * its rows is bounded (about half a second, or 2^22 polls); it cannot expire
 * while every workgroup is resident, which the cooperative launch ensures,
 * but if it did, that tile's Y would be written as NaN (acc_out INT32_MIN)
 * rather than the kernel hanging.
 */
spin_status spin_fwht_quant_gemm(const void* X, spin_dtype x_dtype, int M, int K, int had_n,
                                 const uint8_t* Wq, const float* w_scale, int N, uint8_t* Xq,
                                 float* x_scale, float* Y, int32_t* acc_out, uint32_t* workspace,
                                 void* stream);

/*
 * spin_fwht_quant_gemm_noalloc — spin_fwht_quant_gemm for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  The same arguments, outputs and
 * guarantees without the workspace: the flags live in an array of
 * SPIN_FWHT_QUANT_GEMM_WORKSPACE_WORDS words that the library holds in every
 * GPU it runs on until the process ends (its address is looked up on the
 * first call on each device; nothing is allocated).  The array holds the
 * flags of up to 1024 workgroups; the kernel's grid (one workgroup per
 * compute unit) is capped there, so no call needs more.  It is zero before
 * the first call and every call leaves it zero.  All calls on one GPU share
 * it: calls that overlap on one GPU race (calls on one stream do not
 * overlap).  Errors as for spin_fwht_quant_gemm; SPIN_ERR_HIP if the array's
 * address cannot be obtained.
 */
spin_status spin_fwht_quant_gemm_noalloc(const void* X, spin_dtype x_dtype, int M, int K, int had_n,
                                         const uint8_t* Wq, const float* w_scale, int N, uint8_t* Xq,
                                         float* x_scale, float* Y, int32_t* acc_out, void* stream);

/*
 * spin_kv_quant — head-wise Hadamard (R3) + INT4 KV cache (page "SpinQuant,
 * Reproduced", Q5: R3 in the KV path is an online Hadamard; abstract: 4-bit
 * KV cache).
 *
 *   X       [T][H][D] float32 / float16, D == 128
 *   rotate  1: y = x . H_128 / sqrt(128) per (t, h) vector (K and Q); 0: y = x (V)
 *   codes   [T][H][D/2] uint8 or NULL   OUTPUT: packed codes of y per (t, h)
 *   scale   [T][H] uint16 (IEEE fp16 bits) or NULL   OUTPUT:
 *           s16 = fp16_rne(fl32(max |y| / 7)); codes use float(s16):
 *           clamp(rne(fl32(y / float(s16))), -7, 7), and s16 == 0 gives zeros
 *   X_rot   [T][H][D] float32 or NULL   OUTPUT: the float32 values y
 * codes and scale are both NULL or both non-NULL; when both are NULL, X_rot
 * must be non-NULL (rotate-only, used for Q).  Requirements: T, H >= 0,
 * T * H <= SPIN_KV_MAX_VECTORS, D == 128, rotate in {0, 1}.
 */
spin_status spin_kv_quant(const void* X, spin_dtype x_dtype, int T, int H, int D, int rotate,
                          uint8_t* codes, uint16_t* scale, float* X_rot, void* stream);

/*
 * The 8-bit-activation variant, W4A8KV8 (page "SpinQuant, Reproduced", Q7
 * lists it among the settings the paper evaluates): activations and KV
 * vectors are quantized to symmetric INT8 with the same rules as above and
 * 127 in place of 7 (s = fl32(max |y| / 127), codes clamp(rne(fl32(y / s)),
 * -127, 127), one signed byte per code, natural order); weights stay INT4.
 */

/* Largest K spin_w4a8_gemm accepts: 127 * 7 * 16 * K must stay below 2^31
   (weight codes are scaled by 16 in the int32 accumulation). */
#define SPIN_GEMM8_MAX_K 150912

/*
 * spin_fwht_quant8 — spin_fwht_quant with per-token INT8 codes.
 *
 *   Xq8      [M][K] int8      OUTPUT: codes of y
 *   x_scale  [M] float32      OUTPUT: s = fl32(max_k |y[m][k]| / 127)
 * Every other argument, requirement and guarantee as for spin_fwht_quant.
 */
spin_status spin_fwht_quant8(const void* X, spin_dtype x_dtype, int M, int K, int had_n,
                             int8_t* Xq8, float* x_scale, float* X_rot, void* stream);

/*
 * spin_w4a8_gemm — INT8 activations x INT4 weights (W4A8).
 *
 *   Xq8      [M][K] int8      activation codes (from spin_fwht_quant8)
 *   x_scale  [M] float32
 *   Wq       [N][K/2] uint8   packed weight codes (from spin_fold_rotation)
 *   w_scale  [N] float32
 *   Y, acc_out as for spin_w4a4_gemm; the integer product is exact for
 *   activation codes in [-127, 127] and weight codes in [-7, 7] (the ranges
 *   the library produces).
 * Requirements: M, N >= 0, K > 0, K % 128 == 0, K <= SPIN_GEMM8_MAX_K.
 */
spin_status spin_w4a8_gemm(const int8_t* Xq8, const float* x_scale, const uint8_t* Wq,
                           const float* w_scale, int M, int N, int K, float* Y,
                           int32_t* acc_out, void* stream);

/*
 * spin_kv_quant8 — spin_kv_quant with INT8 KV codes (KV8).
 *
 *   codes   [T][H][D] int8 or NULL   OUTPUT: codes of y per (t, h)
 *   scale   [T][H] uint16 (fp16 bits) or NULL   OUTPUT:
 *           s16 = fp16_rne(fl32(max |y| / 127)); codes
 *           clamp(rne(fl32(y / float(s16))), -127, 127), s16 == 0 gives zeros
 * Every other argument, requirement and guarantee as for spin_kv_quant.
 */
spin_status spin_kv_quant8(const void* X, spin_dtype x_dtype, int T, int H, int D, int rotate,
                           int8_t* codes, uint16_t* scale, float* X_rot, void* stream);

/*
 * spin_kv_qkv — the KV-path step of one attention layer in a single launch
 * (page "SpinQuant, Reproduced", Q5: R3 rotates queries and keys online, so
 * Q . K^T is unchanged, while values carry the folded R2 and are only
 * quantized; abstract: 4-bit KV cache).
 *
 *   Q        [T][Hq][D] float32 / float16, or NULL (no query rotation)
 *   Q_rot    [T][Hq][D] float32, NULL exactly when Q is NULL   OUTPUT:
 *            y = q . H_128 / sqrt(128) per (t, h) vector, not quantized
 *   K, V     [T][Hkv][D], the same dtype as Q; Hq need not equal Hkv
 *            (grouped-query attention)
 *   bits     4: packed INT4 codes, [T][Hkv][D/2] bytes, rules of spin_kv_quant;
 *            8: INT8 codes, [T][Hkv][D] bytes, rules of spin_kv_quant8
 *   K_codes, K_scale   OUTPUT: codes and fp16 scales of K . H_128 / sqrt(128):
 *            the same bytes spin_kv_quant(K, rotate = 1) (spin_kv_quant8 at
 *            bits = 8) writes
 *   K_rot    [T][Hkv][D] float32 or NULL   OUTPUT: the rotated K values
 *   V_codes, V_scale   OUTPUT: codes and fp16 scales of V, not rotated: the
 *            same bytes spin_kv_quant(V, rotate = 0) writes
 * Requirements: T, Hkv >= 0, Hq >= 0 when Q is non-NULL (ignored otherwise),
 * D == 128, bits in {4, 8}; K, V and the four K / V outputs non-NULL.
 * Errors: SPIN_ERR_NULL for a missing pointer or a Q / Q_rot pair with one
 * NULL, SPIN_ERR_UNSUPPORTED for a dtype or bits value outside the above,
 * SPIN_ERR_BAD_SHAPE for a size out of range (2 ceil(T Hkv / 32) + ceil(T Hq / 32)
 * workgroups of 256 above 2^24 - 1, i.e. more than one launch can hold),
 * SPIN_ERR_MISALIGNED as for every call.
 */
spin_status spin_kv_qkv(const void* Q, const void* K, const void* V, spin_dtype x_dtype, int T, int Hq,
                        int Hkv, int D, int bits, float* Q_rot, uint8_t* K_codes, uint16_t* K_scale,
                        float* K_rot, uint8_t* V_codes, uint16_t* V_scale, void* stream);

/*
 * The paged KV cache, written by spin_kv_append and read by spin_kv_attn and
 * spin_kv_attn_shared (the abstract's 4-bit KV cache in the form a server
 * keeps it; the pages fix no storage).  A pool of n_pages pages of page_size
 * tokens, a power of two from SPIN_KV_MIN_PAGE to SPIN_KV_MAX_PAGE, for Hkv
 * heads of D = 128 values, bits = 4 or 8 per code, codes and scales as
 * spin_kv_quant (spin_kv_quant8) defines them:
 *   K_codes  uint8  [n_pages][Hkv][page_size][16 * bits]
 *            a token's 128 codes in order (4 bits: even code in the low nibble)
 *   V_codes  uint8  [n_pages][Hkv][page_size / 4][16][4][bits]
 *            the bytes of codes 8 o .. 8 o + 7 (o = 0 .. 15) of four
 *            consecutive tokens beside each other: the second product of
 *            attention sums over tokens and takes them eight at a time
 *   K_scale, V_scale  uint16 (fp16 bits) [n_pages][Hkv][page_size]
 *
 * A batch of B sequences:
 *   q_start     [B + 1] int32, not falling: rows q_start[b] .. q_start[b + 1] - 1
 *               of the T query rows are sequence b's new tokens (none is
 *               allowed).  Rows before q_start[0] and from q_start[B] on belong
 *               to no sequence: nothing of them is read or written.
 *   kv_len      [B] int32: tokens of the sequence in its own pages, the new
 *               ones among them, so that the i-th new token has place
 *               kv_len[b] - (q_start[b + 1] - q_start[b]) + i
 *   page_table  [B][max_pages] int32: its place p lies in slot p % page_size
 *               of page page_table[b][p / page_size].  Entries past the
 *               sequence's pages are not used.
 * These arrays lie on the device; what they hold cannot be checked by the
 * host, and is checked by the kernels: an entry that is no page of the pool
 * (-1, say) has no tokens (nothing is stored there, nothing is seen there), and
 * so have places from max_pages * page_size on: with a kv_len above that, the
 * sequence's other tokens keep their places.  A kv_len below 0 counts as 0,
 * above 2^30 as 2^30.  With q_start not rising as it should, the rows concerned
 * get wrong values, and nothing is read or written outside the arrays.  A page
 * may stand in several tables (a shared prefix), as long as no two rows of one
 * spin_kv_append call are stored in the same slot.
 */
#define SPIN_KV_MIN_PAGE 16
#define SPIN_KV_MAX_PAGE 1024
/* Most tokens of a sequence: max_pages * page_size, prefix_len, rotary positions. */
#define SPIN_KV_MAX_CONTEXT (1 << 29)

/*
 * spin_rope_table — cosines and sines of the position rotation, for
 * spin_kv_append.
 *
 *   inv_freq    [n] float64: the turn of pair i per position, 1 <= n <= 64.
 *               Scaling for long contexts lies in it (frequencies divided by a
 *               factor, another base, a factor per frequency).
 *   attn_scale  multiplies every entry (1 for none)
 *   table       [P][2 n] float32   OUTPUT: row p holds n cosines, then n sines
 *               of the angles (pos0 + p) * inv_freq[i], times attn_scale
 * Angles and functions are computed in float64 and rounded once.
 * Requirements: pos0, P >= 0, pos0 + P <= SPIN_KV_MAX_CONTEXT.
 */
spin_status spin_rope_table(const double* inv_freq, int n, int pos0, int P, double attn_scale, float* table,
                            void* stream);

/*
 * spin_kv_append — the KV step of an attention layer on the rows qkv_proj
 * wrote: norms of the heads, position rotation, R3, and the codes of keys and
 * values into the paged cache, in one launch (page "SpinQuant, Reproduced",
 * Q5: R3 rotates queries and keys online, after the position rotation, with
 * which it does not commute; abstract: 4-bit KV cache).
 *
 *   Q, K, V   [T] rows of Hq (Hkv) vectors of D = 128 values, float32 or
 *             float16; q_stride, k_stride, v_stride values from a token to the
 *             next (of the [T][(Hq + 2 Hkv) 128] product of qkv_proj:
 *             (Hq + 2 Hkv) 128 for each).  Q and Q_out may both be NULL.
 *   q_norm, k_norm  [128] float32 or NULL: x <- x / sqrt(mean(x^2) + eps) * w,
 *             per head
 *   rope      [rope_len][rot_dim] float32 from spin_rope_table, or NULL with
 *             rot_dim 0: the first rot_dim values of a head are turned in pairs
 *             (i, i + rot_dim / 2) (interleaved 0) or (2 i, 2 i + 1)
 *             (interleaved 1) by the row of the token's position, pos0 + place;
 *             rot_dim a multiple of 16 up to 128.  pos0 is 0, or the length of a
 *             prefix that lies in other pages (spin_kv_attn_shared).
 *   K_codes, K_scale, V_codes, V_scale, bits   the cache   UPDATED: codes of
 *             the keys, y = x . H_128 / sqrt(128) after norm and rotation, and
 *             of the values as they are, by the rules of spin_kv_quant at 4 and
 *             spin_kv_quant8 at 8 bits.  y is computed in float64 and rounded
 *             once to float32, which is what is quantized.
 *   Q_out     [T][Hq][128] fp16   OUTPUT: the queries, the same way, rounded
 *             (float32 sums)
 * A token whose place is negative, beyond its table, or whose position has no
 * row in rope, is not stored, and its queries are zeros; one whose page is not
 * in the pool is not stored.
 * Requirements: T, B >= 0, strides >= the heads' values, multiples of 16 bytes
 * and at most 2^40, pages as above, at most 2^24 - 1 workgroups of 16 vectors.
 * Errors: SPIN_ERR_NULL (a Q / Q_out pair with one NULL, rope without rot_dim),
 * SPIN_ERR_UNSUPPORTED (dtype, bits, interleaved, an eps that is negative or
 * not finite), SPIN_ERR_BAD_SHAPE, SPIN_ERR_MISALIGNED (every pointer 16 bytes).
 */
spin_status spin_kv_append(const void* Q, const void* K, const void* V, spin_dtype x_dtype, int T, int Hq, int Hkv,
                           int D, int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_norm,
                           const float* k_norm, float eps, const float* rope, int rope_len, int rot_dim,
                           int interleaved, int pos0, int bits, uint8_t* K_codes, uint16_t* K_scale,
                           uint8_t* V_codes, uint16_t* V_scale, int n_pages, int page_size, int B,
                           const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table, int max_pages,
                           uint16_t* Q_out, void* stream);

/*
 * spin_kv_append_at — spin_kv_append where `positions` [T] int32 says which
 * position each row is turned by (its row of rope), in place of pos0 + place: for
 * drafted tokens, which stand behind each other in the cache and beside each
 * other in the tree (spin_kv_tree), and for a cache that tokens have left
 * (spin_kv_choose), where places lag behind positions.  Places, pages and
 * everything else as there; a row whose position has no row in rope is one whose
 * position has none there.
 * Errors: as for spin_kv_append, SPIN_ERR_NULL without positions.
 */
spin_status spin_kv_append_at(const void* Q, const void* K, const void* V, spin_dtype x_dtype, int T, int Hq, int Hkv,
                              int D, int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* q_norm,
                              const float* k_norm, float eps, const float* rope, int rope_len, int rot_dim,
                              int interleaved, const int32_t* positions, int bits, uint8_t* K_codes,
                              uint16_t* K_scale, uint8_t* V_codes, uint16_t* V_scale, int n_pages, int page_size, int B,
                              const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table, int max_pages,
                              uint16_t* Q_out, void* stream);

/*
 * spin_kv_attn — attention of the new tokens of every sequence over its pages
 * (page "SpinQuant, Reproduced", Q5: queries and keys both carry R3, which
 * leaves their products unchanged; the values' R2 is undone in o_proj).
 * Prompts, chunks and single tokens may stand in one batch.
 *
 *   Q    [T][Hq][D] fp16 (from spin_kv_append), Hq a multiple of Hkv: query
 *        head h reads key head h / (Hq / Hkv)
 *   O    [T][Hq][D] fp16   OUTPUT: sum_j softmax_j(z) v_j over the visible
 *        tokens j, zeros where none is; k_j and v_j are code * scale
 *        z_j = scale * (q . k_j)
 *        z_j <- softcap * tanh(z_j / softcap)   where softcap > 0
 *        z_j <- z_j - slopes[h] * |p - j|       slopes [Hq] float32 or NULL
 *        for a query at position p, visible if j < kv_len[b], and
 *          causal 1: j <= p, or j < bidir_len[b] (bidir_len [B] int32 or NULL:
 *                    a prefix that every row sees whole); causal 0: any
 *          window > 0: |p - j| < window
 *   workspace  device memory of the bytes spin_kv_attn_workspace names (it may
 *        be NULL if that is 0); its content before and after means nothing,
 *        and calls that overlap need one each
 * Scores (with the logarithm of the value's scale added: a score of size z
 * carries it to 2^-24 z), maxima and sums are float32; a capped score is off by
 * 2^-18 of itself at most, at caps up to 64 by 2^-20 of the cap.  Softmax
 * weights are rounded to fp16 (relative to the row's largest weighted term) for
 * the product with the codes, which are exact.  A row that sees a token whose scale is not finite is NaN;
 * one that does not is not touched by it.  A row of Q that is not finite gives
 * NaN or zeros, and the others what they are without it, up to their rounding.
 * Errors: SPIN_ERR_NULL, SPIN_ERR_UNSUPPORTED (bits, causal, a scale that is
 * not finite, a softcap that is negative or not finite), SPIN_ERR_BAD_SHAPE
 * (also a workspace that is too small, Hkv above 65535, more than 2^22 - 1
 * workgroups or 2^26 rows of Q),
 * SPIN_ERR_MISALIGNED (every pointer 16 bytes).
 */
spin_status spin_kv_attn(const uint16_t* Q, int T, int Hq, int Hkv, int D, int bits, const uint8_t* K_codes,
                         const uint16_t* K_scale, const uint8_t* V_codes, const uint16_t* V_scale, int n_pages,
                         int page_size, int B, const int32_t* q_start, const int32_t* kv_len,
                         const int32_t* page_table, int max_pages, float scale, float softcap, const float* slopes,
                         int window, int causal, const int32_t* bidir_len, uint16_t* O, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * spin_kv_attn_shared — spin_kv_attn for sequences that all begin with the
 * same prefix_len tokens, whose pages prefix_table ([ceil(prefix_len /
 * page_size)] int32) names once.  Each sequence's own pages hold what follows:
 * places 0, 1, ... of its table are positions prefix_len, prefix_len + 1, ...
 * kv_len and the table count own tokens only; positions, window, bias and
 * bidir_len count from the prefix's first token.  The prefix is read once for
 * the rows of all sequences together.  The result is that of spin_kv_attn with
 * the prefix's pages in front of every table, up to rounding.
 * prefix_len 0 is spin_kv_attn.  Errors as there.
 */
spin_status spin_kv_attn_shared(const uint16_t* Q, int T, int Hq, int Hkv, int D, int bits, const uint8_t* K_codes,
                                const uint16_t* K_scale, const uint8_t* V_codes, const uint16_t* V_scale,
                                int n_pages, int page_size, const int32_t* prefix_table, int prefix_len, int B,
                                const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                                int max_pages, float scale, float softcap, const float* slopes, int window,
                                int causal, const int32_t* bidir_len, uint16_t* O, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Words of a row of the tree at most: 4096 drafted tokens of a sequence. */
#define SPIN_KV_TREE_MAX_WORDS 128

/*
 * spin_kv_tree — ancestors and positions of drafted tokens (speculative decoding:
 * several continuations of a sequence, as a tree, are verified in one step).
 *
 *   parent     [T] int32: of a sequence's i-th new token the number, among its new
 *              tokens, of the one before it in its continuation; -1 if that is the
 *              context's last.  A parent comes before its children; any value that
 *              is not in 0 .. i - 1 counts as -1.
 *   tree       [T][words] uint32   OUTPUT: bit i % 32 of word i / 32 of a row is set
 *              if new token i of its sequence is the row's token or one of its
 *              ancestors
 *   positions  [T] int32   OUTPUT: pos0 + the context's tokens (kv_len less the new
 *              ones) + the token's depth (0 with parent -1)
 * New tokens of a sequence from 32 words on have rows of zeros and depth 0; nobody
 * sees them.  Rows of no sequence are not written.
 * Requirements: 0 <= T <= 2^26, B >= 0, 0 <= pos0 <= SPIN_KV_MAX_CONTEXT,
 * 1 <= words <= SPIN_KV_TREE_MAX_WORDS.
 * Errors: SPIN_ERR_NULL, SPIN_ERR_UNSUPPORTED (tree or positions that overlap parent),
 * SPIN_ERR_BAD_SHAPE, SPIN_ERR_MISALIGNED.
 */
spin_status spin_kv_tree(const int32_t* parent, int T, int B, const int32_t* q_start, const int32_t* kv_len, int pos0,
                         int words, uint32_t* tree, int32_t* positions, void* stream);

/*
 * spin_kv_attn_ex — spin_kv_attn_shared (spin_kv_attn at prefix_len 0) with two
 * more things.
 *
 *   tree, tree_words, positions   tree non-NULL: which of its sequence's new tokens
 *        a row sees ([T][tree_words] uint32 as spin_kv_tree writes them; any bits
 *        are taken).  It sees the prefix and the context, all tokens before the
 *        sequence's first new one, as well; a row whose bits are all zero sees
 *        nothing else.  `causal` is then of no effect, and bidir_len NULL.  Distances,
 *        of the window and the bias, go by positions [T] int32 for the rows and
 *        the new tokens (held to 0 .. 2^30), by places (behind the prefix) for the
 *        context's tokens; positions may be NULL without a window and slopes.
 *        Bits of new tokens that have no place are of no effect.
 *   lse  [T][Hq] float32 or NULL   OUTPUT: the natural logarithm of the sum of e^z
 *        over the tokens that the row sees, -infinity where there is none; not
 *        finite for a row that sees a scale that is not finite, or is not finite
 *        itself.  For spin_kv_weights.  It is as far off as attention's scores are,
 *        whose products with 4-bit codes are rounded more than those of
 *        spin_kv_weights: at queries of 2 and scales up to 0.5, on 300 to 4000 tokens,
 *        by 3e-5 at most and 9e-6 rms (8 bits: 3e-6 and 1e-6).  A weight taken with it
 *        is off by as much of itself; with exact logarithms by 2e-6 at most.
 * tree NULL and lse NULL: the bits of spin_kv_attn_shared.  The workspace is the same.
 * Errors: as for spin_kv_attn_shared; SPIN_ERR_NULL for a tree without positions
 * where a window or slopes need them, SPIN_ERR_UNSUPPORTED for a tree with
 * bidir_len, SPIN_ERR_BAD_SHAPE for tree_words outside 1 .. SPIN_KV_TREE_MAX_WORDS.
 */
spin_status spin_kv_attn_ex(const uint16_t* Q, int T, int Hq, int Hkv, int D, int bits, const uint8_t* K_codes,
                            const uint16_t* K_scale, const uint8_t* V_codes, const uint16_t* V_scale, int n_pages,
                            int page_size, const int32_t* prefix_table, int prefix_len, int B, const int32_t* q_start,
                            const int32_t* kv_len, const int32_t* page_table, int max_pages, float scale,
                            float softcap, const float* slopes, int window, int causal, const int32_t* bidir_len,
                            const uint32_t* tree, int tree_words, const int32_t* positions, uint16_t* O, float* lse,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * spin_kv_weights — the attention weight that every cached token of a sequence
 * draws, for eviction from the cache.
 *
 *   Q, lse   [T][Hq][D] fp16 and [T][Hq] float32: queries, and the logarithms that
 *            spin_kv_attn_ex left for them (with the same scale, softcap, slopes,
 *            window, causal and bidir_len)
 *   pos0     position of the first token of the tables: 0, or the length of a prefix
 *            in other pages
 *   prior    [n_pages][Hkv][page_size] float32 or NULL; W itself is allowed.  It has to
 *            hold a weight for every token, new ones among them (spin_kv_weights_ex)
 *   W        [n_pages][Hkv][page_size] float32   OUTPUT: at the slot of every token
 *            j < kv_len[b] of every sequence, per key head
 *              W_j = decay * prior_j + sum over rows and heads of e^(z_j - lse)
 *            over the sequence's rows and the query heads of the key head that see
 *            the token (without prior, the sum alone).  Other slots keep what they
 *            hold.
 *   workspace  device memory of the bytes spin_kv_weights_workspace names (it may
 *            be NULL if that is 0); its content before and after means nothing, and
 *            calls that overlap need one each
 * Rows are a sequence's last tokens, in order, or some of its last ones.  Of a
 * drafted tree the accepted rows are passed, behind spin_kv_move: the logarithms
 * that the tree's attention left for them are the plain sequence's.
 * A row whose lse is not finite adds nothing, and a token whose scale is not finite
 * draws nothing.  Sums are float32, in an order that goes by the sizes alone.  A page
 * may stand in one table of the batch only.  T == 0 is valid: W = decay * prior.
 * Errors: as for spin_kv_attn; SPIN_ERR_UNSUPPORTED for a decay that is not finite
 * and a prior that overlaps W in part, SPIN_ERR_BAD_SHAPE for more than 2^24 - 1
 * workgroups of 128 of a head's tokens.
 */
spin_status spin_kv_weights(const uint16_t* Q, const float* lse, int T, int Hq, int Hkv, int D, int bits,
                            const uint8_t* K_codes, const uint16_t* K_scale, int n_pages, int page_size, int B,
                            const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table, int max_pages,
                            int pos0, float scale, float softcap, const float* slopes, int window, int causal,
                            const int32_t* bidir_len, const float* prior, float decay, float* W, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * spin_kv_weights_ex — spin_kv_weights where prior_len [B] int32 says how many of
 * each sequence's tokens, the first ones, have a prior; that of the others is 0, and
 * what prior holds at their slots is not read.  NULL: all have one.
 *
 * A slot outlives its token: what W held of a token that has left (spin_kv_choose,
 * spin_kv_move) or of another sequence's, whose pages came back, is there still when
 * new tokens are appended to that slot.  In a loop that adds up weights prior_len is
 * the length that the last call of the sequence saw, or that spin_kv_choose left of
 * it since, and 0 for a sequence that has had none.
 * Errors: as for spin_kv_weights.
 */
spin_status spin_kv_weights_ex(const uint16_t* Q, const float* lse, int T, int Hq, int Hkv, int D, int bits,
                               const uint8_t* K_codes, const uint16_t* K_scale, int n_pages, int page_size, int B,
                               const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                               int max_pages, int pos0, float scale, float softcap, const float* slopes, int window,
                               int causal, const int32_t* bidir_len, const float* prior, const int32_t* prior_len,
                               float decay, float* W, void* workspace, size_t workspace_bytes, void* stream);

/*
 * spin_kv_weights_workspace — bytes of workspace a spin_kv_weights or
 * spin_kv_weights_ex call of these sizes takes (0: none).  It goes by the sizes alone.
 */
spin_status spin_kv_weights_workspace(int T, int Hq, int Hkv, int B, int max_pages, int page_size, size_t* bytes);

/*
 * spin_kv_choose — which tokens of each sequence stay, per key head: those of
 * greatest weight.
 *
 *   W      [n_pages][Hkv][page_size] float32 (from spin_kv_weights)
 *   keep   how many stay of a longer sequence, 1 or more; its first `first` and its last
 *          `recent` tokens are always among them (first + recent <= keep)
 *   kept   [B][Hkv][keep] int32   OUTPUT: their places, ascending, -1 behind the
 *          places of a sequence that has no more than keep tokens (all stay)
 *   lens   [B] int32   OUTPUT: how many stay, min(kv_len[b], keep); kv_len itself is
 *          allowed (the lengths are then replaced, in a launch of their own)
 * Of equal weights the lowest place stays (-0 equals 0).  NaN, and a token
 * that lies in no page of the pool, are below all weights.
 *   workspace  device memory of the bytes spin_kv_choose_workspace names (it may be
 *          NULL if that is 0); its content before and after means nothing, and calls
 *          that overlap need one each
 * Errors: SPIN_ERR_NULL, SPIN_ERR_UNSUPPORTED (lens that overlaps kv_len in part),
 * SPIN_ERR_BAD_SHAPE (also a workspace that is too small, and more than 2^22 - 1
 * sequences times heads, of tables above 32768 tokens a third of that, or as many
 * times 8192 tokens), SPIN_ERR_MISALIGNED.
 */
spin_status spin_kv_choose(const float* W, int Hkv, int n_pages, int page_size, int B, const int32_t* kv_len,
                           const int32_t* page_table, int max_pages, int keep, int first, int recent, int32_t* kept,
                           int32_t* lens, void* workspace, size_t workspace_bytes, void* stream);

/*
 * spin_kv_choose_workspace — bytes of workspace a spin_kv_choose call of these sizes
 * takes (0: none, up to 32768 tokens a table).  It goes by the sizes alone.
 */
spin_status spin_kv_choose_workspace(int Hkv, int B, int max_pages, int page_size, size_t* bytes);

/*
 * spin_kv_move — tokens of the cache to other slots, codes and scales as they are.
 *
 *   kept   [B][kept_heads][n] int32, kept_heads 1 (all heads alike) or Hkv: the token
 *          at place at[b] + kept[b][h][i] goes to place at[b] + i; entries below 0
 *          are passed over.  at [B] int32, NULL for 0.
 *   to_table   [B][to_pages] int32: the pages that it goes to, none of which may be
 *          one that tokens of this call come from.  NULL, or page_table
 *          again: places of page_table itself; with B == 1 to_pages may then differ from
 *          max_pages (the first pages of the row alone).  The entries of a list (but for
 *          those below 0) then ascend, and kept[b][h][i] >= i: the tokens that spin_kv_choose
 *          names, or the accepted path of a tree behind at[b] tokens of context.
 *          (With other lists the slots hold wrong tokens.)
 *   W      [n_pages][Hkv][page_size] float32 or NULL: moves with the tokens
 * A page that tokens go to may stand in one table of the call only; another sequence
 * that reads it (a shared prefix in the tables) sees what is moved there.
 * A token that comes from or goes to a place beyond its table, or a page that is
 * none of the pool, is passed over.  Slots that nothing goes to keep what they hold,
 * their weights too, which are not those of tokens that come there later
 * (spin_kv_weights_ex).
 * Position rotations are in the keys, so that a token keeps its position wherever it
 * lies; what attention takes from places (windows, distances, causal order among new
 * tokens) goes by the new ones.
 * Errors: SPIN_ERR_NULL, SPIN_ERR_UNSUPPORTED (bits), SPIN_ERR_BAD_SHAPE (also more
 * than 2^24 - 1 groups of 64 tokens of a head, and page_table again for several
 * sequences with another number of pages), SPIN_ERR_MISALIGNED (16 bytes; 4
 * for page_table, kept, at and to_table, which are cut out of longer lists).
 */
spin_status spin_kv_move(uint8_t* K_codes, uint16_t* K_scale, uint8_t* V_codes, uint16_t* V_scale, float* W, int Hkv,
                         int D, int bits, int n_pages, int page_size, int B, const int32_t* page_table, int max_pages,
                         const int32_t* kept, int kept_heads, int n, const int32_t* at, const int32_t* to_table,
                         int to_pages, void* stream);

/*
 * spin_kv_attn_workspace — bytes of workspace a spin_kv_attn (prefix_len 0) or
 * spin_kv_attn_shared (or spin_kv_attn_ex) call of these sizes takes.  It goes by the sizes alone,
 * not by what the arrays on the device hold.
 */
spin_status spin_kv_attn_workspace(int T, int Hq, int Hkv, int B, int max_pages, int page_size, int prefix_len,
                                   size_t* bytes);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* spin_status_string(spin_status s);

/* Library version as MAJOR * 10000 + MINOR * 100 + PATCH. */
int spin_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBSPIN_H */
