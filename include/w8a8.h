/*
 * w8a8.h -- 8-bit floating-point (e4m3) products with block scales, and the
 * operators that make their activations, beside the W4A16 ones of w4a16.h:
 *
 *     w8a8_rms_norm      residual addition and RMS norm, rows in e4m3 with scales
 *     w8a8_quantize      rows, or silu(gate) * up of rows, in e4m3 with scales
 *     w8a8_gemm          Y = X . W^T, both in e4m3
 *     w8a8_gemm_grouped  the same by expert, on the slot lists of w4a16_moe_route
 *     w8a8_quantize_weights  weights to e4m3 with block scales, on the host
 *
 * The format: e4m3 has a sign, 4 exponent bits (bias 7) and 3 mantissa bits; its
 * largest value is 448, it has no infinities, and codes 0x7F and 0xFF are NaN.
 * One fp32 scale stands for 128 neighbouring features of one activation row, and
 * for a block of 128 x 128 of the weights:
 *   X   uint8 [M][K]   codes     xs  float [M][KB]      KB = ceil(K / 128)
 *   W   uint8 [N][K]   codes     ws  float [NB][KB]     NB = ceil(N / 128)
 *   value of X[m][k] = e4m3(X[m][k]) * xs[m][k / 128],
 *   value of W[n][k] = e4m3(W[n][k]) * ws[n / 128][k / 128].
 * All arrays are row-major and contiguous.  K is a multiple of 16 (rows of codes
 * begin at 16-byte addresses); its last block may be shorter than 128, and so may
 * N's last.
 *
 * Memory, errors, streams, status codes and W4A16_DTYPE_* are those of w4a16.h:
 * pointers are DEVICE memory owned by the caller (w8a8_quantize_weights: HOST),
 * nothing is allocated, no workspace is needed, nothing waits for the GPU, every
 * call can be captured into a HIP graph, argument errors are found on the host
 * before anything is launched, and results do not depend on timing.
 */
#ifndef W8A8_H
#define W8A8_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

#define W8A8_BLOCK 128
/* Largest extents; M, R and T are rows. */
#define W8A8_MAX_M ((int64_t)1 << 30)
#define W8A8_MAX_N ((int64_t)1 << 30)
#define W8A8_MAX_K W4A16_MAX_K
/* widest row of w8a8_rms_norm (a row is held in one workgroup's registers) */
#define W8A8_NORM_MAX_K ((int64_t)1 << 15)

/*
 * Quantize fp32 weights W[N][K] (HOST memory) into codes[N][K] and
 * scales[NB][KB] (HOST memory, caller-allocated).  Per block of 128 x 128, a the
 * block's largest magnitude: scale = 0 if a is 0, else a / 448 (fp32 division), at
 * least 2^-126; code = w / scale (fp32 division) to the nearest e4m3 value, ties to
 * even, magnitudes past 448 to 448; +0 where the scale is 0.  Synchronous, no GPU use.
 * W4A16_ERR_NONFINITE (outputs untouched) if a weight is NaN or infinite,
 * W4A16_ERR_SHAPE if K % 16 != 0 or an extent is past its limit, W4A16_ERR_ARG on
 * NULL pointers, negative extents, K == 0 or block != 128.  N == 0 is a no-op.
 */
int w8a8_quantize_weights(const float *W, uint8_t *codes, float *scales, int64_t N, int64_t K,
                          int32_t block);

/*
 * Rows to e4m3: for every run of 128 features of a row (the last may be shorter),
 * v its values in fp32 and a their largest magnitude,
 *     scale = 0 if a is 0, else a / 448, at least 2^-126,
 *     code  = v / scale to the nearest e4m3 value, ties to even.
 * v / scale is formed in fp32: within 2^-23 of its value of a tie the code may be
 * either neighbour's.  A run that holds an infinity or
 * NaN has a NaN scale and NaN codes.
 *   X         [M][K], or [M][2K] with swiglu; dtype
 *   num_rows  int32 [1]  rows in use, clamped to [0, M]; NULL: all M.  Rows of codes
 *                        and scales from there on are left as they were.
 *   codes     uint8 [M][K], scales float [M][KB]
 * swiglu != 0: v = g / (1 + exp(-g)) * u in fp32, g the row's first K values and u the
 * others (what a gate/up product of 2K rows gives), within 4 units of 2^-23 and 2^-148 |u|;
 * below g = -88.72, where exp(-g) passes fp32's range, v is 0; an infinite g of the sign
 * where the definition is 0 times infinity gives NaN.
 * M == 0 is a no-op.  W4A16_ERR_ARG for a NULL pointer (num_rows may be), an unknown
 * dtype, negative extents, K == 0 or an output that overlaps an input or the other
 * output; W4A16_ERR_SHAPE for K % 16 != 0 or an extent past W8A8_MAX_*;
 * W4A16_ERR_ALIGN for X or codes not 16-byte aligned or others not 4.
 */
int w8a8_quantize(const void *X, const int32_t *num_rows, uint8_t *codes, float *scales,
                  int64_t M, int64_t K, int32_t swiglu, int32_t dtype, void *stream);

/*
 * Residual addition, root-mean-square norm and quantization:
 *     h = X + residual                      (fp32; residual may be NULL: h = X)
 *     y = h * weight / sqrt(mean(h^2) + eps)   (fp32)
 *     H = h, Y = y rounded to dtype; codes, scales = y as w8a8_quantize
 * y comes from h before H's rounding.  Sums of squares past fp32's range (with eps), or
 * far below its least, are formed from the row scaled by a power of two.  As the formula
 * has it, an infinity in h gives NaN there and 0 in the rest of its row, a NaN gives
 * NaN in all of it.
 *   X, residual  [M][K], dtype; weight [K], weight_dtype (dtype or W4A16_DTYPE_F32)
 *   H            [M][K], dtype, or NULL; may be X or residual themselves
 *   Y            [M][K], dtype, or NULL
 *   codes, scales  as w8a8_quantize, or both NULL
 * M == 0 is a no-op.  W4A16_ERR_ARG where no output is asked for, one of codes and
 * scales is NULL, eps is not positive and finite, weight_dtype is another, or an output
 * overlaps an input (H: otherwise than by being it) or another output; W4A16_ERR_SHAPE
 * also for K > W8A8_NORM_MAX_K or rows that would take 2^32 threads or more (64 a row
 * up to K = 2048, 256 up to 8192, 1024 past that); W4A16_ERR_ALIGN for X, residual,
 * weight, H, Y or codes not 16-byte aligned; otherwise as w8a8_quantize.
 */
int w8a8_rms_norm(const void *X, const void *residual, const void *weight, void *H, void *Y,
                  uint8_t *codes, float *scales, int64_t M, int64_t K, float eps, int32_t dtype,
                  int32_t weight_dtype, void *stream);

/*
 * Y[M][N] = X . W^T, the values of X and W as above:
 *     Y[m][n] = sum over b of xs[m][b] * ws[n / 128][b] * (sum over k in block b of
 *               e4m3(X[m][k]) * e4m3(W[n][k])),
 * added up in fp32 and rounded once to dtype (W4A16_DTYPE_*).  Every product is exact
 * in fp32.  With 16-bit outputs the kernel for many rows (W8A8_KERNEL_TILE) adds products
 * 8 at a time, cut off 13 bits below the largest one's power of two: at most 7 * 2^-13 of
 * sum |x w| off, in the root mean square 2^-16 of the result for normally distributed
 * values (2^-14.5 where a hundredth of the activations is 20 times the others, 2^-14 where
 * that holds for the weights as well).  That adds 0.2% to the error of stored fp16 results
 * (1.2%, 4%; 6.5% with a twentieth of both operands 50 times the others), and at most 0.1% to
 * bf16's.  fp32 outputs, and any of W8A8_KERNEL_SKINNY, have no such cut; who wants 16-bit
 * results without it takes fp32 ones and rounds them.  So a row's result may differ by it,
 * beside fp32 sums' order, between a call of few rows and one of many.
 * The scales' products xs * ws are formed in fp32 and have to stay in its normal range.
 * A NaN code or scale gives NaN in the outputs that it enters.
 * Which kernel runs: w8a8_kernel.  M == 0 or N == 0 is a no-op.  W4A16_ERR_ARG for
 * NULL pointers, negative extents, K == 0, block != 128, an unknown dtype or Y
 * overlapping an input; W4A16_ERR_SHAPE for K % 16 != 0, an extent past W8A8_MAX_*, or
 * where tiles of every size would take 2^32 threads or more (W8A8_KERNEL_SKINNY has one size,
 * 16 rows of W by 512 threads, by expert 32 by 256); W4A16_ERR_ALIGN for X or W not
 * 16-byte aligned, the scales not 4 and Y not to its elements.
 */
int w8a8_gemm(const uint8_t *X, const float *xs, const uint8_t *W, const float *ws, void *Y,
              int64_t M, int64_t N, int64_t K, int32_t block, int32_t dtype, void *stream);

/*
 * w8a8_gemm by expert: Y[r] = X[token_index[r]] . W_e^T for slot r of expert e.
 *   X               uint8 [T][K], xs float [T][KB]   tokens
 *   token_index     int32 [R], or NULL: slot r reads row r (T >= R)
 *   expert_offsets  int32 [E+1]  as w4a16_gemm_grouped; offsets[E] may be below R:
 *                                rows of Y from offsets[E] on are left as they were
 *   W               uint8 [E][N][K], ws float [E][NB][KB]
 *   Y               [R][N], dtype
 * token_index and expert_offsets are clamped into range on the device (malformed lists
 * give wrong values, never an access out of bounds).  The weights of an expert without
 * slots are not read.  R == 0 or N == 0 is a no-op; T == 0 with R > 0, or T < R without
 * token_index, is W4A16_ERR_ARG; E < 1 W4A16_ERR_ARG, E > 65535 W4A16_ERR_SHAPE;
 * otherwise errors as w8a8_gemm.
 */
int w8a8_gemm_grouped(const uint8_t *X, const float *xs, const int32_t *token_index,
                      const int32_t *expert_offsets, const uint8_t *W, const float *ws, void *Y,
                      int64_t T, int64_t R, int64_t E, int64_t N, int64_t K, int32_t block,
                      int32_t dtype, void *stream);

/* Kernels behind w8a8_gemm and w8a8_gemm_grouped. */
#define W8A8_KERNEL_SKINNY 1 /* few rows: weights and activations from memory to registers,
                                  fp16 matrix instructions on the exact codes */
#define W8A8_KERNEL_TILE 2   /* many: tiles through LDS; 16-bit outputs on the fp8 matrix
                                instructions, fp32 outputs on fp16 ones */

/* The kernel (one of W8A8_KERNEL_*) of w8a8_gemm for R rows (E = 0), or of
 * w8a8_gemm_grouped for R slots over E experts: the skinny one for up to 4 rows, or 10 slots
 * per expert (of the fewer of R and E).  With it a slot's result does not depend on the other
 * slots of the call.  0 for extents that are refused or a no-op.  Host only. */
int w8a8_kernel(int64_t R, int64_t E);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H */
