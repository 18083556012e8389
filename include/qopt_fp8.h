/*
 * qopt_fp8.h -- C ABI of the 8-bit floating point products in libqopt.so, for AMD
 * Instinct MI355X (gfx950): a quantizer of 128-value blocks and the matrix products
 * over its codes.
 *
 * They carry the block-wise idea of the 8-bit optimizers summary page
 * (wiki.neutronadmin.com/news/16836, §2 "Block-wise Quantization": blocks normalised by
 * their own absmax, so that an outlier only affects its own block) from the optimizer's
 * state to the products of a linear layer: y = x w^T, dx = dy w, dw = dy^T x.
 *
 * A quantized matrix is a pair (codes, scales):
 *   codes   e4m3 bytes, row-major [rows, kp], kp = cols rounded up to a multiple of 128,
 *           the bytes behind a row's end 0;
 *   scales  one byte s (0 .. 247) per block, standing for 2^(s - 127):
 *           QOPT_FP8_ROWS   a block is 128 consecutive values of a row:
 *                           [kp / 128, rp], rp = rows rounded up to a multiple of 16: the
 *                           scales of consecutive rows lie side by side, as a product
 *                           reads them (those from rows on are not read for a result)
 *           QOPT_FP8_TILES  a block is a tile of 128 x 128 values:
 *                           [ceil(rows / 128), kp / 128]
 * An element is the value of its code times its block's 2^(s - 127).
 * Powers of two make every scaling exact, are what the scaled matrix instructions take,
 * and let one quantization of a weight serve both its orientations.
 *
 * Conventions are those of qopt.h (status codes, dtypes, *_dev pointers in device memory
 * of the current HIP device, caller-owned buffers, host-side argument checks before
 * anything is enqueued, asynchronous work on `stream`).  Every entry point may be
 * captured into a graph.  Sizes are at most QOPT_FP8_MAX_DIM each, and a matrix of
 * more than 2^22 tiles of 128 x 128 is refused (QOPT_EINVAL).
 */
#ifndef QOPT_FP8_H
#define QOPT_FP8_H

#include <stddef.h>
#include <stdint.h>

#include "qopt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values per block along the axis that a product sums over. */
#define QOPT_FP8_BLOCK 128
/* Largest number of rows or columns of a matrix here. */
#define QOPT_FP8_MAX_DIM 8388608
/* Up to this many rows qopt_fp8_linear quantizes and multiplies in one launch. */
#define QOPT_FP8_FEW_ROWS 32

typedef enum { QOPT_FP8_ROWS = 0, QOPT_FP8_TILES = 1 } qopt_fp8_form;

/*
 * Quantize x_dev [rows, cols] (dtype QOPT_F32 or QOPT_BF16, rows ldx >= cols elements
 * apart) and, at the same time, its transpose.  For a block with the largest finite
 * magnitude A: e = the least integer with A <= 448 * 2^e, at least -127 (0 when A = 0);
 * its scale byte is e + 127 and each code is x * 2^-e rounded to e4m3, ties to even.
 * Infinities and NaN become the NaN code and leave the block's scale to its finite values.
 *   codes_dev, scales_dev      the matrix [rows, cols] in `form`, or both NULL;
 *   codes_t_dev, scales_t_dev  its transpose [cols, rows] in `form`, or both NULL
 *                              (blocks along the rows of the transpose; the tiles of
 *                              QOPT_FP8_TILES are the same ones, so their codes are too).
 * Codes are 16-byte aligned.  The outputs must not overlap x or each other.  rows or cols 0: nothing is written.
 * Errors: QOPT_EINVAL (null x with elements, no output or half of one, sizes negative
 * or too large, ldx < cols), QOPT_EUNSUPPORTED (dtype, form), QOPT_EALIGN, QOPT_ELAUNCH.
 */
int qopt_fp8_quantize(const void* x_dev, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                      int form, uint8_t* codes_dev, uint8_t* scales_dev, uint8_t* codes_t_dev,
                      uint8_t* scales_t_dev, void* stream);

/*
 * out[i, j] = sum over l < k of A[i, l] * B[j, l]: the product of a quantized A [m, k]
 * with the transpose of a quantized B [n, k], A in QOPT_FP8_ROWS and B in `b_form`.  Sums
 * are binary32 and rounded once, to out_dtype, and their order is fixed: equal calls give
 * equal bits.  Codes are 16-byte aligned, scales 4-byte.
 *   out_dtype QOPT_BF16: 8-bit matrix instructions.  Of every 8 places that follow each other they
 *     cut the products toward zero at 2^-13 of the largest one's power of two, so the error goes by
 *     the operands, not by the result: for every 8 places at most 2^-10 of the product of the two
 *     operands' largest magnitudes there (each counted as 2^-6 of its scale at least), besides the
 *     rounding to bf16.  That is 1.2e-5 to 1.8e-5 of the result's size on normal data and, where
 *     no products cancel and none are that small, at most 2^-10 of it; where large products cancel
 *     it may be all that is left.
 *   out_dtype QOPT_F32: the codes are widened to bf16, exactly, and multiplied by the
 *     bf16 matrix instructions, whose products and sums are binary32.  Element values
 *     under 2^-126 may count as 0 here, and 2^128, to which magnitudes from 1.9375 * 2^127 on
 *     round, counts as an infinity.
 * A NaN element makes its whole row (of A) or column (of B) of the result NaN.
 * out_dev: rows ldo >= n elements apart; elements between n and ldo are left as they are.  It
 * must not overlap an operand.
 * workspace_dev: at least qopt_fp8_matmul_workspace(m, n, k, ...) bytes, 16-byte aligned
 * (NULL if that is 0); scratch whose contents need no preparation, for one call at a time.
 * m or n 0: nothing is written; k 0: out is all 0.
 * Errors as for qopt_fp8_quantize, and QOPT_EINVAL for a workspace that is too small.
 */
int qopt_fp8_matmul(const uint8_t* a_codes_dev, const uint8_t* a_scales_dev,
                    const uint8_t* b_codes_dev, const uint8_t* b_scales_dev, int b_form, int64_t m,
                    int64_t n, int64_t k, void* out_dev, int out_dtype, int64_t ldo,
                    void* workspace_dev, size_t workspace_bytes, void* stream);
int qopt_fp8_matmul_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes);

/*
 * out = x w^T for x_dev [m, k] as it is and a quantized w [n, k]: x is quantized in rows
 * as qopt_fp8_quantize does, then multiplied.  Up to QOPT_FP8_FEW_ROWS rows that is one
 * launch, in which the weights are read once; above, the result is that of the two calls.
 * Instructions and precision by out_dtype are those of qopt_fp8_matmul.
 * workspace_dev as above, of qopt_fp8_linear_workspace bytes.
 */
int qopt_fp8_linear(const void* x_dev, int dtype, int64_t m, int64_t k, int64_t ldx,
                    const uint8_t* w_codes_dev, const uint8_t* w_scales_dev, int w_form, int64_t n,
                    void* out_dev, int out_dtype, int64_t ldo, void* workspace_dev,
                    size_t workspace_bytes, void* stream);
int qopt_fp8_linear_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* QOPT_FP8_H */
