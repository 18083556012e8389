/*
 * qopt_fp4.h -- C ABI of the 4-bit floating point products in libqopt.so, for AMD Instinct
 * MI355X (gfx950): a quantizer of 32-value blocks, its inverse, and the matrix products over
 * its codes.
 *
 * The format is the microscaled 4-bit format of the OCP Microscaling specification (MXFP4):
 * e2m1 codes with one power-of-two scale per 32 values.  It stands next to the 8-bit products of
 * qopt_fp8.h: half the bytes of a weight, and twice their rate in the matrix units.
 *
 * A quantized matrix [rows, cols] is a pair (codes, scales):
 *   codes   row-major [rows, kp / 2] bytes, kp = cols rounded up to a multiple of 256: the
 *           code of an even column in the low half of a byte, that of the odd column behind it
 *           in the high half; codes behind a row's end are 0.  A code is a sign (8) and the number
 *           of a magnitude: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   scales  [kp / 128, rp, 4] bytes, rp = rows rounded up to a multiple of 16: byte [i, r, j]
 *           belongs to columns 128 i + 32 j to 128 i + 32 j + 31 of row r and stands for
 *           2^(s - 127); 255 makes the whole block NaN.  (The four scales of a row's 128 values
 *           are one word, and the words of consecutive rows lie side by side, as a product
 *           reads them.)
 *
 * Conventions are those of qopt.h (status codes, dtypes, *_dev pointers in device memory
 * of the current HIP device, caller-owned buffers, host-side argument checks before
 * anything is enqueued, asynchronous work on `stream`).  Every entry point may be
 * captured into a graph.  Sizes are at most QOPT_FP4_MAX_DIM each, and a matrix of
 * more than 2^22 tiles of 128 x 128 is refused (QOPT_EINVAL).
 */
#ifndef QOPT_FP4_H
#define QOPT_FP4_H

#include <stddef.h>
#include <stdint.h>

#include "qopt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values per block along the axis that a product sums over. */
#define QOPT_FP4_BLOCK 32
/* A row of codes is padded to a multiple of so many values. */
#define QOPT_FP4_PAD 256
/* Largest number of rows or columns of a matrix here. */
#define QOPT_FP4_MAX_DIM 8388608
/* Up to this many rows qopt_fp4_linear quantizes and multiplies in one launch. */
#define QOPT_FP4_FEW_ROWS 32

/*
 * Quantize x_dev [rows, cols] (dtype QOPT_F32 or QOPT_BF16, rows ldx >= cols elements apart).
 * For a block with the largest magnitude A: e = the least integer with A <= 6 * 2^e, at least
 * -127 (0 when A = 0); its scale byte is e + 127 and each code is x * 2^-e rounded to e2m1, ties
 * to the even code.  A block with an infinity or a NaN has scale 255 and codes 0.
 * codes_dev is 16-byte aligned, scales_dev 4-byte.  The outputs must not overlap x or each
 * other; all of them is written, padding included (codes 0, scales 127).  rows or cols 0: nothing
 * is written.
 * Errors: QOPT_EINVAL (null pointers with elements, sizes negative or too large, ldx < cols),
 * QOPT_EUNSUPPORTED (dtype), QOPT_EALIGN, QOPT_ELAUNCH.
 */
int qopt_fp4_quantize(const void* x_dev, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                      uint8_t* codes_dev, uint8_t* scales_dev, void* stream);

/*
 * out_dev [rows, cols] (dtype, rows ldo >= cols elements apart): the values that codes and scales
 * stand for, exactly where the type holds them (a code of 4 or 6 at the largest scales is an
 * infinity, values below the subnormals round).
 */
int qopt_fp4_dequantize(const uint8_t* codes_dev, const uint8_t* scales_dev, int64_t rows,
                        int64_t cols, void* out_dev, int dtype, int64_t ldo, void* stream);

/*
 * out[i, j] = sum over l < k of A[i, l] * B[j, l]: the product of a quantized A [m, k] with the
 * transpose of a quantized B [n, k], in out_dtype (QOPT_F32 or QOPT_BF16).  The products of one
 * block's codes are exact, sums are binary32 in a fixed order (equal calls give equal bits) and
 * rounded once.  Products of two elements under 2^-126 may count as 0.
 * A NaN block makes its whole row (of A) or column (of B) of the result NaN.
 * out_dev: rows ldo >= n elements apart; elements between n and ldo are left as they are.  It
 * must not overlap an operand.
 * workspace_dev: at least qopt_fp4_matmul_workspace(m, n, k, ...) bytes, 16-byte aligned
 * (NULL if that is 0); scratch whose contents need no preparation, for one call at a time.
 * m or n 0: nothing is written; k 0: out is all 0.
 * Errors as for qopt_fp4_quantize, and QOPT_EINVAL for a workspace that is too small.
 */
int qopt_fp4_matmul(const uint8_t* a_codes_dev, const uint8_t* a_scales_dev,
                    const uint8_t* b_codes_dev, const uint8_t* b_scales_dev, int64_t m, int64_t n,
                    int64_t k, void* out_dev, int out_dtype, int64_t ldo, void* workspace_dev,
                    size_t workspace_bytes, void* stream);
int qopt_fp4_matmul_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes);

/*
 * out = x w^T for x_dev [m, k] as it is and a quantized w [n, k]: x is quantized as
 * qopt_fp4_quantize does, then multiplied.  Up to QOPT_FP4_FEW_ROWS rows that is one launch, in
 * which the weights are read once; above, the result is that of the two calls.
 * workspace_dev as above, of qopt_fp4_linear_workspace bytes.
 */
int qopt_fp4_linear(const void* x_dev, int dtype, int64_t m, int64_t k, int64_t ldx,
                    const uint8_t* w_codes_dev, const uint8_t* w_scales_dev, int64_t n,
                    void* out_dev, int out_dtype, int64_t ldo, void* workspace_dev,
                    size_t workspace_bytes, void* stream);
int qopt_fp4_linear_workspace(int64_t m, int64_t n, int64_t k, int out_dtype, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* QOPT_FP4_H */
