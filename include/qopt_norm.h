/*
 * qopt_norm.h -- C ABI of the layer normalisation in libqopt.so, for AMD Instinct MI355X
 * (gfx950): the forward pass, and the backward pass with the reduction of the weight's and
 * the bias's gradients.
 *
 * The Stable Embedding layer (qopt_embedding.h) normalises rows that it looks up; here the
 * rows are an activation's, as in front of the products of qopt_fp8.h and qopt_fp4.h.
 *
 *   y[i, j] = (x[i, j] - mean_i) * rstd_i * w[j] + b[j]
 *   mean_i  = mean of x[i, :],  rstd_i = 1 / sqrt(mean of (x[i, :] - mean_i)^2 + eps)
 *
 * Statistics and sums are binary32, the variance is the mean of squared distances (no
 * difference of squares), and every result is rounded once, to its type.  So a row r times its
 * spread away from zero is off by the rounding of its mean, some r 2^-23 of its spread, and a row
 * whose squared distances sum to 2^128 or more has rstd 0 and comes out as b.  The order of
 * each sum depends on the sizes alone: equal calls give equal bits.
 *
 * Conventions are those of qopt.h (status codes, dtypes, *_dev pointers in device memory of
 * the current HIP device, host-side argument checks before anything is enqueued,
 * asynchronous work on `stream`).  Every entry point may be captured into a graph.
 */
#ifndef QOPT_NORM_H
#define QOPT_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "qopt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of values in a row. */
#define QOPT_NORM_MAX_DIM 8388608
/* Largest number of rows. */
#define QOPT_NORM_MAX_ROWS 1099511627776

/*
 * out_dev [rows, dim] (dtype, rows ldo >= dim elements apart) from x_dev [rows, dim] (dtype
 * QOPT_F32 or QOPT_BF16, rows ldx >= dim apart).
 *   w_dev, b_dev         [dim] in w_dtype (QOPT_F32 or QOPT_BF16); NULL counts as all 1, all 0
 *   mean_dev, rstd_dev   [rows] binary32, or NULL: not written
 * out must not overlap x, w or b, other than by lying in other columns of the rows.  A row with
 * an infinity or a NaN comes out NaN.  rows or dim 0: nothing is written.
 * Errors: QOPT_EINVAL (null x or out with elements, sizes negative or too large, a row
 * distance below dim, eps negative or not finite), QOPT_EUNSUPPORTED (dtypes), QOPT_EALIGN
 * (an address that is no multiple of its element's size), QOPT_ELAUNCH.
 */
int qopt_layer_norm_forward(const void* x_dev, int dtype, int64_t rows, int64_t dim, int64_t ldx,
                            const void* w_dev, const void* b_dev, int w_dtype, float eps,
                            void* out_dev, int64_t ldo, float* mean_dev, float* rstd_dev,
                            void* stream);

/*
 * Gradients for the upstream dout_dev [rows, dim] (x's dtype), from x and the statistics that
 * the forward pass saved.  With v = dout * w and h = (x - mean) rstd:
 *   dx = (v - mean of v - h * mean of v h) * rstd,  dw = sum over rows of dout h,
 *   db = sum over rows of dout
 * dx_dev [rows, dim] in x's dtype, dw_dev and db_dev [dim] in w_dtype (which applies to them
 * also where w_dev is NULL); each may be NULL and is not computed then.  They must not overlap
 * an input or each other.
 * workspace_dev: at least qopt_layer_norm_backward_workspace(rows, dim) bytes, 16-byte aligned;
 * scratch whose contents need no preparation, for one call at a time; not used where dw_dev and
 * db_dev are both NULL.
 * rows 0: dw and db are all 0.
 * Errors as above, and QOPT_EINVAL for null statistics with rows or a workspace that is too small.
 */
int qopt_layer_norm_backward(const void* x_dev, int dtype, int64_t rows, int64_t dim, int64_t ldx,
                             const void* w_dev, int w_dtype, const float* mean_dev,
                             const float* rstd_dev, const void* dout_dev, int64_t lddo,
                             void* dx_dev, int64_t lddx, void* dw_dev, void* db_dev,
                             void* workspace_dev, size_t workspace_bytes, void* stream);
int qopt_layer_norm_backward_workspace(int64_t rows, int64_t dim, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* QOPT_NORM_H */
