/*
 * qopt_muon.h -- C ABI of the orthogonalised optimizer steps in libqopt.so, for AMD Instinct
 * MI355X (gfx950): Newton-Schulz orthogonalisation of matrices, and the Muon step over many of
 * them with its momentum held as block-wise 8-bit codes or in binary32.
 *
 * It stands next to the AdamW steps of qopt.h: Muon for a model's matrices, AdamW for its
 * vectors and embeddings, and the 8-bit state of both is the one code of the 8-bit optimizers
 * summary page (signed codebook, blocks of 2048, each normalised by its own absmax).
 *
 * Newton-Schulz.  For U [rows, cols]: X = U / max(|U|, eps) with the Frobenius norm, then
 * `steps` times
 *     X = (a I + b A + c A^2) X,  A = X X^T,  a, b, c = 3.4445, -4.775, 2.0315
 * (of U's transpose where rows > cols), which moves every singular value s to
 * a s + b s^3 + c s^5 and so, after five, to between 0.68 and 1.14 where it was not tiny.
 *
 * Precision.  Every value between the products is held as the sum of two binary16 numbers (22
 * bits) under a fixed power of two, and a product of two such values is three matrix instructions
 * with binary32 sums; the result is rounded once, to the destination's type.  After five iterations
 * it is, before that, 0.5 to 2 times as far off as products of binary32 numbers leave it: 7e-7 to
 * 3e-5 of the result for 64 x 64 to 4096 x 4096, least where one entry holds nearly all of the norm, most
 * where the singular values spread (5e-7 to 4e-5 with those), and more where a few directions are
 * all that there is (2e-4 and 4e-4 for one of 2048; 9e-4 and 1e-4 where that one is rows of equal
 * values).  A bfloat16 result of the former is as far from the exact one as that one rounded,
 * 1.66e-3, to three digits.  The values' power of two is that of the largest possible one, so that
 * what lies 2^-15 under it or further down is held to 2^-37 of it instead: after 12 iterations rows whose
 * sizes spread by e^9 are 2e-4 off, 1e-5 with products of binary32 numbers.  What rounding adds in
 * directions that U does not have grows 3.4445 times per iteration, as in any such iteration, until
 * it counts, after some 12; no singular value leaves 1.21.
 * Matrices of up to 32 rows or columns are iterated in binary64.
 *
 * Conventions are those of qopt.h (status codes, dtypes, *_dev pointers in device memory
 * of the current HIP device, caller-owned buffers, host-side argument checks before
 * anything is enqueued, asynchronous work on `stream`).  Every entry point may be
 * captured into a graph.  Sums have a fixed order: equal calls give equal bits.
 */
#ifndef QOPT_MUON_H
#define QOPT_MUON_H

#include <stddef.h>
#include <stdint.h>

#include "qopt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of rows or columns of a matrix here. */
#define QOPT_MUON_MAX_DIM 131072
/* Largest number of iterations. */
#define QOPT_MUON_MAX_STEPS 32

/*
 * out_dev [batch, rows, cols] (out_dtype) = the orthogonalised matrices of x_dev [batch, rows,
 * cols] (dtype QOPT_F32 or QOPT_BF16), both contiguous.  A matrix of zeros stays one; a matrix
 * with an infinity or a NaN becomes all NaN, and leaves the others.  out must not overlap x.
 * workspace_dev: at least qopt_orthogonalize_workspace(batch, rows, cols, ...) bytes, 256-byte
 * aligned; scratch whose contents need no preparation, for one call at a time.
 * batch, rows or cols 0: nothing is written.
 * Errors: QOPT_EINVAL (null pointers with elements, sizes negative or too large, eps not finite,
 * negative or zero, steps outside 1 .. QOPT_MUON_MAX_STEPS, a workspace that is too small),
 * QOPT_EUNSUPPORTED (dtypes), QOPT_EALIGN, QOPT_ELAUNCH, QOPT_EINTERNAL (no host memory for the list of matrices).
 */
int qopt_orthogonalize(const void* x_dev, int dtype, int64_t batch, int64_t rows, int64_t cols,
                       int steps, float eps, void* out_dev, int out_dtype, void* workspace_dev,
                       size_t workspace_bytes, void* stream);
int qopt_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, size_t* bytes);

/* One matrix of a Muon step.  All pointers are device memory, the arrays contiguous. */
typedef struct qopt_muon_tensor {
  void* param;       /* [rows, cols] in the call's param dtype, updated */
  const void* grad;  /* [rows, cols] in the call's grad dtype */
  void* m;           /* [rows, cols] momentum, updated: uint8 codes, or binary32 */
  float* m_absmax;   /* [ceil(rows cols / 2048)] block maxima, updated; 32-bit: not used */
  int64_t rows;
  int64_t cols;
} qopt_muon_tensor;

/* How the rate of a matrix follows from its shape. */
typedef enum {
  QOPT_MUON_ORIGINAL = 0,        /* lr sqrt(max(1, rows / cols)) */
  QOPT_MUON_MATCH_RMS_ADAMW = 1  /* lr 0.2 sqrt(max(rows, cols)): the size of an AdamW update */
} qopt_muon_adjust;

typedef struct qopt_muon_hparams {
  float lr;
  float momentum;
  float weight_decay;
  float eps;
  int32_t nesterov; /* 0 or 1 */
  int32_t adjust;   /* a qopt_muon_adjust */
  int32_t steps;    /* Newton-Schulz iterations */
} qopt_muon_hparams;

/*
 * One Muon step over ntensors matrices of any shapes.  Per element, binary32, one rounding per
 * operation:
 *   g = grad * s                           m = mu * m + (1 - mu) * g
 *   u = nesterov ? mu * m + (1 - mu) * g : m
 *   p = param * decay - O(u) * rate
 * with O(u) the orthogonalised u (precision by the param dtype, as above), decay = fl32(1 - lr *
 * weight_decay) and rate as qopt_muon_adjust says, both evaluated in binary64 from the binary32
 * hyper-parameters, and s the fp32 value at grad_scale_dev (read when the work runs; NULL for
 * 1).  u comes from m before it is requantized; a bf16 parameter is rounded once.
 *   qopt_muon8bit_step   m is kept as signed block-wise codes (cb_m_dev, 16-byte aligned: a
 *                        QOPT_CB_SIGNED codebook), requantized as qopt_adam8bit_step does
 *   qopt_muon32bit_step  m is kept in binary32
 * A matrix whose u has an infinity or a NaN gets NaN parameters; the others are as without it.
 * No tensor may overlap another.  Matrices without elements are left out.
 * workspace_dev: at least qopt_muon_workspace(tensors, ...) bytes, 256-byte aligned; scratch
 * whose contents need no preparation, for one call at a time.  It holds what the matrices that
 * share their launches need, not all of them: 12 bytes per element and 20 per value of their m x m
 * (m the shorter side), and partial sums (1.0 GB for 4096 x 11008).
 * Errors: QOPT_EINVAL (null pointers with elements, sizes, hyper-parameters: lr, weight_decay and
 * eps finite, lr and weight_decay >= 0, eps > 0, momentum in [0, 1), steps in 1 ..
 * QOPT_MUON_MAX_STEPS, nesterov 0 or 1; a workspace that is too small), QOPT_EUNSUPPORTED
 * (dtypes, adjust), QOPT_EALIGN, QOPT_ELAUNCH, QOPT_EINTERNAL.  The hyper-parameters are checked also for a step of no tensors.
 */
int qopt_muon8bit_step(const qopt_muon_tensor* tensors, int32_t ntensors, int param_dtype,
                       int grad_dtype, const qopt_codebook* cb_m_dev, const qopt_muon_hparams* hp,
                       const float* grad_scale_dev, void* workspace_dev, size_t workspace_bytes,
                       void* stream);
int qopt_muon32bit_step(const qopt_muon_tensor* tensors, int32_t ntensors, int param_dtype,
                        int grad_dtype, const qopt_muon_hparams* hp, const float* grad_scale_dev,
                        void* workspace_dev, size_t workspace_bytes, void* stream);
/* Only the sizes of the tensors are read. */
int qopt_muon_workspace(const qopt_muon_tensor* tensors, int32_t ntensors, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* QOPT_MUON_H */
