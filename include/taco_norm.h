/*
 * libtaco_norm -- layer norm for training on AMD Instinct MI355X (gfx950),
 * with an 8-bit checkpoint of the normalised activation that serves both the
 * norm's backward pass and the weight gradient of the linear layer behind it.
 *
 * Over a [rows, hidden] tensor, row t and column k:
 *
 *     m_t = mean_k x_tk              r_t = (mean_k (x_tk - m_t)^2 + eps)^(-1/2)
 *     h_tk = (x_tk - m_t) r_t        y_tk = h_tk w_k + b_k
 *
 *     g = dy w,   c1_t = mean_k g_tk,   c2_t = mean_k g_tk h_tk
 *     dx_tk = r_t (g_tk - c1_t - h_tk c2_t)
 *     dw_k  = sum_t dy_tk h_tk       db_k = sum_t dy_tk
 *
 * Checkpoint: a training step keeps a norm's input x for its backward pass
 * and its output y for the weight gradient of the linear layer it feeds.
 * Both follow from h, which is kept here as one E4M3 code per element (the
 * operator's format, TACO_FORMAT_E4M3 of taco.h):
 *
 *     codes_tk = E4M3(S h_tk),   S = taco_norm_checkpoint_scale(hidden) = 2^p,
 *     p the largest integer with hidden * 4^p <= 448^2.
 *
 * A row of h has sum_k h^2 <= hidden, hence |S h| <= 448: the codes never
 * overflow and need no scalars beside them -- the norm is itself the
 * adaptive scaling.  decode(code) / S is within 2^-4 of h relative (for
 * |S h| >= 2^-6, and within 2^-10 / S below).  taco_decode of taco.h decodes.
 *
 * Conventions (those of taco.h, except where stated)
 *   - Tensor pointers are DEVICE pointers owned by the caller.  The library
 *     allocates nothing and keeps no state.
 *   - Activations (x, y, dy, dx) are of one type, `dtype`; a row is
 *     contiguous, and consecutive rows are ld elements apart (ld >= row
 *     length; rows of a wider tensor are fine).  codes is contiguous.
 *     weight, bias, dweight and dbias are of `param_dtype`: dtype itself or
 *     float32.  weight and bias may be NULL (1 and 0).
 *   - Any alignment of the elements' own size is accepted; rows that start
 *     on 16-byte boundaries (8-byte for codes) are read and written faster.
 *   - Statistics and every sum are float32; results are rounded once, to
 *     nearest even.  Results do not depend on timing: no atomics.  A row's
 *     squared deviations have to fit float32: beyond 3e38 they overflow, and
 *     with eps = 0 those below 1e-38 are lost.
 *   - Calls are asynchronous on `stream`.  Checks run in this order: types
 *     (FORMAT); sizes and row pitches (SHAPE); eps (PARAM); required
 *     pointers (NULL); alignment (ALIGN); overlaps (ALIAS); workspace size
 *     (PARAM); the launch (HIP).  On an error found by a check nothing is
 *     launched or written; after a launch that failed (HIP) the outputs are
 *     unspecified, and a call must not be made again on one that it adds to.
 *   - rows == 0: forward calls are no-ops; gradients of parameters are sums
 *     over no rows, so the backward calls write zeros to them (and the
 *     weight gradient adds nothing when it accumulates).
 *   - NaN and infinities propagate as the formulas say, within their row
 *     (and, for parameter gradients, their column).
 *   - An output may not overlap an input or another output, except that dx
 *     may be dy itself (same pointer and pitch).  Rows of one pitch may lie
 *     side by side (column slices of one tensor); rows of different pitches
 *     count as overlapping where the memory from the first to the last does.
 *   - Thread-safe; calls on different streams may overlap if their buffers
 *     (workspaces included) do not.
 */
#ifndef TACO_NORM_H
#define TACO_NORM_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "taco.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TACO_NORM_BF16 = 0,
    TACO_NORM_F16 = 1,
    TACO_NORM_F32 = 2
} taco_norm_dtype;

/* Widest row accepted. */
#define TACO_NORM_MAX_HIDDEN 1048576

/* S of the checkpoint above for a row length (a power of two), or 0 for a
 * row length outside 1..TACO_NORM_MAX_HIDDEN. */
float taco_norm_checkpoint_scale(int64_t hidden);

/*
 * Forward.  mean, rstd: [rows] float32 outputs, each may be NULL.
 * eps: finite, >= 0 (with 0, a constant row divides by zero).
 */
taco_status taco_norm_forward(const void *x, int64_t ldx, int64_t rows, int64_t hidden,
                              taco_norm_dtype dtype, const void *weight, const void *bias,
                              taco_norm_dtype param_dtype, float eps, void *y, int64_t ldy,
                              float *mean, float *rstd, hipStream_t stream);

/* Forward that also writes the checkpoint: codes [rows, hidden] and rstd
 * [rows] (both required). */
taco_status taco_norm_checkpoint(const void *x, int64_t ldx, int64_t rows, int64_t hidden,
                                 taco_norm_dtype dtype, const void *weight, const void *bias,
                                 taco_norm_dtype param_dtype, float eps, void *y, int64_t ldy,
                                 uint8_t *codes, float *rstd, hipStream_t stream);

/* Bytes of workspace the two backward calls need for parameter gradients
 * (0 with rows == 0; -1 for a bad shape).  A call with dweight and dbias
 * both NULL needs none. */
int64_t taco_norm_backward_workspace(int64_t rows, int64_t hidden);

/*
 * Backward from the saved input: mean and rstd as written by
 * taco_norm_forward.  dweight, dbias: [hidden], each may be NULL.
 * workspace: 16-byte aligned device memory of at least
 * taco_norm_backward_workspace bytes, contents unspecified.
 */
taco_status taco_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               const float *mean, const float *rstd, const void *weight,
                               int64_t rows, int64_t hidden, taco_norm_dtype dtype,
                               taco_norm_dtype param_dtype, void *dx, int64_t lddx,
                               void *dweight, void *dbias, void *workspace,
                               int64_t workspace_bytes, hipStream_t stream);

/* Backward from the checkpoint: codes and rstd as written by
 * taco_norm_checkpoint; h = decode(codes) / S in the formulas above. */
taco_status taco_norm_checkpoint_backward(const void *dy, int64_t lddy, const uint8_t *codes,
                                          const float *rstd, const void *weight, int64_t rows,
                                          int64_t hidden, taco_norm_dtype dtype,
                                          taco_norm_dtype param_dtype, void *dx, int64_t lddx,
                                          void *dweight, void *dbias, void *workspace,
                                          int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace of taco_norm_weight_grad for these operands (0 where it
 * needs none, -1 for a bad shape).  The pointers are looked at for their
 * alignment only: an operand whose rows do not all start on 16-byte boundaries
 * (or, dy, that has a number of columns other than a multiple of 8) is
 * copied, which takes its size. */
int64_t taco_norm_weight_grad_workspace(const void *dy, int64_t lddy, const uint8_t *codes,
                                        int64_t rows, int64_t out_features, int64_t hidden);

/*
 * Weight gradient of z = y W^T (+ a bias) from the checkpoint of y's norm:
 *
 *     dW_nk = (w_k / S) sum_t dy_tn decode(codes_tk) + b_k db_n
 *     db_n  = sum_t dy_tn
 *
 *   dy        [rows, out_features] of dtype (TACO_NORM_BF16 or TACO_NORM_F16).
 *   weight, bias   the norm's, of param_dtype, each may be NULL.
 *   dw        [out_features, hidden], contiguous, of dw_dtype (dtype or
 *             float32); with accumulate != 0 (float32 only) the gradient is
 *             added to it.
 *   dbias     [out_features] float32 output db, may be NULL.
 *   workspace as above, taco_norm_weight_grad_workspace bytes (NULL where
 *             that is 0).
 * Both operands enter unrounded: a code times a bf16 or fp16 value is exact in
 * float32.  The sums over the rows, their joining, the scaling by w_k / S, the
 * bias term and the accumulation round in float32 (an element is off by less
 * than (rows + 24) 2^-24 of the sum of its terms' magnitudes), and the result
 * once to dw_dtype.  The sums are those of dy times S h, S up to 256: dy near
 * float32's largest values (bf16's beyond 10^35) may overflow them.
 */
taco_status taco_norm_weight_grad(const void *dy, int64_t lddy, const uint8_t *codes,
                                  int64_t rows, int64_t out_features, int64_t hidden,
                                  taco_norm_dtype dtype, const void *weight, const void *bias,
                                  taco_norm_dtype param_dtype, void *dw,
                                  taco_norm_dtype dw_dtype, int32_t accumulate, float *dbias,
                                  void *workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TACO_NORM_H */
