/*
 * libtaco_rms -- root-mean-square norm on AMD Instinct MI355X (gfx950), with the
 * residual's addition, into rows of the same type or of 8-bit codes with block
 * scales, and its backward pass.
 *
 * Over [rows, hidden] tensors, row t and column k:
 *
 *     s = x + residual     q_t = (mean_k s_tk^2 + eps)^(-1/2)     y_tk = s_tk q_t w_k
 *
 *     g = dy w,   h_tk = s_tk q_t
 *     dx_tk = dtotal_tk + q_t (g_tk - h_tk mean_k(g_tk h_tk))     dw_k = sum_t dy_tk h_tk
 *
 * dx is the gradient of x and of residual alike; dtotal is the gradient that
 * arrives at s by its other ways.
 *
 * Conventions (those of taco_norm.h: pointers, types, row pitches, alignment,
 * float32 statistics and sums, the order of the checks), and
 *   - weight, residual and dtotal may be NULL (1, 0 and 0); the row pitches of what
 *     is NULL are not looked at.
 *   - total [rows, hidden] is s, for the next addition and the backward pass.  It
 *     may be NULL, and has to be without a residual (PARAM; s is x then).  y is
 *     formed from s before it is rounded.
 *   - y and total may each be x itself or residual itself (same pointer and
 *     pitch), dx may be dy or dtotal itself.  Otherwise an output may not overlap
 *     an input or another output.
 *   - A row's squares have to fit float32: a mean beyond 3e38 overflows.
 *   - rows == 0: forward calls are no-ops, dweight is zeros.
 */
#ifndef TACO_RMS_H
#define TACO_RMS_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "taco.h"
#include "taco_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Forward.  rstd: [rows] float32 output q, may be NULL. */
taco_status taco_rms_forward(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                             int64_t rows, int64_t hidden, taco_norm_dtype dtype,
                             const void *weight, taco_norm_dtype param_dtype, float eps,
                             void *y, int64_t ldy, void *total, int64_t ldt, float *rstd,
                             hipStream_t stream);

/* Forward into 8 bits: y as codes [rows, hidden] and scales [rows, hidden / 32], the
 * block-scaled form of taco_gated.h, which taco_gated_forward_mx reads; formed
 * from y in float32.  hidden is a multiple of 32 (SHAPE). */
taco_status taco_rms_mx(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                        int64_t rows, int64_t hidden, taco_norm_dtype dtype,
                        const void *weight, taco_norm_dtype param_dtype, float eps,
                        uint8_t *codes, uint8_t *scales, void *total, int64_t ldt,
                        hipStream_t stream);

/* Bytes of workspace that taco_rms_backward needs for dweight (0 with rows
 * == 0; -1 for a bad shape).  A call with dweight NULL needs none. */
int64_t taco_rms_backward_workspace(int64_t rows, int64_t hidden);

/* Backward from s (x: total as written by the forward pass, or x without a
 * residual) and rstd.  dweight: [hidden] of param_dtype, may be NULL. */
taco_status taco_rms_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                              const float *rstd, const void *dtotal, int64_t lddt,
                              const void *weight, int64_t rows, int64_t hidden,
                              taco_norm_dtype dtype, taco_norm_dtype param_dtype, void *dx,
                              int64_t lddx, void *dweight, void *workspace,
                              int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TACO_RMS_H */
