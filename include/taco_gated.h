/*
 * libtaco_gated -- the gated feed-forward block's first half on AMD Instinct
 * MI355X (gfx950): both projections, the activation and the product in one
 * kernel, its backward pass, and its forward pass on 8-bit codes with block
 * scales.
 *
 * Over X [rows, hidden] and weights Wg, Wu [features, hidden]:
 *
 *     G = X Wg^T     U = X Wu^T     A = act(G) U                (element-wise)
 *
 *     dG = dA U act'(G)             dU = dA act(G)
 *     dX = dG Wg + dU Wu            dWg = dG^T X        dWu = dU^T X
 *
 * act: silu  g / (1 + e^-g); gelu  g (1 + erf(g / sqrt 2)) / 2; and gelu_tanh
 * g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2.
 *
 * Codes with block scales (MX): of each 32 neighbours y of a row,
 *
 *     scale = 2^e, e the least integer >= -127 with max|y| <= 448 2^e
 *     code  = E4M3(y / scale), to nearest even
 *
 * kept as one byte a code (TACO_FORMAT_E4M3 of taco.h; zeros are code 0) and one
 * byte e + 127 a block; a block that holds an infinity or a NaN has scale byte
 * 255 and codes 127, NaN both.  taco_rms_mx of taco_rms.h writes rows in this
 * form.
 *
 * Conventions (those of taco_norm.h, except where stated)
 *   - Tensor pointers are DEVICE pointers owned by the caller.  The library
 *     allocates nothing and keeps no state.
 *   - dtype is TACO_NORM_BF16 or TACO_NORM_F16; all tensors of a call are of
 *     it.  A row is contiguous, consecutive rows are ld elements apart.  Rows of
 *     codes and scales, and weight gradients, are contiguous.
 *   - Any alignment of the elements' own size is accepted (codes: 16 bytes).
 *     Operands whose rows do not all start on 16-byte boundaries, or whose
 *     length is no multiple of 8 elements, are first copied to where they do,
 *     which takes their size of workspace and time (few rows excepted, forward: up
 *     to 16, and up to 64 where the library reads them as they are).
 *   - Sums are float32 (matrix instructions; for codes see below); the activation
 *     and its product are formed in float32 from the unrounded sums, and results are rounded once.
 *     dG and dU are rounded to dtype before their products: fp16 gradients need
 *     the usual loss scale.  Results do not depend on timing: no atomics.
 *   - Calls are asynchronous on `stream`.  Checks run in this order: types
 *     (FORMAT); sizes and row pitches (SHAPE); activation (PARAM); required
 *     pointers (NULL); alignment (ALIGN); overlaps (ALIAS); workspace size
 *     (PARAM); the launch (HIP).  On an error found by a check nothing is
 *     launched or written; after a launch that failed the outputs are
 *     unspecified.
 *   - rows == 0: forward calls are no-ops, weight gradients are zeros.
 *   - NaN and infinities propagate as the formulas say, to the rows and
 *     columns that they enter.
 *   - An output (the workspace among them) may not overlap an input or another
 *     output.
 *   - Thread-safe; calls on different streams may overlap if their buffers
 *     (workspaces included) do not.
 */
#ifndef TACO_GATED_H
#define TACO_GATED_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "taco.h"
#include "taco_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TACO_GATED_SILU = 0,
    TACO_GATED_GELU = 1,
    TACO_GATED_GELU_TANH = 2
} taco_gated_activation;

/* Largest hidden and features accepted.  A launch has to hold a call's tiles of 128 by
 * 64 elements, so those of [rows, the larger of hidden and features], and twice those
 * of [features, hidden], have to be fewer than 2^24, and rows fewer than 2^31 (SHAPE). */
#define TACO_GATED_MAX_WIDTH 1048576

/* Bytes of workspace of taco_gated_forward for these operands (-1 for a bad
 * shape).  The pointers are looked at for their alignment only. */
int64_t taco_gated_forward_workspace(const void *x, int64_t ldx, const void *gate_weight,
                                     int64_t ldg, const void *up_weight, int64_t ldu, int64_t rows,
                                     int64_t hidden, int64_t features);

/* Forward.  a [rows, features], lda apart.  gate, up: G and U, as the backward
 * pass takes them, both or neither (NULL); rows ldgu apart.
 * workspace: 16-byte aligned device memory, contents unspecified (NULL where
 * none is needed). */
taco_status taco_gated_forward(const void *x, int64_t ldx, const void *gate_weight, int64_t ldg,
                               const void *up_weight, int64_t ldu, int64_t rows, int64_t hidden,
                               int64_t features, taco_norm_dtype dtype,
                               taco_gated_activation activation, void *a, int64_t lda, void *gate,
                               void *up, int64_t ldgu, void *workspace, int64_t workspace_bytes,
                               hipStream_t stream);

/* Bytes of workspace of taco_gated_backward (-1 for a bad shape); want_dx and
 * want_dw: whether it is asked for dX, and for the weights' gradients. */
int64_t taco_gated_backward_workspace(const void *x, int64_t ldx, const void *gate_weight,
                                      int64_t ldg, const void *up_weight, int64_t ldu,
                                      int64_t rows, int64_t hidden, int64_t features,
                                      int32_t want_dx, int32_t want_dw);

/* Backward from da, x and the saved gate and up.  dx [rows, hidden], lddx
 * apart, may be NULL; dgate_weight, dup_weight [features, hidden], both or
 * neither NULL.  (What serves only an output that is not asked for may be NULL:
 * x without the weights' gradients, the weights without dx.) */
taco_status taco_gated_backward(const void *da, int64_t ldda, const void *x, int64_t ldx,
                                const void *gate, const void *up, int64_t ldgu,
                                const void *gate_weight, int64_t ldg, const void *up_weight,
                                int64_t ldu, int64_t rows, int64_t hidden, int64_t features,
                                taco_norm_dtype dtype, taco_gated_activation activation, void *dx,
                                int64_t lddx, void *dgate_weight, void *dup_weight,
                                void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace of taco_gated_forward_mx (-1 for a bad shape). */
int64_t taco_gated_forward_mx_workspace(int64_t rows, int64_t hidden, int64_t features);

/* Forward on codes [.., hidden] and scales [.., hidden / 32] of x and of both
 * weights; hidden is a multiple of 32.  a is of dtype.  The matrix instructions add
 * the products of codes in groups of eight neighbours, each to within 2^-12 of the
 * largest product of its group, and the groups in float32. */
taco_status taco_gated_forward_mx(const uint8_t *x_codes, const uint8_t *x_scales,
                                  const uint8_t *gate_codes, const uint8_t *gate_scales,
                                  const uint8_t *up_codes, const uint8_t *up_scales, int64_t rows,
                                  int64_t hidden, int64_t features, taco_norm_dtype dtype,
                                  taco_gated_activation activation, void *a, int64_t lda,
                                  void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* Codes and scales of x [rows, hidden] (weights, once; any of the three
 * types); hidden is a multiple of 32. */
taco_status taco_gated_mx_encode(const void *x, int64_t ldx, int64_t rows, int64_t hidden,
                                 taco_norm_dtype dtype, uint8_t *codes, uint8_t *scales,
                                 hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TACO_GATED_H */
