// Declarations shared by the translation units of libtaco_rms: the row kernels
// (taco_rms_rows.hpp, compiled once per activation type) and the C ABI
// (taco_rms_abi.hip).
#pragma once

#include "taco_norm_internal.hpp"

namespace taco_norm {

// Arguments of the root-mean-square norm's kernels; rows >= 1.  codes != nullptr
// selects the 8-bit form (codes and scales instead of y and rstd).
struct RmsForward {
    const void *x, *residual;      // residual may be null
    const void *weight;            // may be null
    void *y, *total;               // total may be null
    float *rstd;                   // may be null
    uint8_t *codes, *scales;
    int64_t ldx, ldr, ldy, ldt, rows;
    int32_t hidden;
    int32_t params_f32;
    float eps;
};
struct RmsBackward {
    const void *dy, *x, *dtotal;   // dtotal may be null
    const float *rstd;
    const void *weight;            // may be null
    void *dx, *dweight;
    float *partial;                // workspace, unless dweight is null
    int64_t lddy, ldx, lddt, lddx, rows;
    int32_t hidden;
    int32_t params_f32;
    int32_t row_groups;            // work-groups that walk over rows
};
// Partial sums that the weight's gradient is made of, one per work-group: rows of the
// workspace, [hidden] float32.  As many as layer norm's, but 512 already from 2048 turns
// of rows on where rows are narrow, because there is one sum to write, not two: 256 and
// 512 parts take, with dtotal,
//     bf16     2048 / 4096 x 1536  12.9, 19.6 and 12.1, 16.3 us
//     bf16     2048 / 4096 x 2560  16.4, 25.6 and 15.9, 22.6 us
//     float32  2048 x 2560         22.9 and 23.1 us
//     bf16     2048 x 4096         19.7 and 21.4 us (the rule stays)
inline int64_t rms_parts(int64_t rows, int64_t hidden) {
    const int per = rows_per_group(hidden);
    if (hidden <= 2560 && (rows + per - 1) / per >= 2048) return 512;
    return backward_parts(rows, hidden);
}

// Whether the weight's gradient is made beside dx instead, from a second look at the
// rows: one launch, where the work-groups of 64 columns do not take longer than what
// they save.  Parts and this, with dtotal, in a graph:
//     bf16     1 / 64 / 256 x 2560     5.2, 6.4, 7.0 and 3.0, 3.3, 6.4 us
//     float32  1 / 64 / 256 x 2560     5.0, 6.3, 7.7 and 2.9, 3.2, 8.0 us
//     bf16     64 / 256 x 12288        9.1, 14.7 and 4.9, 19.6 us
//     bf16     512 x 2560              10.4 and 12.1 us
inline bool rms_apart(int64_t rows, int64_t hidden) { return rows <= 256 && rows * hidden <= 1 << 20; }

template <typename K>
struct Rms {
    static taco_status forward(const RmsForward &a, hipStream_t stream);
    static taco_status backward(const RmsBackward &a, hipStream_t stream);
};
extern template struct Rms<BF16>;
extern template struct Rms<F16>;
extern template struct Rms<F32>;

}  // namespace taco_norm
