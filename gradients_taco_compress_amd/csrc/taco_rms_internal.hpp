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
    int32_t segments;              // of the rows, for the weight's gradient apart (0: not apart)
};
// Partial sums that the weight's gradient is made of, one per work-group: rows of the
// workspace, [hidden] float32.  As many as layer norm's, but 512 already from 2048 turns
// of rows on where rows are narrow, because there is one sum to write, not two: 256 and
// 512 parts take, with dtotal,
//     bf16     2048 / 4096 x 1536  12.9, 19.6 and 12.1, 16.3 us
//     bf16     2048 / 4096 x 2560  16.4, 25.6 and 15.9, 22.6 us
//     float32  2048 x 2560         22.9 and 23.1 us
//     bf16     2048 x 4096         19.7 and 21.4 us (the rule stays)
// (float32 gains nothing and loses 1 %; the workspace's size, which follows from this, is
// asked for by rows and columns alone.)
inline int64_t rms_parts(int64_t rows, int64_t hidden) {
    const int per = rows_per_group(hidden);
    if (hidden <= 2560 && (rows + per - 1) / per >= 2048) return 512;
    return backward_parts(rows, hidden);
}

// Segments of the rows whose weight gradients are made beside dx, from a second look at
// the rows (0: not so, but as parts).  One segment leaves nothing to join: one launch
// instead of two, up to 128 rows; several are a second launch too, but narrow rows finish
// sooner.  With dtotal, in a graph, in us, parts and this:
//     bf16     64 / 128 x 2567      7.5, 9.3 and 4.4, 6.1
//     bf16     64 / 128 x 12288     10.3, 13.1 and 5.9, 8.2
//     float32  64 / 128 x 2567      7.6, 10.1 and 4.8, 8.0
//     float32  256 x 2567           10.5 and 15.9 in one segment, 11.3 in four (as parts)
//     bf16     256 / 512 x 1024     7.2, 8.6 and 5.0, 5.7; 777 x 1024 9.8 and 10.5 (as parts)
//     float32  256 / 512 x 1024     7.8, 10.0 and 5.6, 6.5
//     bf16     512 / 2048 x 128     6.2, 8.0 and 4.8, 5.9
inline int32_t rms_segments(int64_t rows, int64_t hidden) {
    if (rows <= 128) return 1;
    if (hidden <= 128 && rows <= 2048) return 16;
    return hidden <= 1024 && rows <= 512 ? 8 : 0;
}
// Rows of the workspace.
inline int64_t rms_sums(int64_t rows, int64_t hidden) {
    const int64_t parts = rms_parts(rows, hidden), segments = rms_segments(rows, hidden);
    return parts > segments ? parts : segments;
}

template <typename K>
struct Rms {
    static taco_status forward(const RmsForward &a, hipStream_t stream);
    static taco_status backward(const RmsBackward &a, hipStream_t stream);
};
extern template struct Rms<BF16>;
extern template struct Rms<F16>;
extern template struct Rms<F32>;

}  // namespace taco_norm
