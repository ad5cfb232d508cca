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
};
template <typename K>
struct Rms {
    static taco_status forward(const RmsForward &a, hipStream_t stream);
    static taco_status backward(const RmsBackward &a, hipStream_t stream);
};
extern template struct Rms<BF16>;
extern template struct Rms<F16>;
extern template struct Rms<F32>;

}  // namespace taco_norm
