// Declarations shared by the translation units of libtaco_norm: the row
// kernels (taco_norm_rows.hpp, compiled once per activation type), the
// weight gradient (taco_norm_weight_grad.hip) and the C ABI
// (taco_norm_abi.hip).
#pragma once

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "taco_norm.h"

namespace taco_norm {

// Arguments of the forward kernels, validated by the caller; rows >= 1.
// codes != nullptr selects the checkpointing forward.
struct Forward {
    const void *x;
    void *y;
    const void *weight, *bias;     // may be null
    float *mean, *rstd;            // may be null
    uint8_t *codes;
    int64_t ldx, ldy, rows;
    int32_t hidden;
    int32_t params_f32;            // weight and bias are float32, else of the activations' type
    float eps, scale;
};

// Arguments of the backward kernels; rows >= 1.  codes != nullptr: h comes
// from the checkpoint, else from x, mean and rstd.
struct Backward {
    const void *dy, *x;
    const uint8_t *codes;
    const float *mean, *rstd;
    const void *weight;
    void *dx;
    void *dweight, *dbias;         // may be null
    float *partial;                // workspace, unless both are null
    int64_t lddy, ldx, lddx, rows;
    int32_t hidden;
    int32_t params_f32;
    float inv_scale;
};

// Rows of this many columns at most are held in registers (some kernels hold
// fewer).
constexpr int kMaxHeld = 16384;

// Rows that share a work-group of the backward kernels.
inline int rows_per_group(int64_t hidden) { return hidden <= 128 ? 16 : hidden <= 1024 ? 4 : 1; }

// Partial sums the parameter gradients are made of, one per work-group: rows
// of the workspace, each [2][hidden] float32 (dweight, then dbias).  More
// work-groups finish their rows sooner but leave more to write and add up:
// half as many as turns of rows, at most one to a CU (777x2560: 256 parts
// 11.1 us, 512 14.5 us; 256x2560: 128 parts 7.7 us, 256 9.1 us), and two only
// for long sums over narrow rows.  256 and 512 parts, from x, in us:
//     bf16     2048 / 4096 / 8192 x 1536  11.7, 17.1, 27.5 and 12.6, 16.2, 23.2
//     bf16     2048 / 4096 / 8192 x 2560  15.3, 23.3, 36.7 and 16.8, 23.0, 32.2
//     bf16     2048 / 8192 / 16384 x 4096 18.5, 41.7, 74.3 and 22.6, 45.5, 78.4
//     float32  2048 / 8192 / 16384 x 2560 19.8, 57.3, 108.3 and 21.8, 57.2, 107.7
//     float32  2048 / 8192 / 16384 x 4096 27.2, 82.3, 160.4 and 31.5, 84.5, 158.2
// So the rule is not the best one everywhere: bf16 rows of up to 2560 columns
// would gain from 512 parts from about 4096 turns on (up to 15 % at 8191), and
// bf16 rows of 4096 columns lose 5 to 9 % by them.
inline int64_t backward_parts(int64_t rows, int64_t hidden) {
    if (hidden > kMaxHeld) return rows < 64 ? rows : 64;
    const int per = rows_per_group(hidden);
    const int64_t turns = (rows + per - 1) / per;
    if (turns <= 64) return turns;
    if (turns >= 8192 && hidden <= 4096) return 512;
    return turns / 2 < 256 ? turns / 2 : 256;
}

struct BF16 { typedef __bf16 type; };
struct F16 { typedef _Float16 type; };
struct F32 { typedef float type; };

template <typename K>
struct Rows {
    static taco_status forward(const Forward &a, hipStream_t stream);
    static taco_status backward(const Backward &a, hipStream_t stream);
};
extern template struct Rows<BF16>;
extern template struct Rows<F16>;
extern template struct Rows<F32>;

// Writes n zeros of the given type (a kernel, so that a graph can hold it).
taco_status fill_zero(void *p, int64_t n, taco_norm_dtype dtype, hipStream_t stream);

struct WeightGrad {
    const void *dy;
    const uint8_t *codes;
    const void *weight, *bias;     // may be null
    void *dw;
    float *dbias;                  // may be null
    float *workspace;
    int64_t lddy, rows;
    int64_t ldcodes;               // set by the launcher
    int32_t out_features, hidden;
    int32_t params_f32, dw_f32, accumulate;
    float inv_scale;
};
int64_t weight_grad_workspace(const WeightGrad &a);
taco_status weight_grad(const WeightGrad &a, taco_norm_dtype dtype, hipStream_t stream);

// The status is the launch's own (not an earlier error left in the runtime).
template <typename... Args>
taco_status launch(const void *fn, dim3 grid, int threads, hipStream_t stream, Args... args) {
    void *ptrs[] = {static_cast<void *>(&args)...};
    const hipError_t err = hipLaunchKernel(fn, grid, dim3((unsigned)threads), ptrs, 0, stream);
    return err == hipSuccess ? TACO_OK : TACO_ERR_HIP;
}

}  // namespace taco_norm
