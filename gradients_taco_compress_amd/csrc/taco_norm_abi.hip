// libtaco_norm C ABI (declared in include/taco_norm.h): argument validation
// and dispatch.  Every check runs on the host before anything is launched.
#include <stdint.h>
#include <stddef.h>
#include <math.h>
#include <hip/hip_runtime.h>

#include "taco_norm.h"
#include "taco_norm_internal.hpp"

using namespace taco_norm;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool valid(taco_norm_dtype d) {
    return d == TACO_NORM_BF16 || d == TACO_NORM_F16 || d == TACO_NORM_F32;
}
int64_t size_of(taco_norm_dtype d) { return d == TACO_NORM_F32 ? 4 : 2; }

// Largest tensor extent accepted, in elements: byte sizes stay far inside 64 bits.
constexpr int64_t kMaxElements = INT64_C(1) << 48;

// [rows, width] with rows ld apart.
bool valid_rows(int64_t rows, int64_t width, int64_t ld) {
    if (rows < 0 || width <= 0 || ld < width) return false;
    return rows == 0 || ld <= kMaxElements / rows;
}

// A buffer that a call touches: rows of `width` bytes, `pitch` apart, over
// `bytes` in all (pitch 0: one row).
struct Span {
    const void *p;
    int64_t bytes;
    int64_t width, pitch;
};
Span rows_span(const void *p, int64_t rows, int64_t width, int64_t ld, int64_t size) {
    return {p, rows > 0 ? ((rows - 1) * ld + width) * size : 0, width * size, ld * size};
}
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    if (a0 >= b0 + (uintptr_t)b.bytes || b0 >= a0 + (uintptr_t)a.bytes) return false;
    // Columns of one wider tensor: with one pitch, the rows lie the same in
    // every stretch of that length.
    if (a.pitch == 0 || a.pitch != b.pitch) return true;
    const int64_t pitch = a.pitch, d = (int64_t)(b0 - a0) % pitch, from = d < 0 ? d + pitch : d;
    return from < a.width || from + b.width > pitch;
}
// Whether an output overlaps an input or another output.
template <int NO, int NI>
bool any_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlap(outs[o], ins[i])) return true;
        for (int i = 0; i < o; ++i)
            if (overlap(outs[o], outs[i])) return true;
    }
    return false;
}

taco_status check_types(taco_norm_dtype dtype, taco_norm_dtype param_dtype) {
    if (!valid(dtype) || !valid(param_dtype)) return TACO_ERR_FORMAT;
    if (param_dtype != dtype && param_dtype != TACO_NORM_F32) return TACO_ERR_FORMAT;
    return TACO_OK;
}

bool valid_hidden(int64_t hidden) { return hidden > 0 && hidden <= TACO_NORM_MAX_HIDDEN; }

float scale_of(int64_t hidden) {
    // hidden * 4^p <= 448^2 in whole numbers: hidden <= 2^20, so p is -2..8.
    for (int p = 8; p > -3; --p) {
        const int64_t left = p < 0 ? hidden : hidden << (2 * p);
        const int64_t right = p < 0 ? (INT64_C(448) * 448) << (-2 * p) : INT64_C(448) * 448;
        if (left <= right) return ldexpf(1.0f, p);
    }
    return 0.0f;
}

template <typename Fn>
taco_status with_type(taco_norm_dtype dtype, Fn &&fn) {
    switch (dtype) {
        case TACO_NORM_BF16: return fn(Rows<BF16>{});
        case TACO_NORM_F16: return fn(Rows<F16>{});
        default: return fn(Rows<F32>{});
    }
}

taco_status forward(const void *x, int64_t ldx, int64_t rows, int64_t hidden,
                    taco_norm_dtype dtype, const void *weight, const void *bias,
                    taco_norm_dtype param_dtype, float eps, void *y, int64_t ldy, bool checkpoint,
                    uint8_t *codes, float *mean, float *rstd, hipStream_t stream) {
    const taco_status st = check_types(dtype, param_dtype);
    if (st != TACO_OK) return st;
    if (!valid_hidden(hidden) || !valid_rows(rows, hidden, ldx) || !valid_rows(rows, hidden, ldy))
        return TACO_ERR_SHAPE;
    if (!(eps >= 0.0f) || isinf(eps)) return TACO_ERR_PARAM;
    if (rows == 0) return TACO_OK;
    if (!x || !y || (checkpoint && (!codes || !rstd))) return TACO_ERR_NULL;
    const int64_t e = size_of(dtype), p = size_of(param_dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(weight, p) || !aligned(bias, p) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return TACO_ERR_ALIGN;
    const Span outs[] = {rows_span(y, rows, hidden, ldy, e), {codes, rows * hidden},
                         {mean, rows * 4}, {rstd, rows * 4}};
    const Span ins[] = {rows_span(x, rows, hidden, ldx, e), {weight, hidden * p},
                        {bias, hidden * p}};
    if (any_overlap(outs, ins)) return TACO_ERR_ALIAS;
    Forward a = {};
    a.x = x; a.y = y; a.weight = weight; a.bias = bias;
    a.mean = mean; a.rstd = rstd; a.codes = codes;
    a.ldx = ldx; a.ldy = ldy; a.rows = rows; a.hidden = (int32_t)hidden;
    a.params_f32 = param_dtype == TACO_NORM_F32;
    a.eps = eps; a.scale = scale_of(hidden);
    return with_type(dtype, [&](auto k) { return decltype(k)::forward(a, stream); });
}

taco_status backward(const void *dy, int64_t lddy, bool checkpoint, const void *x, int64_t ldx,
                     const uint8_t *codes, const float *mean, const float *rstd,
                     const void *weight, int64_t rows, int64_t hidden, taco_norm_dtype dtype,
                     taco_norm_dtype param_dtype, void *dx, int64_t lddx, void *dweight,
                     void *dbias, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    taco_status st = check_types(dtype, param_dtype);
    if (st != TACO_OK) return st;
    if (!valid_hidden(hidden) || !valid_rows(rows, hidden, lddy) ||
        !valid_rows(rows, hidden, lddx) || (!checkpoint && !valid_rows(rows, hidden, ldx)))
        return TACO_ERR_SHAPE;
    const int64_t e = size_of(dtype), p = size_of(param_dtype);
    if (rows == 0) {
        if (!aligned(dweight, p) || !aligned(dbias, p)) return TACO_ERR_ALIGN;
        const Span sums[] = {{dweight, hidden * p}, {dbias, hidden * p}};
        const Span ins[] = {{weight, hidden * p}};
        if (any_overlap(sums, ins)) return TACO_ERR_ALIAS;
        st = dweight ? fill_zero(dweight, hidden, param_dtype, stream) : TACO_OK;
        return st != TACO_OK || !dbias ? st : fill_zero(dbias, hidden, param_dtype, stream);
    }
    const bool sums = dweight || dbias;
    if (!dy || !dx || !rstd || (checkpoint ? !codes : !x || !mean) || (sums && !workspace))
        return TACO_ERR_NULL;
    if (!aligned(dy, e) || !aligned(dx, e) || !aligned(x, e) || !aligned(weight, p) ||
        !aligned(dweight, p) || !aligned(dbias, p) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        (sums && !aligned(workspace, 16)))
        return TACO_ERR_ALIGN;
    const int64_t need = sums ? taco_norm_backward_workspace(rows, hidden) : 0;
    // dx may be dy itself: every row is read before it is written.
    const bool in_place = dx == dy && lddx == lddy;
    const Span outs[] = {rows_span(dx, rows, hidden, lddx, e), {dweight, hidden * p},
                         {dbias, hidden * p}, {sums ? workspace : nullptr, need}};
    const Span dy_span = rows_span(dy, rows, hidden, lddy, e);
    const Span ins[] = {in_place ? Span{} : dy_span,
                        rows_span(checkpoint ? nullptr : x, rows, hidden, ldx, e),
                        {checkpoint ? codes : nullptr, rows * hidden},
                        {checkpoint ? nullptr : mean, rows * 4},
                        {rstd, rows * 4}, {weight, hidden * p}};
    if (any_overlap(outs, ins)) return TACO_ERR_ALIAS;
    if (workspace_bytes < need) return TACO_ERR_PARAM;
    Backward a = {};
    a.dy = dy; a.x = x; a.codes = checkpoint ? codes : nullptr;
    a.mean = mean; a.rstd = rstd; a.weight = weight;
    a.dx = dx; a.dweight = dweight; a.dbias = dbias;
    a.partial = sums ? static_cast<float *>(workspace) : nullptr;
    a.lddy = lddy; a.ldx = ldx; a.lddx = lddx; a.rows = rows; a.hidden = (int32_t)hidden;
    a.params_f32 = param_dtype == TACO_NORM_F32;
    a.inv_scale = 1.0f / scale_of(hidden);
    return with_type(dtype, [&](auto k) { return decltype(k)::backward(a, stream); });
}

template <typename T>
__global__ __launch_bounds__(256) void zero_kernel(T *p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        p[i] = T(0);
}

}  // namespace

taco_status taco_norm::fill_zero(void *p, int64_t n, taco_norm_dtype dtype, hipStream_t stream) {
    const int64_t groups = (n + 255) / 256;
    const dim3 grid((unsigned)(groups < 4096 ? groups : 4096));
    if (dtype == TACO_NORM_F32)
        return launch(reinterpret_cast<const void *>(&zero_kernel<uint32_t>), grid, 256, stream,
                      static_cast<uint32_t *>(p), n);
    return launch(reinterpret_cast<const void *>(&zero_kernel<uint16_t>), grid, 256, stream,
                  static_cast<uint16_t *>(p), n);
}

extern "C" {

float taco_norm_checkpoint_scale(int64_t hidden) {
    return valid_hidden(hidden) ? scale_of(hidden) : 0.0f;
}

taco_status taco_norm_forward(const void *x, int64_t ldx, int64_t rows, int64_t hidden,
                              taco_norm_dtype dtype, const void *weight, const void *bias,
                              taco_norm_dtype param_dtype, float eps, void *y, int64_t ldy,
                              float *mean, float *rstd, hipStream_t stream) {
    return forward(x, ldx, rows, hidden, dtype, weight, bias, param_dtype, eps, y, ldy, false,
                   nullptr, mean, rstd, stream);
}

taco_status taco_norm_checkpoint(const void *x, int64_t ldx, int64_t rows, int64_t hidden,
                                 taco_norm_dtype dtype, const void *weight, const void *bias,
                                 taco_norm_dtype param_dtype, float eps, void *y, int64_t ldy,
                                 uint8_t *codes, float *rstd, hipStream_t stream) {
    return forward(x, ldx, rows, hidden, dtype, weight, bias, param_dtype, eps, y, ldy, true,
                   codes, nullptr, rstd, stream);
}

int64_t taco_norm_backward_workspace(int64_t rows, int64_t hidden) {
    if (!valid_hidden(hidden) || !valid_rows(rows, hidden, hidden)) return -1;
    return rows == 0 ? 0 : backward_parts(rows, hidden) * 2 * hidden * (int64_t)sizeof(float);
}

taco_status taco_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               const float *mean, const float *rstd, const void *weight,
                               int64_t rows, int64_t hidden, taco_norm_dtype dtype,
                               taco_norm_dtype param_dtype, void *dx, int64_t lddx,
                               void *dweight, void *dbias, void *workspace,
                               int64_t workspace_bytes, hipStream_t stream) {
    return backward(dy, lddy, false, x, ldx, nullptr, mean, rstd, weight, rows, hidden, dtype,
                    param_dtype, dx, lddx, dweight, dbias, workspace, workspace_bytes, stream);
}

taco_status taco_norm_checkpoint_backward(const void *dy, int64_t lddy, const uint8_t *codes,
                                          const float *rstd, const void *weight, int64_t rows,
                                          int64_t hidden, taco_norm_dtype dtype,
                                          taco_norm_dtype param_dtype, void *dx, int64_t lddx,
                                          void *dweight, void *dbias, void *workspace,
                                          int64_t workspace_bytes, hipStream_t stream) {
    return backward(dy, lddy, true, nullptr, hidden, codes, nullptr, rstd, weight, rows, hidden,
                    dtype, param_dtype, dx, lddx, dweight, dbias, workspace, workspace_bytes,
                    stream);
}

int64_t taco_norm_weight_grad_workspace(const void *dy, int64_t lddy, const uint8_t *codes,
                                        int64_t rows, int64_t out_features, int64_t hidden) {
    if (!valid_hidden(hidden) || !valid_hidden(out_features) ||
        !valid_rows(rows, out_features, lddy) || !valid_rows(rows, hidden, hidden))
        return -1;
    if (rows == 0) return 0;
    WeightGrad a = {};
    a.dy = dy; a.lddy = lddy; a.codes = codes; a.rows = rows;
    a.out_features = (int32_t)out_features; a.hidden = (int32_t)hidden;
    return weight_grad_workspace(a);
}

taco_status taco_norm_weight_grad(const void *dy, int64_t lddy, const uint8_t *codes,
                                  int64_t rows, int64_t out_features, int64_t hidden,
                                  taco_norm_dtype dtype, const void *weight, const void *bias,
                                  taco_norm_dtype param_dtype, void *dw,
                                  taco_norm_dtype dw_dtype, int32_t accumulate, float *dbias,
                                  void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    taco_status st = check_types(dtype, param_dtype);
    if (st != TACO_OK) return st;
    if (dtype == TACO_NORM_F32 || !valid(dw_dtype) ||
        (dw_dtype != dtype && dw_dtype != TACO_NORM_F32) ||
        (accumulate && dw_dtype != TACO_NORM_F32))
        return TACO_ERR_FORMAT;
    if (!valid_hidden(hidden) || !valid_hidden(out_features) ||
        !valid_rows(rows, out_features, lddy) || !valid_rows(rows, hidden, hidden))
        return TACO_ERR_SHAPE;
    if (!dw) return TACO_ERR_NULL;
    const int64_t p = size_of(param_dtype), d = size_of(dw_dtype);
    const Span dw_span = {dw, out_features * hidden * d}, db_span = {dbias, out_features * 4};
    const Span w_span = {weight, hidden * p}, b_span = {bias, hidden * p};
    if (rows == 0) {
        if (!aligned(dw, d) || !aligned(dbias, 4)) return TACO_ERR_ALIGN;
        const Span outs[] = {dw_span, db_span};
        const Span ins[] = {w_span, b_span};
        if (any_overlap(outs, ins)) return TACO_ERR_ALIAS;
        st = accumulate ? TACO_OK : fill_zero(dw, out_features * hidden, dw_dtype, stream);
        return st != TACO_OK || !dbias ? st : fill_zero(dbias, out_features, TACO_NORM_F32, stream);
    }
    const int64_t need =
        taco_norm_weight_grad_workspace(dy, lddy, codes, rows, out_features, hidden);
    if (!dy || !codes || (need && !workspace)) return TACO_ERR_NULL;
    if (!aligned(dy, 2) || !aligned(weight, p) || !aligned(bias, p) || !aligned(dw, d) ||
        !aligned(dbias, 4) || (need && !aligned(workspace, 16)))
        return TACO_ERR_ALIGN;
    const Span outs[] = {dw_span, db_span, {workspace, need}};
    const Span ins[] = {rows_span(dy, rows, out_features, lddy, 2), {codes, rows * hidden}, w_span,
                        b_span};
    if (any_overlap(outs, ins)) return TACO_ERR_ALIAS;
    if (workspace_bytes < need) return TACO_ERR_PARAM;
    WeightGrad a = {};
    a.dy = dy; a.codes = codes; a.weight = weight; a.bias = bias; a.dw = dw; a.dbias = dbias;
    a.workspace = static_cast<float *>(workspace);
    a.lddy = lddy; a.rows = rows;
    a.out_features = (int32_t)out_features; a.hidden = (int32_t)hidden;
    a.params_f32 = param_dtype == TACO_NORM_F32;
    a.dw_f32 = dw_dtype == TACO_NORM_F32; a.accumulate = accumulate != 0;
    a.inv_scale = 1.0f / scale_of(hidden);
    return weight_grad(a, dtype, stream);
}

}  // extern "C"
