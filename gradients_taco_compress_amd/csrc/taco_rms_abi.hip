// libtaco_rms C ABI (declared in include/taco_rms.h): argument validation and
// dispatch.  Every check runs on the host before anything is launched.
#include <stdint.h>
#include <stddef.h>
#include <math.h>
#include <hip/hip_runtime.h>

#include "taco_rms.h"
#include "taco_checks.hpp"
#include "taco_rms_internal.hpp"

using namespace taco_norm;

namespace {

taco_status check_types(taco_norm_dtype dtype, taco_norm_dtype param_dtype) {
    if (!valid(dtype) || !valid(param_dtype)) return TACO_ERR_FORMAT;
    if (param_dtype != dtype && param_dtype != TACO_NORM_F32) return TACO_ERR_FORMAT;
    return TACO_OK;
}

bool valid_hidden(int64_t hidden) { return hidden > 0 && hidden <= TACO_NORM_MAX_HIDDEN; }

template <typename Fn>
taco_status with_rms_type(taco_norm_dtype dtype, Fn &&fn) {
    switch (dtype) {
        case TACO_NORM_BF16: return fn(Rms<BF16>{});
        case TACO_NORM_F16: return fn(Rms<F16>{});
        default: return fn(Rms<F32>{});
    }
}

// An output may stand in the place of an input that has its rows (each element
// is read before it is written, by the thread that writes it).
bool same_place(const Span &a, const Span &b) { return a.p && a.p == b.p && a.pitch == b.pitch; }

taco_status rms_forward(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                        int64_t rows, int64_t hidden, taco_norm_dtype dtype, const void *weight,
                        taco_norm_dtype param_dtype, float eps, bool mx, void *y, int64_t ldy,
                        uint8_t *codes, uint8_t *scales, void *total, int64_t ldt, float *rstd,
                        hipStream_t stream) {
    const taco_status st = check_types(dtype, param_dtype);
    if (st != TACO_OK) return st;
    if (!valid_hidden(hidden) || !valid_rows(rows, hidden, ldx) ||
        (residual && !valid_rows(rows, hidden, ldr)) || (total && !valid_rows(rows, hidden, ldt)) ||
        (mx ? hidden % 32 != 0 : !valid_rows(rows, hidden, ldy)))
        return TACO_ERR_SHAPE;
    if (!(eps >= 0.0f) || isinf(eps) || (total && !residual)) return TACO_ERR_PARAM;
    if (rows == 0) return TACO_OK;
    if (!x || (mx ? !codes || !scales : !y)) return TACO_ERR_NULL;
    const int64_t e = size_of(dtype), p = size_of(param_dtype);
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(y, e) || !aligned(total, e) ||
        !aligned(weight, p) || !aligned(rstd, 4))
        return TACO_ERR_ALIGN;
    const Span outs[] = {rows_span(y, rows, hidden, ldy, e), rows_span(total, rows, hidden, ldt, e),
                         {codes, rows * hidden}, {scales, rows * (hidden / 32)}, {rstd, rows * 4}};
    const Span ins[] = {rows_span(x, rows, hidden, ldx, e),
                        rows_span(residual, rows, hidden, ldr, e), {weight, hidden * p}};
    for (const Span &o : outs) {
        const Span rest[] = {same_place(o, ins[0]) ? Span{} : ins[0],
                             same_place(o, ins[1]) ? Span{} : ins[1], ins[2]};
        const Span one[] = {o};
        if (any_overlap(one, rest)) return TACO_ERR_ALIAS;
    }
    const Span none[] = {Span{}};
    if (any_overlap(outs, none)) return TACO_ERR_ALIAS;
    RmsForward a = {};
    a.x = x; a.residual = residual; a.weight = weight;
    a.y = y; a.total = total; a.rstd = rstd; a.codes = codes; a.scales = scales;
    a.ldx = ldx; a.ldr = ldr; a.ldy = ldy; a.ldt = ldt; a.rows = rows;
    a.hidden = (int32_t)hidden; a.params_f32 = param_dtype == TACO_NORM_F32; a.eps = eps;
    return with_rms_type(dtype, [&](auto k) { return decltype(k)::forward(a, stream); });
}

// A row of n zeros (a kernel, so that a graph can hold it).
template <typename T>
__global__ __launch_bounds__(256) void zero_row_kernel(T *p, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = T(0);
}
taco_status zero_row(void *p, int64_t n, taco_norm_dtype dtype, hipStream_t stream) {
    const dim3 grid((unsigned)((n + 255) / 256));
    if (dtype == TACO_NORM_F32)
        return launch(reinterpret_cast<const void *>(&zero_row_kernel<uint32_t>), grid, 256, stream,
                      static_cast<uint32_t *>(p), (int)n);
    return launch(reinterpret_cast<const void *>(&zero_row_kernel<uint16_t>), grid, 256, stream,
                  static_cast<uint16_t *>(p), (int)n);
}

}  // namespace

extern "C" {

taco_status taco_rms_forward(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                             int64_t rows, int64_t hidden, taco_norm_dtype dtype,
                             const void *weight, taco_norm_dtype param_dtype, float eps,
                             void *y, int64_t ldy, void *total, int64_t ldt, float *rstd,
                             hipStream_t stream) {
    return rms_forward(x, ldx, residual, ldr, rows, hidden, dtype, weight, param_dtype, eps, false,
                       y, ldy, nullptr, nullptr, total, ldt, rstd, stream);
}

taco_status taco_rms_mx(const void *x, int64_t ldx, const void *residual, int64_t ldr,
                        int64_t rows, int64_t hidden, taco_norm_dtype dtype,
                        const void *weight, taco_norm_dtype param_dtype, float eps,
                        uint8_t *codes, uint8_t *scales, void *total, int64_t ldt,
                        hipStream_t stream) {
    return rms_forward(x, ldx, residual, ldr, rows, hidden, dtype, weight, param_dtype, eps, true,
                       nullptr, hidden, codes, scales, total, ldt, nullptr, stream);
}

int64_t taco_rms_backward_workspace(int64_t rows, int64_t hidden) {
    if (!valid_hidden(hidden) || !valid_rows(rows, hidden, hidden)) return -1;
    return rows == 0 ? 0 : rms_sums(rows, hidden) * hidden * (int64_t)sizeof(float);
}

taco_status taco_rms_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                              const float *rstd, const void *dtotal, int64_t lddt,
                              const void *weight, int64_t rows, int64_t hidden,
                              taco_norm_dtype dtype, taco_norm_dtype param_dtype, void *dx,
                              int64_t lddx, void *dweight, void *workspace,
                              int64_t workspace_bytes, hipStream_t stream) {
    const taco_status st = check_types(dtype, param_dtype);
    if (st != TACO_OK) return st;
    if (!valid_hidden(hidden) || !valid_rows(rows, hidden, lddy) ||
        !valid_rows(rows, hidden, ldx) || !valid_rows(rows, hidden, lddx) ||
        (dtotal && !valid_rows(rows, hidden, lddt)))
        return TACO_ERR_SHAPE;
    const int64_t e = size_of(dtype), p = size_of(param_dtype);
    const Span dw = {dweight, hidden * p}, w = {weight, hidden * p};
    if (rows == 0) {
        if (!aligned(dweight, p)) return TACO_ERR_ALIGN;
        if (overlap(dw, w)) return TACO_ERR_ALIAS;
        return dweight ? zero_row(dweight, hidden, param_dtype, stream) : TACO_OK;
    }
    if (!dy || !x || !rstd || !dx || (dweight && !workspace)) return TACO_ERR_NULL;
    if (!aligned(dy, e) || !aligned(x, e) || !aligned(dx, e) || !aligned(dtotal, e) ||
        !aligned(weight, p) || !aligned(dweight, p) || !aligned(rstd, 4) ||
        (dweight && !aligned(workspace, 16)))
        return TACO_ERR_ALIGN;
    const int64_t need = dweight ? taco_rms_backward_workspace(rows, hidden) : 0;
    const Span dx_span = rows_span(dx, rows, hidden, lddx, e);
    const Span dy_span = rows_span(dy, rows, hidden, lddy, e);
    const Span dt_span = rows_span(dtotal, rows, hidden, lddt, e);
    const Span outs[] = {dx_span, dw, {dweight ? workspace : nullptr, need}};
    const Span others[] = {rows_span(x, rows, hidden, ldx, e), {rstd, rows * 4}, w};
    // dx may be dy or dtotal itself: every element is read before it is written.
    const Span into_dx[] = {same_place(dx_span, dy_span) ? Span{} : dy_span,
                            same_place(dx_span, dt_span) ? Span{} : dt_span};
    const Span sums[] = {dw, outs[2]}, one[] = {dx_span}, grads[] = {dy_span, dt_span};
    if (any_overlap(outs, others) || any_overlap(one, into_dx) || any_overlap(sums, grads))
        return TACO_ERR_ALIAS;
    if (workspace_bytes < need) return TACO_ERR_PARAM;
    RmsBackward a = {};
    a.dy = dy; a.x = x; a.dtotal = dtotal; a.rstd = rstd; a.weight = weight;
    a.dx = dx; a.dweight = dweight;
    a.partial = dweight ? static_cast<float *>(workspace) : nullptr;
    a.lddy = lddy; a.ldx = ldx; a.lddt = lddt; a.lddx = lddx; a.rows = rows;
    a.hidden = (int32_t)hidden; a.params_f32 = param_dtype == TACO_NORM_F32;
    return with_rms_type(dtype, [&](auto k) { return decltype(k)::backward(a, stream); });
}

}  // extern "C"
