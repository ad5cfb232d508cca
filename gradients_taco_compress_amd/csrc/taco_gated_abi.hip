// libtaco_gated C ABI (declared in include/taco_gated.h): argument validation
// and dispatch.  Every check runs on the host before anything is launched.
#include <stdint.h>
#include <stddef.h>
#include <hip/hip_runtime.h>

#include "taco_gated.h"
#include "taco_checks.hpp"
#include "taco_gated_internal.hpp"

using namespace taco_gated;

namespace {

constexpr int64_t kSize = 2;           // bytes of an element

int64_t round_up(int64_t n, int64_t d) { return (n + d - 1) / d * d; }

// Sizes accepted: the products' smallest tiles (256 threads to 128x64 outputs at
// the least) stay inside a grid's 2^32 threads.
constexpr int64_t kMaxTiles = INT64_C(1) << 24;

int64_t tiles(int64_t m, int64_t n) { return (m + 127) / 128 * ((n + 63) / 64); }

bool valid_width(int64_t n) { return n > 0 && n <= TACO_GATED_MAX_WIDTH; }
bool valid_sizes(int64_t rows, int64_t hidden, int64_t features) {
    if (rows < 0 || rows > kMaxElements || !valid_width(hidden) || !valid_width(features)) return false;
    const int64_t wide = hidden > features ? hidden : features;
    return rows / 128 < kMaxTiles && tiles(rows, wide) < kMaxTiles &&
           2 * tiles(features, hidden) < kMaxTiles;
}
bool valid(taco_gated_activation a) {
    return a == TACO_GATED_SILU || a == TACO_GATED_GELU || a == TACO_GATED_GELU_TANH;
}
bool valid_type(taco_norm_dtype d) { return d == TACO_NORM_BF16 || d == TACO_NORM_F16; }

Span rows16(const void *p, int64_t rows, int64_t width, int64_t ld) {
    return rows_span(p, rows, width, ld, kSize);
}

// An operand [rows, width]: as it is, or as a copy in the workspace whose rows
// start on 16-byte boundaries.
struct Operand {
    const void *p;
    int64_t ld, rows, width;
    bool copied;
    int64_t copy_pitch() const { return round_up(width * kSize, 16); }
    int64_t copy_bytes() const { return copied ? rows * copy_pitch() : 0; }
    int64_t pitch() const { return copied ? copy_pitch() : ld * kSize; }
};
Operand operand(const void *p, int64_t ld, int64_t rows, int64_t width) {
    const bool direct = aligned(p, 16) && (ld * kSize) % 16 == 0 && width % 8 == 0 &&
                        ld * kSize <= kMaxPitch;
    return {p, ld, rows, width, !direct};
}
// Two weights that one kernel reads with one pitch.
void alike(Operand *a, Operand *b) {
    if (a->pitch() != b->pitch() || a->copied != b->copied) a->copied = b->copied = true;
}

// Takes pieces of the workspace, in order, and queues the copies.
struct Arena {
    char *at;
    Repack copies[3];
    int count;
    void *take(int64_t bytes) {
        void *const p = at;
        at += round_up(bytes, 16);
        return p;
    }
    Matrix place(const Operand &o) {
        if (!o.copied) return {o.p, o.pitch()};
        void *const to = take(o.copy_bytes());
        copies[count++] = {o.p, to, o.ld * kSize, o.copy_pitch(), o.rows, o.width * kSize};
        return {to, o.copy_pitch()};
    }
    taco_status copy(hipStream_t stream) const {
        return count ? repack(copies, count, stream) : TACO_OK;
    }
};

template <typename F>
taco_status with_type(taco_norm_dtype dtype, F &&f) {
    return dtype == TACO_NORM_BF16 ? f(Products<BF16>{}) : f(Products<F16>{});
}

// (A plan depends on the sizes only, not on which 16-bit type it is.)
Product sizes(int64_t m, int64_t n, int64_t k) {
    Product p = {};
    p.m = m; p.n = n; p.k = k;
    return p;
}

struct ForwardOperands {
    Operand x, gate, up;
    int64_t slab_bytes, bytes;
    bool few;
};
ForwardOperands forward_operands(const void *x, int64_t ldx, const void *gate, int64_t ldg,
                                 const void *up, int64_t ldu, int64_t rows, int64_t hidden,
                                 int64_t features) {
    ForwardOperands o = {operand(x, ldx, rows, hidden), operand(gate, ldg, features, hidden),
                         operand(up, ldu, features, hidden), 0, 0, false};
    alike(&o.gate, &o.up);
    const int64_t copies = o.x.copy_bytes() + o.gate.copy_bytes() + o.up.copy_bytes();
    const Product p = sizes(rows, features, hidden);
    o.few = Products<BF16>::few_takes(p, copies);
    if (o.few) return o;
    o.slab_bytes = Products<BF16>::workspace(Kind::kForward, p);
    o.bytes = o.slab_bytes + copies;
    return o;
}

struct BackwardOperands {
    Operand x, gate, up;
    int64_t slab_bytes, d_pitch, bytes;       // d_pitch: of dG and dU, in elements
};
BackwardOperands backward_operands(const void *x, int64_t ldx, const void *gate, int64_t ldg,
                                   const void *up, int64_t ldu, int64_t rows, int64_t hidden,
                                   int64_t features, bool want_dx, bool want_dw) {
    BackwardOperands o = {operand(x, ldx, rows, hidden), operand(gate, ldg, features, hidden),
                          operand(up, ldu, features, hidden), 0, 0, 0};
    alike(&o.gate, &o.up);
    o.d_pitch = round_up(features, 8);
    const Product input = sizes(rows, hidden, features), weight = sizes(features, hidden, rows);
    if (want_dx) o.bytes += o.gate.copy_bytes() + o.up.copy_bytes();
    if (want_dw) o.bytes += o.x.copy_bytes();
    o.slab_bytes = want_dx && want_dw ? Products<BF16>::pair_workspace(input, weight)
                   : want_dx          ? Products<BF16>::workspace(Kind::kInput, input)
                                      : Products<BF16>::workspace(Kind::kWeight, weight);
    o.bytes += o.slab_bytes + 2 * rows * o.d_pitch * kSize;
    return o;
}

bool valid_mx(int64_t rows, int64_t hidden, int64_t features) {
    return valid_sizes(rows, hidden, features) && hidden % 32 == 0;
}

}  // namespace

extern "C" {

int64_t taco_gated_forward_workspace(const void *x, int64_t ldx, const void *gate_weight,
                                     int64_t ldg, const void *up_weight, int64_t ldu, int64_t rows,
                                     int64_t hidden, int64_t features) {
    if (!valid_sizes(rows, hidden, features) || !valid_rows(rows, hidden, ldx) ||
        !valid_rows(features, hidden, ldg) || !valid_rows(features, hidden, ldu))
        return -1;
    if (rows == 0) return 0;
    return forward_operands(x, ldx, gate_weight, ldg, up_weight, ldu, rows, hidden, features).bytes;
}

taco_status taco_gated_forward(const void *x, int64_t ldx, const void *gate_weight, int64_t ldg,
                               const void *up_weight, int64_t ldu, int64_t rows, int64_t hidden,
                               int64_t features, taco_norm_dtype dtype,
                               taco_gated_activation activation, void *a, int64_t lda, void *gate,
                               void *up, int64_t ldgu, void *workspace, int64_t workspace_bytes,
                               hipStream_t stream) {
    if (!valid_type(dtype)) return TACO_ERR_FORMAT;
    const bool save = gate || up;
    if (!valid_sizes(rows, hidden, features) || !valid_rows(rows, hidden, ldx) ||
        !valid_rows(features, hidden, ldg) || !valid_rows(features, hidden, ldu) ||
        !valid_rows(rows, features, lda) || (save && !valid_rows(rows, features, ldgu)))
        return TACO_ERR_SHAPE;
    if (!valid(activation)) return TACO_ERR_PARAM;
    if (rows == 0) return TACO_OK;
    const ForwardOperands o =
        forward_operands(x, ldx, gate_weight, ldg, up_weight, ldu, rows, hidden, features);
    if (!x || !gate_weight || !up_weight || !a || (save && (!gate || !up)) ||
        (o.bytes && !workspace))
        return TACO_ERR_NULL;
    if (!aligned(x, 2) || !aligned(gate_weight, 2) || !aligned(up_weight, 2) || !aligned(a, 2) ||
        !aligned(gate, 2) || !aligned(up, 2) || (o.bytes && !aligned(workspace, 16)))
        return TACO_ERR_ALIGN;
    const Span outs[] = {rows16(a, rows, features, lda), rows16(gate, rows, features, ldgu),
                         rows16(up, rows, features, ldgu), {workspace, o.bytes}};
    const Span ins[] = {rows16(x, rows, hidden, ldx), rows16(gate_weight, features, hidden, ldg),
                        rows16(up_weight, features, hidden, ldu)};
    if (any_overlap(outs, ins)) return TACO_ERR_ALIAS;
    if (workspace_bytes < o.bytes) return TACO_ERR_PARAM;
    Product p = sizes(rows, features, hidden);
    p.activation = activation;
    p.out[0] = a; p.out[1] = gate; p.out[2] = up;
    p.out_pitch[0] = lda; p.out_pitch[1] = p.out_pitch[2] = ldgu;
    if (o.few) {
        p.a[0] = {x, ldx * kSize};
        p.b[0] = {gate_weight, ldg * kSize};
        p.b[1] = {up_weight, ldu * kSize};
        return with_type(dtype, [&](auto k) { return decltype(k)::few(p, stream); });
    }
    Arena arena = {static_cast<char *>(workspace), {}, 0};
    p.slabs = static_cast<float *>(arena.take(o.slab_bytes));
    p.a[0] = p.a[1] = arena.place(o.x);
    p.b[0] = arena.place(o.gate);
    p.b[1] = arena.place(o.up);
    const taco_status st = arena.copy(stream);
    if (st != TACO_OK) return st;
    return with_type(dtype, [&](auto k) { return decltype(k)::run(Kind::kForward, p, stream); });
}

int64_t taco_gated_backward_workspace(const void *x, int64_t ldx, const void *gate_weight,
                                      int64_t ldg, const void *up_weight, int64_t ldu,
                                      int64_t rows, int64_t hidden, int64_t features,
                                      int32_t want_dx, int32_t want_dw) {
    if (!valid_sizes(rows, hidden, features) || (want_dw && !valid_rows(rows, hidden, ldx)) ||
        (want_dx && (!valid_rows(features, hidden, ldg) || !valid_rows(features, hidden, ldu))))
        return -1;
    if (rows == 0 || (!want_dx && !want_dw)) return 0;
    return backward_operands(x, ldx, gate_weight, ldg, up_weight, ldu, rows, hidden, features,
                             want_dx, want_dw).bytes;
}

taco_status taco_gated_backward(const void *da, int64_t ldda, const void *x, int64_t ldx,
                                const void *gate, const void *up, int64_t ldgu,
                                const void *gate_weight, int64_t ldg, const void *up_weight,
                                int64_t ldu, int64_t rows, int64_t hidden, int64_t features,
                                taco_norm_dtype dtype, taco_gated_activation activation, void *dx,
                                int64_t lddx, void *dgate_weight, void *dup_weight,
                                void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!valid_type(dtype)) return TACO_ERR_FORMAT;
    const bool want_dx = dx, want_dw = dgate_weight || dup_weight;
    if (!valid_sizes(rows, hidden, features) || !valid_rows(rows, features, ldda) ||
        !valid_rows(rows, features, ldgu) || (want_dw && !valid_rows(rows, hidden, ldx)) ||
        (want_dx && (!valid_rows(rows, hidden, lddx) || !valid_rows(features, hidden, ldg) ||
                     !valid_rows(features, hidden, ldu))))
        return TACO_ERR_SHAPE;
    if (!valid(activation)) return TACO_ERR_PARAM;
    if (want_dw && (!dgate_weight || !dup_weight)) return TACO_ERR_NULL;
    if (!want_dx && !want_dw) return TACO_OK;
    const Span dg_span = {dgate_weight, features * hidden * kSize};
    const Span du_span = {dup_weight, features * hidden * kSize};
    if (rows == 0) {
        if (!want_dw) return TACO_OK;
        if (!aligned(dgate_weight, 2) || !aligned(dup_weight, 2)) return TACO_ERR_ALIGN;
        if (overlap(dg_span, du_span)) return TACO_ERR_ALIAS;
        const taco_status st = fill_zero(dgate_weight, features * hidden, stream);
        return st != TACO_OK ? st : fill_zero(dup_weight, features * hidden, stream);
    }
    const BackwardOperands o = backward_operands(x, ldx, gate_weight, ldg, up_weight, ldu, rows,
                                                 hidden, features, want_dx, want_dw);
    if (!da || !gate || !up || (want_dw && !x) || (want_dx && (!gate_weight || !up_weight)) ||
        !workspace)
        return TACO_ERR_NULL;
    if (!aligned(da, 2) || !aligned(gate, 2) || !aligned(up, 2) || (want_dw && !aligned(x, 2)) ||
        (want_dx && (!aligned(gate_weight, 2) || !aligned(up_weight, 2))) || !aligned(dx, 2) ||
        !aligned(dgate_weight, 2) || !aligned(dup_weight, 2) || !aligned(workspace, 16))
        return TACO_ERR_ALIGN;
    const Span outs[] = {rows16(dx, rows, hidden, lddx), dg_span, du_span, {workspace, o.bytes}};
    const Span ins[] = {rows16(da, rows, features, ldda), rows16(gate, rows, features, ldgu),
                        rows16(up, rows, features, ldgu),
                        rows16(want_dw ? x : nullptr, rows, hidden, ldx),
                        rows16(want_dx ? gate_weight : nullptr, features, hidden, ldg),
                        rows16(want_dx ? up_weight : nullptr, features, hidden, ldu)};
    if (any_overlap(outs, ins)) return TACO_ERR_ALIAS;
    if (workspace_bytes < o.bytes) return TACO_ERR_PARAM;
    Arena arena = {static_cast<char *>(workspace), {}, 0};
    float *const slab = static_cast<float *>(arena.take(o.slab_bytes));
    void *const dgate = arena.take(rows * o.d_pitch * kSize);
    void *const dup = arena.take(rows * o.d_pitch * kSize);
    const Matrix mx = want_dw ? arena.place(o.x) : Matrix{};
    const Matrix mg = want_dx ? arena.place(o.gate) : Matrix{};
    const Matrix mu = want_dx ? arena.place(o.up) : Matrix{};
    ActivationGrad act = {};
    act.da = da; act.gate = gate; act.up = up; act.dgate = dgate; act.dup = dup;
    act.ldda = ldda; act.ldgu = ldgu; act.to_pitch = o.d_pitch; act.rows = rows;
    act.features = (int32_t)features; act.activation = activation;
    const taco_status st =
        activation_grad(act, dtype == TACO_NORM_F16, arena.copies, arena.count, stream);
    if (st != TACO_OK) return st;
    Product input = sizes(rows, hidden, features), weight = sizes(features, hidden, rows);
    input.a[0] = weight.a[0] = {dgate, o.d_pitch * kSize};
    input.a[1] = weight.a[1] = {dup, o.d_pitch * kSize};
    input.slabs = weight.slabs = slab;
    input.b[0] = mg; input.b[1] = mu;
    input.out[0] = dx; input.out_pitch[0] = lddx;
    weight.b[0] = weight.b[1] = mx;
    weight.out[0] = dgate_weight; weight.out[1] = dup_weight;
    weight.out_pitch[0] = weight.out_pitch[1] = hidden;
    return with_type(dtype, [&](auto k) {
        using P = decltype(k);
        if (want_dx && want_dw) return P::run_pair(input, weight, stream);
        return want_dx ? P::run(Kind::kInput, input, stream) : P::run(Kind::kWeight, weight, stream);
    });
}

int64_t taco_gated_forward_mx_workspace(int64_t rows, int64_t hidden, int64_t features) {
    if (!valid_mx(rows, hidden, features)) return -1;
    const Product p = sizes(rows, features, hidden);
    if (Products<Codes>::few_takes(p, 0)) return 0;
    return Products<Codes>::workspace(Kind::kForward, p) + scale_tile_bytes(rows, hidden / 32) +
           2 * scale_tile_bytes(features, hidden / 32);
}

taco_status taco_gated_forward_mx(const uint8_t *x_codes, const uint8_t *x_scales,
                                  const uint8_t *gate_codes, const uint8_t *gate_scales,
                                  const uint8_t *up_codes, const uint8_t *up_scales, int64_t rows,
                                  int64_t hidden, int64_t features, taco_norm_dtype dtype,
                                  taco_gated_activation activation, void *a, int64_t lda,
                                  void *workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!valid_type(dtype)) return TACO_ERR_FORMAT;
    if (!valid_mx(rows, hidden, features) || !valid_rows(rows, features, lda)) return TACO_ERR_SHAPE;
    if (!valid(activation)) return TACO_ERR_PARAM;
    if (rows == 0) return TACO_OK;
    const int64_t need = taco_gated_forward_mx_workspace(rows, hidden, features);
    if (!x_codes || !x_scales || !gate_codes || !gate_scales || !up_codes || !up_scales || !a ||
        (need && !workspace))
        return TACO_ERR_NULL;
    if (!aligned(x_codes, 16) || !aligned(gate_codes, 16) || !aligned(up_codes, 16) ||
        !aligned(a, 2) || (need && !aligned(workspace, 16)))
        return TACO_ERR_ALIGN;
    const int64_t blocks = hidden / 32;
    const Span outs[] = {rows16(a, rows, features, lda), {workspace, need}};
    const Span ins[] = {{x_codes, rows * hidden}, {x_scales, rows * blocks},
                        {gate_codes, features * hidden}, {gate_scales, features * blocks},
                        {up_codes, features * hidden}, {up_scales, features * blocks}};
    if (any_overlap(outs, ins)) return TACO_ERR_ALIAS;
    if (workspace_bytes < need) return TACO_ERR_PARAM;
    Product p = sizes(rows, features, hidden);
    p.activation = activation;
    p.out_f16 = dtype == TACO_NORM_F16;
    p.out[0] = a; p.out_pitch[0] = lda;
    p.a[0] = {x_codes, hidden};
    p.b[0] = {gate_codes, hidden};
    p.b[1] = {up_codes, hidden};
    p.a_scale = {x_scales, blocks};
    p.b_scale[0] = {gate_scales, blocks};
    p.b_scale[1] = {up_scales, blocks};
    if (Products<Codes>::few_takes(p, 0)) return Products<Codes>::few(p, stream);
    Arena arena = {static_cast<char *>(workspace), {}, 0};
    p.slabs = static_cast<float *>(arena.take(Products<Codes>::workspace(Kind::kForward, p)));
    Matrix *const to[] = {&p.a_scale, &p.b_scale[0], &p.b_scale[1]};
    ScaleTiles tiles[3];
    for (int i = 0; i < 3; ++i) {
        const int64_t n = i == 0 ? rows : features;
        void *const place = arena.take(scale_tile_bytes(n, blocks));
        tiles[i] = {static_cast<const uint8_t *>(to[i]->p), static_cast<uint32_t *>(place), n,
                    (int32_t)blocks, i > 0};
        *to[i] = {place, scale_tile_pitch(n)};
    }
    const taco_status st = tile_scales(tiles, 3, stream);
    return st != TACO_OK ? st : Products<Codes>::run(Kind::kForward, p, stream);
}

taco_status taco_gated_mx_encode(const void *x, int64_t ldx, int64_t rows, int64_t hidden,
                                 taco_norm_dtype dtype, uint8_t *codes, uint8_t *scale_bytes,
                                 hipStream_t stream) {
    if (!valid(dtype)) return TACO_ERR_FORMAT;
    if (!valid_width(hidden) || hidden % 32 != 0 || !valid_rows(rows, hidden, ldx))
        return TACO_ERR_SHAPE;
    if (rows == 0) return TACO_OK;
    if (!x || !codes || !scale_bytes) return TACO_ERR_NULL;
    const int64_t size = size_of(dtype);
    if (!aligned(x, size)) return TACO_ERR_ALIGN;
    const Span outs[] = {{codes, rows * hidden}, {scale_bytes, rows * (hidden / 32)}};
    const Span ins[] = {{x, ((rows - 1) * ldx + hidden) * size}};
    if (any_overlap(outs, ins)) return TACO_ERR_ALIAS;
    return encode({x, codes, scale_bytes, ldx, rows, hidden}, dtype, stream);
}

}  // extern "C"
