// Argument checks that the C ABIs of libtaco_norm, libtaco_rms and libtaco_gated
// share (host code).
#pragma once

#include <stdint.h>

#include "taco_norm.h"

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

}  // namespace
