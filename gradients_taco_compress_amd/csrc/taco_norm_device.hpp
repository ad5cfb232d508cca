// Device code that the kernels of libtaco_norm share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace taco_norm {
namespace {

typedef unsigned int u4v __attribute__((ext_vector_type(4)));
typedef unsigned int u2v __attribute__((ext_vector_type(2)));
// The same at any address (gfx950 reads and writes global memory unaligned).
typedef u4v u4v_any __attribute__((aligned(1)));
typedef u2v u2v_any __attribute__((aligned(1)));

constexpr int kWave = 64;

// 16 bytes at p, of which the first n (1..16) belong to a row that starts at
// `row`: the others are zero, and nothing outside the row is read.  TINY: the
// row may be shorter than 16 bytes.
template <bool TINY>
__device__ __forceinline__ u4v load_tail(const char *p, const char *row, int n) {
    if (n >= 16) return *reinterpret_cast<const u4v_any *>(p);
    if (!TINY || p + n - row >= 16) {
        // The row's last 16 bytes, moved down.
        const u4v v = *reinterpret_cast<const u4v_any *>(p + n - 16);
        const uint64_t lo = ((uint64_t)v.y << 32) | v.x, hi = ((uint64_t)v.w << 32) | v.z;
        const int sh = 8 * (16 - n);
        const uint64_t a = sh >= 64 ? hi >> (sh - 64) : (lo >> sh) | (hi << (64 - sh));
        const uint64_t b = sh >= 64 ? 0 : hi >> sh;
        return (u4v){(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
    }
    u4v v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t c = (uint8_t)p[j < n ? j : n - 1];
        v[j >> 2] |= (j < n ? c : 0u) << (8 * (j & 3));
    }
    return v;
}

}  // namespace
}  // namespace taco_norm
