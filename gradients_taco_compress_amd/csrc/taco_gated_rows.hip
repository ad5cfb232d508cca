// The element-wise kernels of libtaco_gated: the gradients of both projections
// from that of their product, copies of operands to aligned rows, and the
// block-scaled 8-bit encoding of weights.  All of them stream HBM once: gradients of
// 8192 x 10240 bf16 140 us (6.0 TB/s), codes of 14336x3584 bf16 27.4 us (5.7) and float32
// 44.1 us (5.9), the scales of 16384 x 14336x3584 6.5 us.
#include "taco_gated_internal.hpp"
#include "taco_gated_device.hpp"
#include "taco_mx.hpp"

namespace taco_gated {
namespace {

template <typename T>
__device__ __forceinline__ void unpack8(u4v raw, float *f) {
    typedef T t8 __attribute__((ext_vector_type(8)));
    const t8 v = __builtin_bit_cast(t8, raw);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (float)v[j];
}
template <typename T>
__device__ __forceinline__ u4v pack8(const float *f) {
    typedef T t8 __attribute__((ext_vector_type(8)));
    typedef float f8 __attribute__((ext_vector_type(8)));
    f8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f[j];
    return __builtin_bit_cast(u4v, __builtin_convertvector(v, t8));
}

// Eight elements of a row, `n` of which exist (the others 0).
template <typename T>
__device__ __forceinline__ void load8(const T *p, const T *row, int n, float *f) {
    unpack8<T>(n >= 8 ? (u4v)*reinterpret_cast<const u4v_any *>(p)
                      : load_tail<true>(reinterpret_cast<const char *>(p),
                                        reinterpret_cast<const char *>(row), 2 * n),
               f);
}

// Work-group `at` of `of` that share the chunks of some rows.
struct Part {
    int64_t at, of;
};
// f(row, chunk) for this thread's chunks, one after the other along the rows: every
// thread has one, whatever a row's length.
template <typename F>
__device__ __forceinline__ void for_chunks(const Part &part, int64_t rows, int chunks, F &&f) {
    for (int64_t block = part.at; block * 256 < rows * chunks; block += part.of) {
        const int64_t first = block * 256 / chunks;
        const uint32_t at = (uint32_t)(block * 256 - first * chunks) + threadIdx.x;
        const uint32_t more = at / (uint32_t)chunks;
        const int64_t row = first + more;
        if (row < rows) f(row, (int)(at - more * (uint32_t)chunks));
    }
}

// A thread to eight neighbours.
template <typename T, int ACT>
__device__ __forceinline__ void activation_grad_rows(const ActivationGrad &a, const Part &part) {
    for_chunks(part, a.rows, (int)(a.to_pitch / 8), [&](int64_t row, int c) {
        const T *const da = static_cast<const T *>(a.da) + row * a.ldda;
        const T *const gate = static_cast<const T *>(a.gate) + row * a.ldgu;
        const T *const up = static_cast<const T *>(a.up) + row * a.ldgu;
        const int n = a.features - 8 * c;
        float d[8], g[8], u[8], dg[8], du[8];
        load8<T>(da + 8 * c, da, n, d);
        load8<T>(gate + 8 * c, gate, n, g);
        load8<T>(up + 8 * c, up, n, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float share = gate_share<ACT>(g[j]);
            dg[j] = d[j] * u[j] * gate_slope<ACT>(g[j], share);
            du[j] = d[j] * (g[j] * share);
            if (j >= n) dg[j] = du[j] = 0.0f;
        }
        *reinterpret_cast<u4v *>(static_cast<T *>(a.dgate) + row * a.to_pitch + 8 * c) = pack8<T>(dg);
        *reinterpret_cast<u4v *>(static_cast<T *>(a.dup) + row * a.to_pitch + 8 * c) = pack8<T>(du);
    });
}

__device__ __forceinline__ void repack_rows(const Repack &r, const Part &part) {
    for_chunks(part, r.rows, (int)(r.to_pitch / 16), [&](int64_t row, int c) {
        const char *const from = static_cast<const char *>(r.from) + row * r.from_pitch;
        const int64_t at = 16 * (int64_t)c, n = r.width - at;
        *reinterpret_cast<u4v *>(static_cast<char *>(r.to) + row * r.to_pitch + at) =
            n > 0 ? load_tail<true>(from + at, from, n < 16 ? (int)n : 16) : (u4v){0u, 0u, 0u, 0u};
    });
}

struct Copies {
    Repack r[3];
    int32_t groups[3];
};
// Work-group b of those that all copies take, one after the other.
__device__ __forceinline__ Part part_of_copies(const Copies &all, int b, int *which) {
    const int second = all.groups[0], third = second + all.groups[1];
    *which = (b >= second) + (b >= third);
    return {b - (b >= third ? third : b >= second ? second : 0), all.groups[*which]};
}
__global__ __launch_bounds__(256) void repack_kernel(Copies all) {
    int which;
    const Part part = part_of_copies(all, blockIdx.x, &which);
    repack_rows(all.r[which], part);
}

// The gradients of the activations, and the copies that the products after them need,
// in one launch.
template <typename T, int ACT>
__global__ __launch_bounds__(256) void activation_grad_kernel(ActivationGrad a, int groups, Copies copies) {
    const int b = (int)blockIdx.x;
    if (b < groups) {
        activation_grad_rows<T, ACT>(a, {b, groups});
    } else {
        int which;
        const Part part = part_of_copies(copies, b - groups, &which);
        repack_rows(copies.r[which], part);
    }
}

// A thread to four rows' bytes (rows r, 16 + r, 32 + r, 48 + r of 64) of four K-tiles.
struct AllScales {
    ScaleTiles s[3];
};
__global__ __launch_bounds__(256) void tile_scales_kernel(AllScales all) {
    const ScaleTiles s = all.s[blockIdx.y];
    const int64_t row_groups = (s.rows + 63) / 64, parts = (s.width + 15) / 16;
    const int64_t n = row_groups * 16 * parts;
    const int tiles = (s.width + 3) / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t part = i / (row_groups * 16), at = i - part * row_groups * 16;
        const int64_t group = at / 16;
        const int r = (int)(at % 16);
        u4v v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int in = 16 * q + r;
            const int64_t row = group * 64 + (s.features ? feature_of_row(in) : in);
            const char *const from = reinterpret_cast<const char *>(s.from) + row * s.width;
            const int left = s.width - (int)part * 16;
            v[q] = row < s.rows ? load_tail<true>(from + part * 16, from, left < 16 ? left : 16)
                                : (u4v){0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int64_t tile = part * 4 + d;
            if (tile >= tiles) break;
            uint32_t *const to = s.to + (tile * row_groups + group) * 64 + r;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t w = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) w |= ((v[q][d] >> (8 * g)) & 255u) << (8 * q);
                to[g * 16] = w;
            }
        }
    }
}

__global__ __launch_bounds__(256) void zero_kernel(uint16_t *p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        p[i] = 0;
}

template <typename T>
__device__ __forceinline__ void load8_any(const T *p, float *f) {
    if constexpr (sizeof(T) == 4) {
        const u4v a = reinterpret_cast<const u4v_any *>(p)[0], b = reinterpret_cast<const u4v_any *>(p)[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = __uint_as_float(a[j]);
            f[4 + j] = __uint_as_float(b[j]);
        }
    } else {
        unpack8<T>(*reinterpret_cast<const u4v_any *>(p), f);
    }
}

// A thread to eight neighbours, four threads to a block.
template <typename T>
__global__ __launch_bounds__(256) void encode_kernel(Encode e) {
    const int64_t per = e.hidden / 8, n = e.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per, c = i - row * per;
        float y[8];
        load8_any<T>(static_cast<const T *>(e.x) + row * e.ldx + 8 * c, y);
        const uint32_t byte = taco_mx::scale_byte(taco_mx::max_of_four(taco_mx::abs_max8(y)));
        *reinterpret_cast<u2v_any *>(e.codes + 8 * i) = taco_mx::codes8(y, byte);
        if ((i & 3) == 0) e.scales[i >> 2] = (uint8_t)byte;
    }
}

unsigned groups_of(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

}  // namespace

namespace {
Copies copies_of(const Repack *r, int count, int64_t *groups) {
    Copies all = {};
    *groups = 0;
    for (int i = 0; i < count; ++i) {
        all.r[i] = r[i];
        all.groups[i] = (int32_t)groups_of((r[i].rows * (r[i].to_pitch / 16) + 255) / 256, 1 << 16);
        *groups += all.groups[i];
    }
    return all;
}
}  // namespace

taco_status activation_grad(const ActivationGrad &a, bool f16, const Repack *r, int count,
                            hipStream_t stream) {
    const int groups = (int)groups_of((a.rows * (a.to_pitch / 8) + 255) / 256, 1 << 17);
    int64_t more;
    const Copies copies = copies_of(r, count, &more);
    const void *fn = nullptr;
    switch (a.activation) {
        case TACO_GATED_SILU:
            fn = f16 ? reinterpret_cast<const void *>(&activation_grad_kernel<_Float16, TACO_GATED_SILU>)
                     : reinterpret_cast<const void *>(&activation_grad_kernel<__bf16, TACO_GATED_SILU>);
            break;
        case TACO_GATED_GELU:
            fn = f16 ? reinterpret_cast<const void *>(&activation_grad_kernel<_Float16, TACO_GATED_GELU>)
                     : reinterpret_cast<const void *>(&activation_grad_kernel<__bf16, TACO_GATED_GELU>);
            break;
        default:
            fn = f16 ? reinterpret_cast<const void *>(&activation_grad_kernel<_Float16, TACO_GATED_GELU_TANH>)
                     : reinterpret_cast<const void *>(&activation_grad_kernel<__bf16, TACO_GATED_GELU_TANH>);
    }
    return launch(fn, dim3((unsigned)(groups + more)), 256, stream, a, groups, copies);
}

taco_status repack(const Repack *r, int count, hipStream_t stream) {
    int64_t groups;
    const Copies all = copies_of(r, count, &groups);
    return launch(reinterpret_cast<const void *>(&repack_kernel), dim3((unsigned)groups), 256, stream, all);
}

taco_status tile_scales(const ScaleTiles *s, int count, hipStream_t stream) {
    AllScales all = {};
    int64_t most = 1;
    for (int i = 0; i < count; ++i) {
        all.s[i] = s[i];
        const int64_t n = (s[i].rows + 63) / 64 * 16 * ((s[i].width + 15) / 16);
        most = n > most ? n : most;
    }
    return launch(reinterpret_cast<const void *>(&tile_scales_kernel),
                  dim3(groups_of((most + 255) / 256, 4096), (unsigned)count), 256, stream, all);
}

taco_status fill_zero(void *p, int64_t n16, hipStream_t stream) {
    return launch(reinterpret_cast<const void *>(&zero_kernel), dim3(groups_of((n16 + 255) / 256, 4096)),
                  256, stream, static_cast<uint16_t *>(p), n16);
}

taco_status encode(const Encode &e, taco_norm_dtype dtype, hipStream_t stream) {
    const dim3 grid(groups_of((e.rows * (e.hidden / 8) + 255) / 256, 8192));
    const void *fn = dtype == TACO_NORM_BF16  ? reinterpret_cast<const void *>(&encode_kernel<__bf16>)
                     : dtype == TACO_NORM_F16 ? reinterpret_cast<const void *>(&encode_kernel<_Float16>)
                                              : reinterpret_cast<const void *>(&encode_kernel<float>);
    return launch(fn, grid, 256, stream, e);
}

}  // namespace taco_gated
