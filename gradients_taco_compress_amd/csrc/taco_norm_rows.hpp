// Layer norm's row kernels for gfx950, templated on the activations' type:
// the forward pass with or without the 8-bit checkpoint, and the backward
// pass from the saved input or from the checkpoint (formulas in taco_norm.h).
//
// All of them stream HBM once: a row is held in registers between the
// reduction over it and the use of its result, so nothing is read twice.
//
//  * Layout.  A row belongs to TPR threads (16, 64, 256 or 512); thread t
//    holds the 8-element chunks c = 0..NV-1 at columns 8 (c TPR + t), so each
//    load instruction of a wave covers 1 KiB of a 16-bit row.  Rows shorter
//    than 256 threads' worth share a work-group.
//  * The reduction is DPP inside 16 lanes, v_readlane across a wave, LDS and
//    one barrier across waves (two LDS buffers alternate, so a row needs no
//    second barrier).  The forward pass merges per-wave means and squared
//    deviations, (n, sum, M2), instead of reducing twice.
//  * Work-groups stay and walk over rows with weight and bias in registers
//    (from L2, two float32 parameters per element would be four times the
//    bytes of the bf16 row itself); the next row's loads are issued before
//    the current row is reduced.
//  * Parameter gradients are sums over rows: each thread owns its columns for
//    all rows of its work-group and adds in registers; the work-groups'
//    sums go to the workspace and a second kernel adds them in a fixed
//    order, so results do not depend on timing.
//  * Rows wider than the registers hold (16384 columns; 12288 of float32 in the
//    backward pass) take the kernels at the end, which re-read the row from
//    the cache.
//
// Measured, bf16: forward 8192x2560 16.8 us (5.0 TB/s), with codes 16384x3584
// 54.3 us (5.4), backward 16384x3584 66.6 us (5.2), from codes 32768x12288 344 us
// (5.85); a 1 GiB copy reaches 5.13.  Calls below about 10 us are bound by their
// launches and the latency of a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "taco_norm.h"
#include "taco_norm_internal.hpp"
#include "taco_norm_device.hpp"

namespace taco_norm {
namespace {

typedef float f2v __attribute__((ext_vector_type(2)));
typedef float f4v __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ elements ----

// Eight elements as they sit in memory.
template <typename T>
struct Raw {
    u4v v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ float elem(const Raw<T> &r, int j) {
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(r.v[j >> 2][j & 3]);
    } else {
        const uint32_t w = r.v[0][j >> 1];
        if constexpr (__is_same(T, __bf16)) {
            return __uint_as_float((j & 1) ? (w & 0xFFFF0000u) : (w << 16));
        } else {
            typedef _Float16 h2 __attribute__((ext_vector_type(2)));
            return (float)__builtin_bit_cast(h2, w)[j & 1];
        }
    }
}

template <typename T>
__device__ __forceinline__ void opaque(Raw<T> &r) {
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) asm volatile("" : "+v"(r.v[i]));
}

// Rounds eight float32 to T, to nearest even.
template <typename T>
__device__ __forceinline__ Raw<T> pack(const float *f) {
    Raw<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.v[j >> 2][j & 3] = __float_as_uint(f[j]);
    } else {
        typedef T t2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r.v[0][j] = __builtin_bit_cast(
                uint32_t, __builtin_convertvector((f2v){f[2 * j], f[2 * j + 1]}, t2));
    }
    return r;
}

// Chunk at p of a row that starts at `row`, of which n elements (0..8) exist.
// WHOLE: rows start on 16-byte boundaries and hold whole chunks, so n is 0 or
// 8.  TINY: a row may be shorter than 16 bytes.  Missing elements are 0.
template <typename T, bool WHOLE, bool TINY>
__device__ __forceinline__ Raw<T> load_chunk(const T *p, const T *row, int n) {
    Raw<T> r;
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 2; ++i) r.v[i] = (u4v){0u, 0u, 0u, 0u};
    if constexpr (WHOLE) {
        if (n > 0) {
#pragma unroll
            for (unsigned i = 0; i < sizeof(T) / 2; ++i)
                r.v[i] = __builtin_nontemporal_load(reinterpret_cast<const u4v *>(p) + i);
        }
    } else if (n >= 8) {
#pragma unroll
        for (unsigned i = 0; i < sizeof(T) / 2; ++i)
            r.v[i] = reinterpret_cast<const u4v_any *>(p)[i];
    } else if (n > 0) {
#pragma unroll
        for (unsigned i = 0; i < sizeof(T) / 2; ++i) {
            const int bytes = n * (int)sizeof(T) - 16 * (int)i;
            if (bytes > 0)
                r.v[i] = load_tail<TINY>(reinterpret_cast<const char *>(p) + 16 * i,
                                         reinterpret_cast<const char *>(row), bytes);
        }
    }
    return r;
}

template <typename T, bool WHOLE>
__device__ __forceinline__ void store_chunk(T *p, int n, const Raw<T> &r) {
    if constexpr (WHOLE) {
        if (n > 0) {
#pragma unroll
            for (unsigned i = 0; i < sizeof(T) / 2; ++i)
                __builtin_nontemporal_store(r.v[i], reinterpret_cast<u4v *>(p) + i);
        }
    } else if (n >= 8) {
#pragma unroll
        for (unsigned i = 0; i < sizeof(T) / 2; ++i) reinterpret_cast<u4v_any *>(p)[i] = r.v[i];
    } else if (n > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= n) break;
            if constexpr (sizeof(T) == 4)
                p[j] = __builtin_bit_cast(T, (uint32_t)r.v[j >> 2][j & 3]);
            else
                p[j] = __builtin_bit_cast(T, (uint16_t)(r.v[0][j >> 1] >> (16 * (j & 1))));
        }
    }
}

template <bool WHOLE, bool TINY>
__device__ __forceinline__ u2v load_codes(const uint8_t *p, const uint8_t *row, int n) {
    u2v r = {0u, 0u};
    if constexpr (WHOLE) {
        if (n > 0) r = *reinterpret_cast<const u2v *>(p);
    } else if (n >= 8) {
        r = *reinterpret_cast<const u2v_any *>(p);
    } else if (n > 0) {
        if (!TINY || p + n - row >= 8) {
            // The row's last 8 bytes, moved down.
            const u2v v = *reinterpret_cast<const u2v_any *>(p + n - 8);
            const uint64_t w = (((uint64_t)v.y << 32) | v.x) >> (8 * (8 - n));
            r = (u2v){(uint32_t)w, (uint32_t)(w >> 32)};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t c = p[j < n ? j : n - 1];
                r[j >> 2] |= (j < n ? c : 0u) << (8 * (j & 3));
            }
        }
    }
    return r;
}

template <bool WHOLE>
__device__ __forceinline__ void store_codes(uint8_t *p, int n, u2v r) {
    if constexpr (WHOLE) {
        if (n > 0) __builtin_nontemporal_store(r, reinterpret_cast<u2v *>(p));
    } else if (n >= 8) {
        *reinterpret_cast<u2v_any *>(p) = r;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = (uint8_t)(r[j >> 2] >> (8 * (j & 3)));
    }
}

// E4M3 codes of S h, to nearest even (|S h| <= 448 up to rounding, far below
// the 464 from which the conversion overflows).  S is a power of two, so S h
// is exact; the +0 addend turns -0 into +0.
__device__ __forceinline__ u2v encode(const float *h, float scale) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __builtin_fmaf(h[j], scale, 0.0f);
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    return (u2v){(uint32_t)lo, (uint32_t)hi};
}

__device__ __forceinline__ void decode(const u2v c, float inv_scale, float *h) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f2v a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false);
        const f2v b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
        h[4 * i] = a.x * inv_scale;
        h[4 * i + 1] = a.y * inv_scale;
        h[4 * i + 2] = b.x * inv_scale;
        h[4 * i + 3] = b.y * inv_scale;
    }
}

// Parameters of a chunk in float32 (`missing` where there is no parameter).
template <typename T, bool TINY>
__device__ __forceinline__ void load_params(const void *p, bool f32, int col, int n, float missing,
                                            float *out) {
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = missing;
    if (!p || n <= 0) return;
    if (f32) {
        const float *q = static_cast<const float *>(p);
        const Raw<float> r = load_chunk<float, false, TINY>(q + col, q, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = elem<float>(r, j);
    } else {
        const T *q = static_cast<const T *>(p);
        const Raw<T> r = load_chunk<T, false, TINY>(q + col, q, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) out[j] = elem<T>(r, j);
    }
}

template <typename T>
__device__ __forceinline__ void store_param(void *p, bool f32, int64_t col, float v) {
    if (f32) static_cast<float *>(p)[col] = v;
    else static_cast<T *>(p)[col] = (T)v;
}

// ---------------------------------------------------------- reductions ----

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(
                   __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// Sum over 16 lanes (a DPP row): quad_perm xor 1 and xor 2, half-row mirror,
// row mirror.  Every lane of the row gets it.
__device__ __forceinline__ float sum16(float v) {
    v = dpp_add<0xB1>(v);
    v = dpp_add<0x4E>(v);
    v = dpp_add<0x141>(v);
    return dpp_add<0x140>(v);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Sum over min(TPR, 64) lanes; with TPR >= 64 every lane of the wave is active.
template <int TPR>
__device__ __forceinline__ float wave_sum(float v) {
    v = sum16(v);
    if constexpr (TPR == 16) return v;
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

template <int TPR>
constexpr int block_threads() { return TPR <= kWave ? 256 : TPR; }

__device__ __forceinline__ int chunk_len(int hidden, int col) {
    const int n = hidden - col;
    return n < 0 ? 0 : n < 8 ? n : 8;
}

// ------------------------------------------------------------- forward ----

template <typename T, int TPR, int NV, bool WHOLE, bool CODES>
__global__ __launch_bounds__(block_threads<TPR>()) void forward_kernel(Forward a) {
    constexpr int RPB = block_threads<TPR>() / TPR;     // rows per work-group
    constexpr int WPR = TPR / kWave;                    // waves per row (0: part of one)
    __shared__ float merge[2][WPR > 1 ? WPR : 1][2];
    const int t = threadIdx.x % TPR;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int hidden = a.hidden;
    const T *const x = static_cast<const T *>(a.x);
    T *const y = static_cast<T *>(a.y);

    int len[NV];
    float count = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        len[c] = chunk_len(hidden, 8 * (c * TPR + t));
        count += (float)len[c];
    }
    const int64_t stride = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    Raw<T> raw[NV];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
            raw[c] = load_chunk<T, WHOLE, TPR == 16>(x + r * a.ldx + 8 * (c * TPR + t),
                                                     x + r * a.ldx, len[c]);
    };
    // The row first: its statistics are needed before the parameters are.
    if (row < a.rows) load(row);
    float w[NV][8], b[NV][8];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int col = 8 * (c * TPR + t);
        load_params<T, TPR == 16>(a.weight, a.params_f32, col, len[c], 1.0f, w[c]);
        load_params<T, TPR == 16>(a.bias, a.params_f32, col, len[c], 0.0f, b[c]);
    }
    // Elements of the row this wave holds (of the 16 lanes, with TPR = 16).
    const float n_wave = wave_sum<TPR>(count);
    const float inv_n_wave = n_wave > 0.0f ? 1.0f / n_wave : 0.0f;
    const float n_row = (float)hidden;

    for (int turn = 0; row < a.rows; row += stride, turn ^= 1) {
        float v[NV][8];
        // Four sums each: shorter chains of additions, which round less.
        float sums[4] = {}, squares[4] = {};
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[c][j] = elem<T>(raw[c], j);
                sums[j & 3] += v[c][j];
            }
        if (row + stride < a.rows) load(row + stride);

        float sum = wave_sum<TPR>((sums[0] + sums[1]) + (sums[2] + sums[3]));
        const float mean_wave = sum * inv_n_wave;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = v[c][j] - mean_wave;
                if (WHOLE ? len[c] > 0 : j < len[c])
                    squares[j & 3] = __builtin_fmaf(d, d, squares[j & 3]);
            }
        float m2 = wave_sum<TPR>((squares[0] + squares[1]) + (squares[2] + squares[3]));
        float mean;
        if constexpr (WPR > 1) {
            // Sum of squared deviations from the row's mean: each wave's from
            // its own mean, plus n (wave mean - row mean)^2.  Only the last
            // waves can hold fewer elements, so n follows from the wave.
            if ((threadIdx.x & (kWave - 1)) == 0) {
                merge[turn][wave][0] = sum;
                merge[turn][wave][1] = m2;
            }
            __syncthreads();
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) sum += merge[turn][i][0];
            mean = sum / n_row;
            m2 = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                float n = 0.0f;
#pragma unroll
                for (int c = 0; c < NV; ++c) {
                    const int left = hidden - 8 * (c * TPR + i * kWave);
                    n += (float)(left < 0 ? 0 : left < 8 * kWave ? left : 8 * kWave);
                }
                const float d = n > 0.0f ? merge[turn][i][0] / n - mean : 0.0f;
                m2 += __builtin_fmaf(n * d, d, merge[turn][i][1]);
            }
        } else {
            mean = sum / n_row;
            const float d = mean_wave - mean;
            m2 = __builtin_fmaf(n_row * d, d, m2);
        }
        const float rstd = 1.0f / sqrtf(m2 / n_row + a.eps);
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            float h[8], o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[j] = (v[c][j] - mean) * rstd;
                o[j] = __builtin_fmaf(h[j], w[c][j], b[c][j]);
            }
            const int col = 8 * (c * TPR + t);
            store_chunk<T, WHOLE>(y + row * a.ldy + col, len[c], pack<T>(o));
            if constexpr (CODES)
                store_codes<WHOLE>(a.codes + row * hidden + col, len[c], encode(h, a.scale));
        }
    }
}

// ------------------------------------------------------------ backward ----

template <typename T, int TPR, int NV, bool WHOLE, bool CODES>
__global__ __launch_bounds__(block_threads<TPR>()) void backward_kernel(Backward a) {
    constexpr int RPB = block_threads<TPR>() / TPR;
    constexpr int WPR = TPR / kWave;
    __shared__ float merge[2][WPR > 1 ? WPR : 1][2];
    // Work-groups of several rows add their threads' column sums here.
    __shared__ f4v sums[RPB > 1 ? 2 : 1][RPB > 1 ? TPR * NV * 2 : 1];
    const int t = threadIdx.x % TPR;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int hidden = a.hidden;
    const T *const dy = static_cast<const T *>(a.dy);
    const T *const x = static_cast<const T *>(a.x);
    T *const dx = static_cast<T *>(a.dx);

    int len[NV];
    float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int col = 8 * (c * TPR + t);
        len[c] = chunk_len(hidden, col);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[c][j] = db[c][j] = 0.0f;
    }
    const float n_row = (float)hidden;
    const int64_t stride = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    // Rows as they are in memory: the current one and the next.  A short row's
    // values are kept in float32 until they are written, and its registers take
    // the row after the next at once (4096x4096 from the checkpoint: 25.1 us
    // with one row ahead, 23.7 us with two); a long one is unpacked again.
    constexpr bool kKeep = NV <= 2;
    struct Row {
        Raw<T> dy[NV], x[CODES ? 1 : NV];
        u2v codes[CODES ? NV : 1];
        float mean, rstd;
    };
    Row held[2];
    auto load = [&](int64_t r, Row &to) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = 8 * (c * TPR + t);
            to.dy[c] = load_chunk<T, WHOLE, TPR == 16>(dy + r * a.lddy + col, dy + r * a.lddy, len[c]);
            if constexpr (CODES)
                to.codes[c] = load_codes<WHOLE, TPR == 16>(a.codes + r * hidden + col,
                                                           a.codes + r * hidden, len[c]);
            else
                to.x[c] = load_chunk<T, WHOLE, TPR == 16>(x + r * a.ldx + col, x + r * a.ldx, len[c]);
        }
        to.rstd = a.rstd[r];
        to.mean = CODES ? 0.0f : a.mean[r];
    };
    // h of a chunk.  A missing element has dy = 0; its h must be finite too.
    auto normalised = [&](const Row &in, int c, float *h) {
        if constexpr (CODES) {
            decode(in.codes[c], a.inv_scale, h);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[j] = (elem<T>(in.x[c], j) - in.mean) * in.rstd;
                if (!(WHOLE ? len[c] > 0 : j < len[c])) h[j] = 0.0f;
            }
        }
    };
    auto process = [&](Row &in, Row &next, int turn) {
        if constexpr (!kKeep)
            if (row + stride < a.rows) load(row + stride, next);
        float g[kKeep ? NV : 1][8], h[kKeep ? NV : 1][8];
        const float r = in.rstd;
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            float *const gc = g[kKeep ? c : 0], *const hc = h[kKeep ? c : 0];
            normalised(in, c, hc);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = elem<T>(in.dy[c], j);
                dw[c][j] = __builtin_fmaf(d, hc[j], dw[c][j]);
                db[c][j] += d;
                gc[j] = d * w[c][j];
                c1 += gc[j];
                c2 = __builtin_fmaf(gc[j], hc[j], c2);
            }
        }
        if constexpr (kKeep)
            if (row + 2 * stride < a.rows) load(row + 2 * stride, in);

        c1 = wave_sum<TPR>(c1);
        c2 = wave_sum<TPR>(c2);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & (kWave - 1)) == 0) {
                merge[turn][wave][0] = c1;
                merge[turn][wave][1] = c2;
            }
            __syncthreads();
            c1 = c2 = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) {
                c1 += merge[turn][i][0];
                c2 += merge[turn][i][1];
            }
        }
        c1 /= n_row;
        c2 /= n_row;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            float *const gc = g[kKeep ? c : 0], *const hc = h[kKeep ? c : 0];
            if constexpr (!kKeep) {
                // Opaque, or the compiler keeps the values after all.
                opaque(in.dy[c]);
                if constexpr (CODES) asm volatile("" : "+v"(in.codes[c]));
                else opaque(in.x[c]);
                normalised(in, c, hc);
#pragma unroll
                for (int j = 0; j < 8; ++j) gc[j] = elem<T>(in.dy[c], j) * w[c][j];
            }
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = r * __builtin_fmaf(-hc[j], c2, gc[j] - c1);
            store_chunk<T, WHOLE>(dx + row * a.lddx + 8 * (c * TPR + t), len[c], pack<T>(o));
        }
        row += stride;
    };
    if (row < a.rows) load(row, held[0]);
    if (kKeep && row + stride < a.rows) load(row + stride, held[1]);
#pragma unroll
    for (int c = 0; c < NV; ++c)
        load_params<T, TPR == 16>(a.weight, a.params_f32, 8 * (c * TPR + t), len[c], 1.0f, w[c]);
    while (row < a.rows) {
        process(held[0], held[1], 0);
        if (row >= a.rows) break;
        process(held[1], held[0], 1);
    }

    if (!a.partial) return;
    float *const part = a.partial + (int64_t)blockIdx.x * 2 * hidden;
    if constexpr (RPB > 1) {
        // In the order of the rows' groups: the sum does not depend on timing.
        for (int group = 0; group < RPB; ++group) {
            if ((int)(threadIdx.x / TPR) == group) {
#pragma unroll
                for (int c = 0; c < NV; ++c)
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const int i = (c * 2 + j / 4) * TPR + t;
                        const f4v w4 = {dw[c][j], dw[c][j + 1], dw[c][j + 2], dw[c][j + 3]};
                        const f4v b4 = {db[c][j], db[c][j + 1], db[c][j + 2], db[c][j + 3]};
                        sums[0][i] = group == 0 ? w4 : sums[0][i] + w4;
                        sums[1][i] = group == 0 ? b4 : sums[1][i] + b4;
                    }
            }
            __syncthreads();
        }
        if (threadIdx.x >= TPR) return;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[c][j] = sums[0][(c * 2 + j / 4) * TPR + t][j % 4];
                db[c][j] = sums[1][(c * 2 + j / 4) * TPR + t][j % 4];
            }
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const int col = 8 * (c * TPR + t);
        if (WHOLE ? len[c] > 0 : len[c] == 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *s = i ? db[c] : dw[c];
                float *p = part + (int64_t)i * hidden + col;
                typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
                *reinterpret_cast<f4_any *>(p) = (f4_any){s[0], s[1], s[2], s[3]};
                *reinterpret_cast<f4_any *>(p + 4) = (f4_any){s[4], s[5], s[6], s[7]};
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < len[c]) {
                    part[col + j] = dw[c][j];
                    part[(int64_t)hidden + col + j] = db[c][j];
                }
        }
    }
}

// Parameter gradients from the work-groups' sums: one column per lane, 16
// lanes along the parts, added in a fixed order.  blockIdx.y: 0 dweight,
// 1 dbias.
constexpr int kSumThreads = 1024;
template <typename T>
__global__ __launch_bounds__(kSumThreads) void parts_kernel(const float *partial, int parts,
                                                            int hidden, void *dweight, void *dbias,
                                                            int params_f32) {
    constexpr int kLanes = kSumThreads / kWave;
    __shared__ float sums[kLanes][kWave];
    void *const out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int col = blockIdx.x * kWave + (threadIdx.x & (kWave - 1));
    const int lane = threadIdx.x / kWave;
    float s = 0.0f;
    if (col < hidden) {
        const float *p = partial + (int64_t)blockIdx.y * hidden + col;
#pragma unroll 8
        for (int i = lane; i < parts; i += kLanes) s += p[(int64_t)i * 2 * hidden];
    }
    sums[lane][threadIdx.x & (kWave - 1)] = s;
    __syncthreads();
    if (lane == 0 && col < hidden) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kLanes; ++i) s += sums[i][threadIdx.x];
        store_param<T>(out, params_f32, col, s);
    }
}

// ---------------------------------------------------------- wide rows -----

// Rows wider than the register kernels hold: one work-group per row, which
// is re-read for each pass over it (it stays in L2).
constexpr int kWideThreads = 1024;

__device__ __forceinline__ float group_sum(float v, float *lds) {
    v = wave_sum<kWave>(v);
    __syncthreads();                       // earlier readers are done
    if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0f;
    for (int i = 0; i < kWideThreads / kWave; ++i) v += lds[i];
    return v;
}

template <typename T>
__device__ __forceinline__ float param(const void *p, int f32, int64_t col, float missing) {
    if (!p) return missing;
    return f32 ? static_cast<const float *>(p)[col] : (float)static_cast<const T *>(p)[col];
}

__device__ __forceinline__ float decode1(uint8_t c) {
    return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}

template <typename T, bool CODES>
__global__ __launch_bounds__(kWideThreads) void forward_wide_kernel(Forward a) {
    __shared__ float lds[kWideThreads / kWave];
    const float n = (float)a.hidden;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.ldx;
        T *y = static_cast<T *>(a.y) + row * a.ldy;
        float s = 0.0f;
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads) s += (float)x[i];
        const float mean = group_sum(s, lds) / n;
        // Deviations from the mean as it is rounded, which is the one that h is
        // formed with: the sum of h^2 cannot pass hidden, whatever the rounding.
        s = 0.0f;
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads) {
            const float d = (float)x[i] - mean;
            s = __builtin_fmaf(d, d, s);
        }
        const float rstd = 1.0f / sqrtf(group_sum(s, lds) / n + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads) {
            const float h = ((float)x[i] - mean) * rstd;
            y[i] = (T)__builtin_fmaf(h, param<T>(a.weight, a.params_f32, i, 1.0f),
                                     param<T>(a.bias, a.params_f32, i, 0.0f));
            if constexpr (CODES) {
                const float q = __builtin_fmaf(h, a.scale, 0.0f);
                a.codes[row * a.hidden + i] =
                    (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false);
            }
        }
    }
}

template <typename T, bool CODES>
__device__ __forceinline__ float wide_h(const Backward &a, int64_t row, int i) {
    if constexpr (CODES) return decode1(a.codes[row * a.hidden + i]) * a.inv_scale;
    return ((float)static_cast<const T *>(a.x)[row * a.ldx + i] - a.mean[row]) * a.rstd[row];
}

template <typename T, bool CODES>
__global__ __launch_bounds__(kWideThreads) void backward_wide_kernel(Backward a) {
    __shared__ float lds[kWideThreads / kWave];
    const float n = (float)a.hidden;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
        T *dx = static_cast<T *>(a.dx) + row * a.lddx;
        float c1 = 0.0f, c2 = 0.0f;
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads) {
            const float g = (float)dy[i] * param<T>(a.weight, a.params_f32, i, 1.0f);
            c1 += g;
            c2 = __builtin_fmaf(g, wide_h<T, CODES>(a, row, i), c2);
        }
        c1 = group_sum(c1, lds) / n;
        c2 = group_sum(c2, lds) / n;
        const float r = a.rstd[row];
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads) {
            const float g = (float)dy[i] * param<T>(a.weight, a.params_f32, i, 1.0f);
            dx[i] = (T)(r * __builtin_fmaf(-wide_h<T, CODES>(a, row, i), c2, g - c1));
        }
    }
}

// Parameter gradients of wide rows: a column per thread, rows blockIdx.y,
// blockIdx.y + gridDim.y, ...  Runs before backward_wide_kernel, which may
// overwrite dy with dx.
template <typename T, bool CODES>
__global__ __launch_bounds__(256) void params_wide_kernel(Backward a) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.hidden) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float d = (float)static_cast<const T *>(a.dy)[row * a.lddy + i];
        dw = __builtin_fmaf(d, wide_h<T, CODES>(a, row, i), dw);
        db += d;
    }
    float *part = a.partial + (int64_t)blockIdx.y * 2 * a.hidden;
    part[i] = dw;
    part[a.hidden + i] = db;
}

// ---------------------------------------------------------------- host ----

// Threads per row and chunks per thread by row length: a wave to a row as long
// as it can hold it (no barrier, and the parameters are loaded once for many
// rows); measured at 16384x3584, a wave of 7 chunks 43 us, 256 threads of 2
// 45-49 us, and at 8192x2560 17.5 against 21.5 us.  Few rows cannot fill the
// GPU anyway, and a row is done sooner by four waves: up to 1024 rows, or 512
// where a quarter or more of their threads would be idle, which costs a 16-bit
// row of whole chunks more than it gains.  Four waves against one, in us:
//     bf16, 1 row of 2560                     2.9 and 3.5
//     bf16, 512 / 768 / 1024 x 1536           3.8, 4.2, 4.5 and 3.4, 3.5, 3.7
//     the same with codes                     3.5, 4.0, 4.4 and 3.5, 3.7, 3.9
//     bf16, 512 / 768 / 1024 x 2560           4.3, 4.8, 5.3 and 4.2, 4.3, 4.6
//     bf16, 512 / 768 / 1024 x 2048           3.9, 4.4, 5.0 and 4.3, 4.5, 4.7
//     bf16, 512 / 1024 / 2048 x 4096          4.8, 6.2, 9.4 and 6.3, 6.9, 9.5
//     float32, 512 / 1024 / 2048 x 2560       5.2, 7.0, 11.0 and 5.8, 6.9, 11.6
//     bf16, ragged, 512 / 1024 / 2048 x 1535  4.2, 6.1, 9.5 and 4.7, 6.0, 7.8
// (ragged with codes, 1024x1111: 6.2 and 6.8).
template <typename F>
taco_status for_forward_width(int64_t rows, int hidden, F &&f) {
    const int chunks = (hidden + 7) / 8;
    const bool idle = chunks <= 192 || (chunks > 256 && chunks <= 320);
    const int64_t few = f.size == 2 && f.whole && idle ? 512 : 1024;
    if (rows <= few && chunks > 64) {
        if (chunks <= 256) return f.template run<256, 1>();
        if (chunks <= 512) return f.template run<256, 2>();
    }
    if (chunks <= 16) return f.template run<16, 1>();
    if (chunks <= 32) return f.template run<16, 2>();
    if (chunks <= 64) return f.template run<64, 1>();
    if (chunks <= 128) return f.template run<64, 2>();
    if (chunks <= 192) return f.template run<64, 3>();
    if (chunks <= 256) return f.template run<64, 4>();
    if (chunks <= 320) return f.template run<64, 5>();
    if (chunks <= 384) return f.template run<64, 6>();
    if (chunks <= 448) return f.template run<64, 7>();
    if (chunks <= 512) return f.template run<64, 8>();
    if (chunks <= 768) return f.template run<256, 3>();
    if (chunks <= 1024) return f.template run<256, 4>();
    if (chunks <= 1536) return f.template run<256, 6>();
    return f.template run<256, 8>();
}
// The backward pass holds twice the row and the sums of its columns, so the
// work-group takes over earlier: waves of their own rows are faster up to 1024
// columns only.
template <typename F>
taco_status for_backward_width(int hidden, F &&f) {
    const int chunks = (hidden + 7) / 8;
    if (chunks <= 16) return f.template run<16, 1>();
    if (chunks <= 64) return f.template run<64, 1>();
    if (chunks <= 128) return f.template run<64, 2>();
    if (chunks <= 256) return f.template run<256, 1>();
    if (chunks <= 512) return f.template run<256, 2>();
    if (chunks <= 768) return f.template run<256, 3>();
    if (chunks <= 1024) return f.template run<512, 2>();
    if (chunks <= 1536 || F::kMaxHeld <= 1536 * 8) return f.template run<512, 3>();
    if constexpr (F::kMaxHeld > 1536 * 8) return f.template run<512, 4>();
}

inline bool on16(const void *p, int64_t ld, int64_t size) {
    return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * size)) & 15u) == 0;
}

inline unsigned grid_rows(int64_t rows, int rows_per_group, int64_t most) {
    const int64_t g = (rows + rows_per_group - 1) / rows_per_group;
    return (unsigned)(g < most ? g : most);
}

template <typename T>
struct ForwardLaunch {
    static constexpr int size = sizeof(T);
    Forward a;
    hipStream_t stream;
    bool whole;
    template <int TPR, int NV, bool WHOLE> taco_status go() const {
        constexpr int threads = block_threads<TPR>();
        // Threads for each of the 256 CUs: fewer where a thread holds more, so
        // that a wave takes several rows for one load of the parameters and
        // 16-32 KiB of rows are on their way to a CU (measured at 8192x2560:
        // 512 threads 17.6 us, 1024 19.3 us, 2048 20.8 us).
        constexpr int per_cu = 2048 / NV < 512 ? 512 : 2048 / NV;
        const unsigned grid = grid_rows(a.rows, threads / TPR, 256 * (per_cu / threads));
        if (a.codes)
            return launch(reinterpret_cast<const void *>(&forward_kernel<T, TPR, NV, WHOLE, true>),
                          dim3(grid), threads, stream, a);
        return launch(reinterpret_cast<const void *>(&forward_kernel<T, TPR, NV, WHOLE, false>),
                      dim3(grid), threads, stream, a);
    }
    template <int TPR, int NV> taco_status run() const {
        return whole ? go<TPR, NV, true>() : go<TPR, NV, false>();
    }
};

template <typename T>
struct BackwardLaunch {
    // Four chunks of float32, their sums and the next row's would not fit.
    static constexpr int kMaxHeld = sizeof(T) == 4 ? 512 * 24 : 512 * 32;
    Backward a;
    hipStream_t stream;
    bool whole;
    int64_t parts;
    template <int TPR, int NV, bool WHOLE> taco_status go() const {
        constexpr int threads = block_threads<TPR>();
        const unsigned grid = (unsigned)parts;
        if (a.codes)
            return launch(reinterpret_cast<const void *>(&backward_kernel<T, TPR, NV, WHOLE, true>),
                          dim3(grid), threads, stream, a);
        return launch(reinterpret_cast<const void *>(&backward_kernel<T, TPR, NV, WHOLE, false>),
                      dim3(grid), threads, stream, a);
    }
    template <int TPR, int NV> taco_status run() const {
        return whole ? go<TPR, NV, true>() : go<TPR, NV, false>();
    }
};

}  // namespace

template <typename K>
taco_status Rows<K>::forward(const Forward &a, hipStream_t stream) {
    using T = typename K::type;
    if (a.hidden > kMaxHeld) {
        const unsigned grid = grid_rows(a.rows, 1, 512);
        if (a.codes)
            return launch(reinterpret_cast<const void *>(&forward_wide_kernel<T, true>),
                          dim3(grid), kWideThreads, stream, a);
        return launch(reinterpret_cast<const void *>(&forward_wide_kernel<T, false>), dim3(grid),
                      kWideThreads, stream, a);
    }
    const bool whole = a.hidden % 8 == 0 && on16(a.x, a.ldx, sizeof(T)) &&
                       on16(a.y, a.ldy, sizeof(T)) &&
                       (reinterpret_cast<uintptr_t>(a.codes) & 7u) == 0;
    return for_forward_width(a.rows, a.hidden, ForwardLaunch<T>{a, stream, whole});
}

template <typename K>
taco_status Rows<K>::backward(const Backward &a, hipStream_t stream) {
    using T = typename K::type;
    const int64_t parts = backward_parts(a.rows, a.hidden);
    taco_status st;
    if (a.hidden > BackwardLaunch<T>::kMaxHeld) {
        if (a.partial) {
            const dim3 grid((unsigned)((a.hidden + 255) / 256), (unsigned)parts);
            st = launch(a.codes ? reinterpret_cast<const void *>(&params_wide_kernel<T, true>)
                                : reinterpret_cast<const void *>(&params_wide_kernel<T, false>),
                        grid, 256, stream, a);
            if (st != TACO_OK) return st;
        }
        st = launch(a.codes ? reinterpret_cast<const void *>(&backward_wide_kernel<T, true>)
                            : reinterpret_cast<const void *>(&backward_wide_kernel<T, false>),
                    dim3(grid_rows(a.rows, 1, 512)), kWideThreads, stream, a);
    } else {
        const bool whole = a.hidden % 8 == 0 && on16(a.dy, a.lddy, sizeof(T)) &&
                           on16(a.dx, a.lddx, sizeof(T)) &&
                           (a.codes ? (reinterpret_cast<uintptr_t>(a.codes) & 7u) == 0
                                    : on16(a.x, a.ldx, sizeof(T)));
        st = for_backward_width(a.hidden, BackwardLaunch<T>{a, stream, whole, parts});
    }
    if (st != TACO_OK || !a.partial) return st;
    return launch(reinterpret_cast<const void *>(&parts_kernel<T>),
                  dim3((unsigned)((a.hidden + kWave - 1) / kWave), 2), kSumThreads, stream,
                  static_cast<const float *>(a.partial), (int)parts, a.hidden, a.dweight, a.dbias,
                  a.params_f32);
}

}  // namespace taco_norm
