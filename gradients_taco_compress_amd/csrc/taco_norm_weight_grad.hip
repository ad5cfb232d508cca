// Weight gradient of a linear layer from the 8-bit checkpoint of its input
// (formula in taco_norm.h): dW = dY^T C, a matrix product whose right operand
// is one E4M3 code per element.
//
//  * A code has 4 significant bits, so it is exact in bf16 and fp16, and the
//    checkpoint's scale is one power of two: the matrix instructions
//    (16x16x32, float32 sums) see dY and the codes unrounded, and scale,
//    weight and bias enter at the end, per output column.
//  * Both operands have the summed index t as their slow one.  Tiles are
//    kept in LDS as they sit in memory ([t][n] and [t][k], the codes as
//    bytes: half the LDS traffic of a converted tile) and turned by the
//    transposing LDS reads on the way to registers; the codes are converted
//    there, four instructions per 16x32 fragment.
//  * LDS rows are a multiple of the banks' cycle, so a fragment's rows would
//    all start on one bank: the 32-byte (dY) or 16-byte (codes) units of row
//    t are stored at unit index XOR f(t), with f such that the rows a half
//    wave reads together fall on different banks.
//  * Global loads go straight to LDS (16 bytes per lane, no registers) where
//    rows start on 16-byte boundaries; other rows, and the last rows of a
//    tensor, pass through registers with every element checked.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "taco_norm.h"
#include "taco_norm_internal.hpp"

namespace taco_norm {
namespace {

typedef unsigned int u4v __attribute__((ext_vector_type(4)));
typedef unsigned int u2v __attribute__((ext_vector_type(2)));
typedef u4v u4v_any __attribute__((aligned(1)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef int i2v __attribute__((ext_vector_type(2)));
typedef short s4v __attribute__((ext_vector_type(4)));

constexpr int kWave = 64;
constexpr int kDepth = 64;             // t per tile

template <typename E>
struct Mfma;
template <>
struct Mfma<__bf16> {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ f4v run(v8 a, v8 b, f4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    static __device__ __forceinline__ v2 codes(uint32_t w) {
        return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
    }
};
template <>
struct Mfma<_Float16> {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ f4v run(v8 a, v8 b, f4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    template <bool HI>
    static __device__ __forceinline__ v2 codes(uint32_t w) {
        return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI);
    }
};

// Position of a unit in LDS row t (see the head of the file).  A fragment
// read of dY takes rows 8 g + (0..3) (then + 4) for g = 0..3, one of codes
// rows 8 g + (0..7); lanes 0-31 are g = 0, 1.
template <int BN>
__device__ __forceinline__ int turn_dy(int t) {
    return BN == 256 ? ((t & 3) | (((t >> 3) & 3) << 2)) : ((t & 3) | (((t >> 3) & 1) << 2));
}
template <int BK>
__device__ __forceinline__ int turn_codes(int t) {
    return BK == 256 ? (t & 15) : ((t >> 1) & 7);
}

template <typename E>
__device__ __forceinline__ float param(const void *p, int f32, int col, float missing) {
    if (!p) return missing;
    return f32 ? static_cast<const float *>(p)[col] : (float)static_cast<const E *>(p)[col];
}

// One output element from its raw sum: (w_k / S) sum + b_k db_n.
template <typename E>
__device__ __forceinline__ void finish(const WeightGrad &a, const float *db, int n, int k,
                                       float sum) {
    float v = sum * (param<E>(a.weight, a.params_f32, k, 1.0f) * a.inv_scale);
    if (a.bias) v = __builtin_fmaf(param<E>(a.bias, a.params_f32, k, 0.0f), db[n], v);
    const int64_t at = (int64_t)n * a.hidden + k;
    if (a.dw_f32) {
        float *p = static_cast<float *>(a.dw) + at;
        *p = a.accumulate ? *p + v : v;
    } else {
        static_cast<E *>(a.dw)[at] = (E)v;
    }
}

// Output tile (n0.., k0..) of BN x BK over rows [t0, t1): WN x WK waves, each
// BN / WN by BK / WK.  parts != null: raw sums go there (one [N][K] slab per
// blockIdx.y) instead of the finished gradient.
template <typename E, int BN, int BK, int WN, int WK, bool DIRECT>
__global__ __launch_bounds__(WN *WK *kWave) void grad_kernel(WeightGrad a, const float *db,
                                                             float *parts, int64_t slice) {
    constexpr int THREADS = WN * WK * kWave;
    constexpr int NI = BN / WN / 16, KI = BK / WK / 16;      // fragments of a wave
    constexpr int DY_BYTES = kDepth * BN * 2, CODE_BYTES = kDepth * BK;
    constexpr int DY_LOADS = DY_BYTES / 16 / THREADS, CODE_LOADS = CODE_BYTES / 16 / THREADS;
    constexpr int DY_CHUNKS = BN / 8, CODE_CHUNKS = BK / 16;  // 16-byte chunks of a row
    using M = Mfma<E>;
    __shared__ __align__(1024) uint8_t lds[2][DY_BYTES + CODE_BYTES];

    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int tiles_n = (a.out_features + BN - 1) / BN;
    const int tile_n = blockIdx.x % tiles_n, tile_k = blockIdx.x / tiles_n;
    const int n0 = tile_n * BN, k0 = tile_k * BK;
    const int64_t t0 = (int64_t)blockIdx.y * slice;
    const int64_t t1 = t0 + slice < a.rows ? t0 + slice : a.rows;
    const int steps = (int)((t1 - t0 + kDepth - 1) / kDepth);
    const char *const dy = static_cast<const char *>(a.dy);
    const char *const codes = reinterpret_cast<const char *>(a.codes);

    // Chunk i of this thread is LDS chunk i * THREADS + tid of the tile:
    // row and source column.
    auto dy_row = [&](int i) { return (i * THREADS + tid) / DY_CHUNKS; };
    auto dy_col = [&](int i) {
        const int c = (i * THREADS + tid) % DY_CHUNKS;
        return 8 * ((((c >> 1) ^ turn_dy<BN>(dy_row(i))) << 1) | (c & 1));
    };
    auto code_row = [&](int i) { return (i * THREADS + tid) / CODE_CHUNKS; };
    auto code_col = [&](int i) {
        return 16 * (((i * THREADS + tid) % CODE_CHUNKS) ^ turn_codes<BK>(code_row(i)));
    };

    // Straight to LDS: every row exists; a chunk past the last column reads
    // the tile's first one instead (its sums are never stored).
    auto load_direct = [&](int step, int buf) {
        const int64_t t = t0 + (int64_t)step * kDepth;
#pragma unroll
        for (int i = 0; i < DY_LOADS; ++i) {
            int col = n0 + dy_col(i);
            col = col < a.out_features ? col : n0;
            const char *p = dy + ((t + dy_row(i)) * a.lddy + col) * 2;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)p,
                (__attribute__((address_space(3))) void *)(lds[buf] +
                                                           (i * THREADS + wave * kWave) * 16),
                16, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < CODE_LOADS; ++i) {
            int col = k0 + code_col(i);
            col = col < a.hidden ? col : k0;
            const char *p = codes + (t + code_row(i)) * a.hidden + col;
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void *)p,
                (__attribute__((address_space(3))) void *)(lds[buf] + DY_BYTES +
                                                           (i * THREADS + wave * kWave) * 16),
                16, 0, 0);
        }
    };
    // Through registers: rows past t1 and columns past the last are zero.
    u4v held_dy[DY_LOADS], held_codes[CODE_LOADS];
    auto load_held = [&](int step) {
        const int64_t t = t0 + (int64_t)step * kDepth;
#pragma unroll
        for (int i = 0; i < DY_LOADS; ++i) {
            const int col = n0 + dy_col(i);
            const char *p = dy + ((t + dy_row(i)) * a.lddy + col) * 2;
            const int n = t + dy_row(i) < t1 ? a.out_features - col : 0;
            held_dy[i] = (u4v){0u, 0u, 0u, 0u};
            if (n >= 8) {
                held_dy[i] = *reinterpret_cast<const u4v_any *>(p);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < n)
                        held_dy[i][j >> 1] |= (uint32_t) reinterpret_cast<const uint16_t *>(p)[j]
                                              << (16 * (j & 1));
            }
        }
#pragma unroll
        for (int i = 0; i < CODE_LOADS; ++i) {
            const int col = k0 + code_col(i);
            const char *p = codes + (t + code_row(i)) * a.hidden + col;
            const int n = t + code_row(i) < t1 ? a.hidden - col : 0;
            held_codes[i] = (u4v){0u, 0u, 0u, 0u};
            if (n >= 16) {
                held_codes[i] = *reinterpret_cast<const u4v_any *>(p);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < n)
                        held_codes[i][j >> 2] |= (uint32_t)(uint8_t)p[j] << (8 * (j & 3));
            }
        }
    };
    auto store_held = [&](int buf) {
#pragma unroll
        for (int i = 0; i < DY_LOADS; ++i)
            *reinterpret_cast<u4v *>(lds[buf] + (i * THREADS + tid) * 16) = held_dy[i];
#pragma unroll
        for (int i = 0; i < CODE_LOADS; ++i)
            *reinterpret_cast<u4v *>(lds[buf] + DY_BYTES + (i * THREADS + tid) * 16) =
                held_codes[i];
    };
    auto is_direct = [&](int step) {
        return DIRECT && t0 + (int64_t)(step + 1) * kDepth <= t1;
    };

    // Fragment addresses: lane (g, r) = (lane / 16, lane % 16) reads 8 bytes
    // of row 8 g + r / 4 (dY; then + 4) or 8 g + r / 2 (codes); the read
    // hands lane (g, r) column r of those rows.
    const int g = lane >> 4, r = lane & 15;
    const int wn = wave / WK, wk = wave % WK;
    int dy_at[NI], code_at[KI];
    {
        const int t = 8 * g + (r >> 2);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            dy_at[i] = t * BN * 2 + (((wn * NI + i) ^ turn_dy<BN>(t)) * 32) + (r & 3) * 8;
    }
    {
        const int t = 8 * g + (r >> 1);
#pragma unroll
        for (int j = 0; j < KI; ++j)
            code_at[j] = DY_BYTES + t * BK + (((wk * KI + j) ^ turn_codes<BK>(t)) * 16) +
                         (r & 1) * 8;
    }

    f4v sum[KI][NI];
#pragma unroll
    for (int j = 0; j < KI; ++j)
#pragma unroll
        for (int i = 0; i < NI; ++i) sum[j][i] = (f4v){0.0f, 0.0f, 0.0f, 0.0f};

    auto multiply = [&](int buf) {
        uint8_t *const tile = lds[buf];
#pragma unroll
        for (int half = 0; half < kDepth / 32; ++half) {
            typename M::v8 fd[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                uint8_t *p = tile + dy_at[i] + half * 32 * BN * 2;
                union { s4v s[2]; typename M::v8 v; } u;
                u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s4v *)p);
                u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s4v *)(p + 4 * BN * 2));
                fd[i] = u.v;
            }
#pragma unroll
            for (int j = 0; j < KI; ++j) {
                uint8_t *p = tile + code_at[j] + half * 32 * BK;
                const i2v c = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (__attribute__((address_space(3))) i2v *)p);
                union { typename M::v2 h[4]; typename M::v8 v; } u;
                u.h[0] = M::template codes<false>((uint32_t)c[0]);
                u.h[1] = M::template codes<true>((uint32_t)c[0]);
                u.h[2] = M::template codes<false>((uint32_t)c[1]);
                u.h[3] = M::template codes<true>((uint32_t)c[1]);
#pragma unroll
                for (int i = 0; i < NI; ++i) sum[j][i] = M::run(u.v, fd[i], sum[j][i]);
            }
        }
    };

    if (is_direct(0)) {
        load_direct(0, 0);
    } else {
        load_held(0);
        store_held(0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (int step = 0; step < steps; ++step) {
        const int buf = step & 1;
        const bool more = step + 1 < steps;
        if (more) {
            if (is_direct(step + 1)) load_direct(step + 1, buf ^ 1);
            else load_held(step + 1);
        }
        multiply(buf);
        if (more && !is_direct(step + 1)) store_held(buf ^ 1);
        // The next tile is in LDS, and this one has been read by all.
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }

    // Lane (g, r) of a fragment's sums: column n = r, rows k = 4 g + (0..3).
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int n = n0 + (wn * NI + i) * 16 + r;
        if (n >= a.out_features) continue;
#pragma unroll
        for (int j = 0; j < KI; ++j) {
            const int k = k0 + (wk * KI + j) * 16 + 4 * g;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (k + e >= a.hidden) break;
                if (parts)
                    parts[((int64_t)blockIdx.y * a.out_features + n) * a.hidden + k + e] =
                        sum[j][i][e];
                else
                    finish<E>(a, db, n, k + e, sum[j][i][e]);
            }
        }
    }
}

// Adds the slabs of a split sum in order and finishes.
template <typename E>
__global__ __launch_bounds__(256) void join_kernel(WeightGrad a, const float *db,
                                                   const float *parts, int splits) {
    const int64_t count = (int64_t)a.out_features * a.hidden;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count;
         i += (int64_t)gridDim.x * 256) {
        float s = 0.0f;
        for (int p = 0; p < splits; ++p) s += parts[p * count + i];
        finish<E>(a, db, (int)(i / a.hidden), (int)(i % a.hidden), s);
    }
}

// Column sums of dY, first over the rows of a work-group (8 row lanes, 32
// lanes of 8 columns), then over the work-groups.
template <typename E>
__global__ __launch_bounds__(256) void column_parts_kernel(const E *dy, int64_t ld, int64_t rows,
                                                           int n, float *parts) {
    __shared__ float lds[8][256];
    const int c = threadIdx.x & 31, lane = threadIdx.x / 32;
    const int col = blockIdx.x * 256 + 8 * c;
    float s[8] = {};
    for (int64_t t = (int64_t)blockIdx.y * 8 + lane; t < rows; t += (int64_t)gridDim.y * 8) {
        const E *p = dy + t * ld + col;
        if (col + 8 <= n) {
            const u4v v = *reinterpret_cast<const u4v_any *>(p);
            typedef E e8 __attribute__((ext_vector_type(8)));
            const e8 e = __builtin_bit_cast(e8, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += (float)e[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < n) s[j] += (float)p[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[lane][8 * c + j] = s[j];
    __syncthreads();
    const int at = blockIdx.x * 256 + threadIdx.x;
    if (at < n) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += lds[i][threadIdx.x];
        parts[(int64_t)blockIdx.y * n + at] = v;
    }
}

__global__ __launch_bounds__(1024) void column_sums_kernel(const float *parts, int count, int n,
                                                           float *db, float *dbias) {
    __shared__ float lds[16][kWave];
    const int c = threadIdx.x & (kWave - 1), lane = threadIdx.x / kWave;
    const int at = blockIdx.x * kWave + c;
    float s = 0.0f;
    if (at < n)
        for (int i = lane; i < count; i += 16) s += parts[(int64_t)i * n + at];
    lds[lane][c] = s;
    __syncthreads();
    if (lane == 0 && at < n) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s += lds[i][c];
        db[at] = s;
        if (dbias) dbias[at] = s;
    }
}

// ---------------------------------------------------------------- host ----

struct Plan {
    bool big;              // 256 x 256 tiles, else 128 x 128
    int64_t tiles;
    int splits;            // of the sum over rows
    int64_t slice;         // rows of a split, a multiple of kDepth
    int column_parts;
    int64_t column_floats, slab_floats;   // workspace: column sums, then slabs
};

int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

Plan plan(int64_t rows, int64_t n, int64_t k) {
    Plan p;
    const int64_t big = up(n, 256) * up(k, 256);
    p.big = big >= 160;
    p.tiles = p.big ? big : up(n, 128) * up(k, 128);
    // Few tiles: the rows are split until every CU has work, but no split
    // is shorter than four tiles deep.
    int64_t s = p.big ? 1 : 512 / p.tiles;
    const int64_t most = up(rows, 4 * kDepth);
    s = s < 1 ? 1 : s < most ? s : most;
    p.slice = up(up(rows, s), kDepth) * kDepth;
    p.splits = (int)up(rows, p.slice);
    const int64_t wide = up(n, 256), deep = up(rows, 32);
    int64_t c = 1024 / wide;
    c = c < 1 ? 1 : c > 256 ? 256 : c;
    p.column_parts = (int)(c < deep ? c : deep);
    p.column_floats = up((p.column_parts + 1) * n, 4) * 4;
    p.slab_floats = p.splits > 1 ? p.splits * n * k : 0;
    return p;
}

template <typename E, int BN, int BK, int WN, int WK>
taco_status launch_grad(const WeightGrad &a, const Plan &p, const float *db, float *parts,
                        hipStream_t stream) {
    const bool direct = ((reinterpret_cast<uintptr_t>(a.dy) | (uintptr_t)(a.lddy * 2) |
                          reinterpret_cast<uintptr_t>(a.codes) | (uintptr_t)a.hidden) & 15u) == 0 &&
                        a.out_features % 8 == 0;
    const dim3 grid((unsigned)p.tiles, (unsigned)p.splits);
    return launch(direct ? reinterpret_cast<const void *>(&grad_kernel<E, BN, BK, WN, WK, true>)
                         : reinterpret_cast<const void *>(&grad_kernel<E, BN, BK, WN, WK, false>),
                  grid, WN * WK * kWave, stream, a, db, parts, p.slice);
}

template <typename E>
taco_status run(const WeightGrad &a, hipStream_t stream) {
    const Plan p = plan(a.rows, a.out_features, a.hidden);
    float *const db = a.workspace;
    float *const columns = db + a.out_features;
    float *const slabs = a.workspace + p.column_floats;
    taco_status st;
    if (a.bias || a.dbias) {
        st = launch(reinterpret_cast<const void *>(&column_parts_kernel<E>),
                    dim3((unsigned)up(a.out_features, 256), (unsigned)p.column_parts), 256, stream,
                    static_cast<const E *>(a.dy), a.lddy, a.rows, a.out_features, columns);
        if (st != TACO_OK) return st;
        st = launch(reinterpret_cast<const void *>(&column_sums_kernel),
                    dim3((unsigned)up(a.out_features, kWave)), 1024, stream,
                    static_cast<const float *>(columns), p.column_parts, a.out_features, db,
                    a.dbias);
        if (st != TACO_OK) return st;
    }
    float *const parts = p.splits > 1 ? slabs : nullptr;
    st = p.big ? launch_grad<E, 256, 256, 4, 2>(a, p, db, parts, stream)
               : launch_grad<E, 128, 128, 2, 2>(a, p, db, parts, stream);
    if (st != TACO_OK || !parts) return st;
    const int64_t groups = up((int64_t)a.out_features * a.hidden, 256);
    return launch(reinterpret_cast<const void *>(&join_kernel<E>),
                  dim3((unsigned)(groups < 8192 ? groups : 8192)), 256, stream, a,
                  static_cast<const float *>(db), static_cast<const float *>(parts), p.splits);
}

}  // namespace

int64_t weight_grad_workspace(int64_t rows, int64_t out_features, int64_t hidden) {
    const Plan p = plan(rows, out_features, hidden);
    return (p.column_floats + p.slab_floats) * (int64_t)sizeof(float);
}

taco_status weight_grad(const WeightGrad &a, taco_norm_dtype dtype, hipStream_t stream) {
    return dtype == TACO_NORM_BF16 ? run<__bf16>(a, stream) : run<_Float16>(a, stream);
}

}  // namespace taco_norm
