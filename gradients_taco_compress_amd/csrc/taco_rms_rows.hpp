// Root-mean-square norm's row kernels for gfx950, templated on the activations'
// type: the forward pass with or without the residual's addition, into rows of
// the same type or into 8-bit codes with block scales, and the backward pass
// (formulas in taco_rms.h, the 8-bit form in taco_mx.hpp).
//
// They are laid out as layer norm's (taco_norm_rows.hpp): a row belongs to TPR
// threads, is held in registers between the reduction over it and the use of its
// result, the next row's loads are issued before the current row is reduced,
// and parameter gradients are added per work-group, then over work-groups in a
// fixed order.  What differs:
//
//  * One sum per row, and no mean: sums of squares are joined by adding.
//  * Few rows have their weight's gradient made by work-groups of its own, in the
//    same launch as dx.
//  * y is formed from the float32 sum x + residual; the sum that is written
//    is that value rounded once.
//  * 8-bit form: a block of 32 columns is four neighbouring lanes' chunks, so its
//    maximum takes two DPP steps, and its scale byte is written by the first
//    of the four.
//
// All are bound by HBM, whose copies reach 5.14 TB/s here (reading and writing): forward with
// residual 16384x3584 bf16 83 us (5.66 TB/s), float32 188 us (5.0) and 2048x2560 float32
// 19.0 us (4.4), into 8 bits 8192x2560 27.6 us (5.3), backward 32768x12288 bf16 with dtotal
// 548 us (5.87); the smallest calls by the launch, 1x2560 forward 2.0 to 2.5 us of kernel in
// a call of 5.3 or more.  Backward, wide rows spill registers: APART beyond 6144 columns (192
// to 568 bytes a thread); else most ragged rows beyond 8192 columns and whole ones with dtotal
// beyond 12288 (float32: 6144 and 8192), 40 to 592 bytes.
#pragma once

#include "taco_norm_rows.hpp"
#include "taco_rms_internal.hpp"
#include "taco_mx.hpp"

namespace taco_norm {
namespace {

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T> &r, float *f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = elem<T>(r, j);
}

// ------------------------------------------------------------- forward ----

template <typename T, int TPR, int NV, bool WHOLE, bool RES, bool MX>
__global__ __launch_bounds__(block_threads<TPR>()) void rms_forward_kernel(RmsForward a) {
    constexpr int RPB = block_threads<TPR>() / TPR;     // rows per work-group
    constexpr int WPR = TPR / kWave;                    // waves per row (0: part of one)
    __shared__ float merge[2][WPR > 1 ? WPR : 1];
    const int t = threadIdx.x % TPR;
    [[maybe_unused]] const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int hidden = a.hidden;
    const T *const x = static_cast<const T *>(a.x);
    const T *const res = static_cast<const T *>(a.residual);

    int len[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) len[c] = chunk_len(hidden, 8 * (c * TPR + t));
    const int64_t stride = (int64_t)gridDim.x * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    Raw<T> raw[NV], more[RES ? NV : 1];
    auto load = [&](int64_t r) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = 8 * (c * TPR + t);
            raw[c] = load_chunk<T, WHOLE, TPR == 16>(x + r * a.ldx + col, x + r * a.ldx, len[c]);
            if constexpr (RES)
                more[c] = load_chunk<T, WHOLE, TPR == 16>(res + r * a.ldr + col, res + r * a.ldr, len[c]);
        }
    };
    // The row first: its statistics are needed before the weight is.
    if (row < a.rows) load(row);
    float w[NV][8];
#pragma unroll
    for (int c = 0; c < NV; ++c)
        load_params<T, TPR == 16>(a.weight, a.params_f32, 8 * (c * TPR + t), len[c], 1.0f, w[c]);

    for (int turn = 0; row < a.rows; row += stride, turn ^= 1) {
        float v[NV][8];
        // Four sums: shorter chains of additions, which round less.
        float squares[4] = {};
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            unpack<T>(raw[c], v[c]);
            if constexpr (RES) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[c][j] += elem<T>(more[c], j);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) squares[j & 3] = __builtin_fmaf(v[c][j], v[c][j], squares[j & 3]);
        }
        if (row + stride < a.rows) load(row + stride);
        float sum = wave_sum<TPR>((squares[0] + squares[1]) + (squares[2] + squares[3]));
        if constexpr (WPR > 1) {
            if ((threadIdx.x & (kWave - 1)) == 0) merge[turn][wave] = sum;
            __syncthreads();
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) sum += merge[turn][i];
        }
        const float rstd = 1.0f / sqrtf(sum / (float)hidden + a.eps);
        if (!MX && t == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = 8 * (c * TPR + t);
            if constexpr (RES)
                if (a.total) store_chunk<T, WHOLE>(static_cast<T *>(a.total) + row * a.ldt + col, len[c], pack<T>(v[c]));
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = v[c][j] * rstd * w[c][j];
            if constexpr (MX) {
                // (rows hold whole blocks: four lanes have a chunk or none has)
                const uint32_t byte = taco_mx::scale_byte(taco_mx::max_of_four(taco_mx::abs_max8(o)));
                store_codes<WHOLE>(a.codes + row * hidden + col, len[c], taco_mx::codes8(o, byte));
                if (len[c] > 0 && (t & 3) == 0) a.scales[row * (hidden / 32) + col / 32] = (uint8_t)byte;
            } else {
                store_chunk<T, WHOLE>(static_cast<T *>(a.y) + row * a.ldy + col, len[c], pack<T>(o));
            }
        }
    }
}

// ------------------------------------------------------------ backward ----

// The weight's gradient of 64 columns over segment `segment` of the rows: eight lanes
// to a row, rows in turn, and the row groups' sums added in order.
template <typename T, int THREADS>
__device__ __forceinline__ void weight_columns(const RmsBackward &a, int col0, int segment) {
    constexpr int GROUPS = THREADS / 8;
    __shared__ f4v sums[GROUPS][8][2];
    const int64_t per = (a.rows + a.segments - 1) / a.segments, begin = segment * per;
    const int64_t end = begin + per < a.rows ? begin + per : a.rows;
    const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
    const int col = col0 + 8 * lane, len = chunk_len(a.hidden, col);
    const T *const dy = static_cast<const T *>(a.dy);
    const T *const x = static_cast<const T *>(a.x);
    float dw[8] = {};
#pragma unroll 4
    for (int64_t row = begin + group; row < end; row += GROUPS) {
        const Raw<T> d = load_chunk<T, false, true>(dy + row * a.lddy + col, dy + row * a.lddy, len);
        const Raw<T> v = load_chunk<T, false, true>(x + row * a.ldx + col, x + row * a.ldx, len);
        const float q = a.rstd[row];
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = __builtin_fmaf(elem<T>(d, j), elem<T>(v, j) * q, dw[j]);
    }
    sums[group][lane][0] = (f4v){dw[0], dw[1], dw[2], dw[3]};
    sums[group][lane][1] = (f4v){dw[4], dw[5], dw[6], dw[7]};
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= 64 || col0 + c >= a.hidden) return;
    float s = 0.0f;
#pragma unroll 8
    for (int g = 0; g < GROUPS; ++g) s += sums[g][c / 8][c / 4 % 2][c % 4];
    if (a.segments == 1) store_param<T>(a.dweight, a.params_f32, col0 + c, s);
    else a.partial[(int64_t)segment * a.hidden + col0 + c] = s;
}

// APART (few rows): the first row_groups work-groups make dx alone, the others the
// weight's gradient, 64 columns of a segment of the rows each, from a second look at dy
// and x, which the caches still hold.  One segment leaves no sums to join: one launch.
template <typename T, int TPR, int NV, bool WHOLE, bool RES, bool APART>
__global__ __launch_bounds__(block_threads<TPR>()) void rms_backward_kernel(RmsBackward a) {
    constexpr int RPB = block_threads<TPR>() / TPR;
    constexpr int WPR = TPR / kWave;
    if constexpr (APART) {
        if ((int)blockIdx.x >= a.row_groups) {
            const int b = (int)blockIdx.x - a.row_groups, columns = (a.hidden + 63) / 64;
            weight_columns<T, block_threads<TPR>()>(a, b % columns * 64, b / columns);
            return;
        }
    }
    __shared__ float merge[2][WPR > 1 ? WPR : 1];
    // Work-groups of several rows add their threads' column sums here.
    __shared__ f4v sums[RPB > 1 && !APART ? TPR * NV * 2 : 1];
    const int t = threadIdx.x % TPR;
    [[maybe_unused]] const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int hidden = a.hidden;
    const T *const dy = static_cast<const T *>(a.dy);
    const T *const x = static_cast<const T *>(a.x);
    const T *const dt = static_cast<const T *>(a.dtotal);

    int len[NV];
    float w[NV][8];
    [[maybe_unused]] float dw[NV][8];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        len[c] = chunk_len(hidden, 8 * (c * TPR + t));
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[c][j] = 0.0f;
    }
    const int64_t stride = (int64_t)a.row_groups * RPB;
    int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    // Rows as they are in memory: the current one and the next.
    struct Row {
        Raw<T> dy[NV], x[NV], dt[RES ? NV : 1];
        float rstd;
    };
    Row held[2];
    auto load = [&](int64_t r, Row &to) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const int col = 8 * (c * TPR + t);
            to.dy[c] = load_chunk<T, WHOLE, TPR == 16>(dy + r * a.lddy + col, dy + r * a.lddy, len[c]);
            to.x[c] = load_chunk<T, WHOLE, TPR == 16>(x + r * a.ldx + col, x + r * a.ldx, len[c]);
            if constexpr (RES)
                to.dt[c] = load_chunk<T, WHOLE, TPR == 16>(dt + r * a.lddt + col, dt + r * a.lddt, len[c]);
        }
        to.rstd = a.rstd[r];
    };
    auto process = [&](Row &in, Row &next, int turn) {
        if (row + stride < a.rows) load(row + stride, next);
        const float q = in.rstd;
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // (a missing element has dy = 0 and x = 0)
                const float d = elem<T>(in.dy[c], j), h = elem<T>(in.x[c], j) * q;
                if constexpr (!APART) dw[c][j] = __builtin_fmaf(d, h, dw[c][j]);
                dot = __builtin_fmaf(d * w[c][j], h, dot);
            }
        dot = wave_sum<TPR>(dot);
        if constexpr (WPR > 1) {
            if ((threadIdx.x & (kWave - 1)) == 0) merge[turn][wave] = dot;
            __syncthreads();
            dot = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) dot += merge[turn][i];
        }
        const float c2 = dot / (float)hidden;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            // Unpacked again (opaque, or the compiler keeps the values after all).
            opaque(in.dy[c]);
            opaque(in.x[c]);
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float h = elem<T>(in.x[c], j) * q;
                o[j] = q * __builtin_fmaf(-h, c2, elem<T>(in.dy[c], j) * w[c][j]);
                if constexpr (RES) o[j] += elem<T>(in.dt[c], j);
            }
            store_chunk<T, WHOLE>(static_cast<T *>(a.dx) + row * a.lddx + 8 * (c * TPR + t), len[c], pack<T>(o));
        }
        row += stride;
    };
    if (row < a.rows) load(row, held[0]);
#pragma unroll
    for (int c = 0; c < NV; ++c)
        load_params<T, TPR == 16>(a.weight, a.params_f32, 8 * (c * TPR + t), len[c], 1.0f, w[c]);
    while (row < a.rows) {
        process(held[0], held[1], 0);
        if (row >= a.rows) break;
        process(held[1], held[0], 1);
    }

    if constexpr (APART) return;
    if (!a.partial) return;
    float *const part = a.partial + (int64_t)blockIdx.x * hidden;
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
                        sums[i] = group == 0 ? w4 : sums[i] + w4;
                    }
            }
            __syncthreads();
        }
        if (threadIdx.x >= TPR) return;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) dw[c][j] = sums[(c * 2 + j / 4) * TPR + t][j % 4];
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        float *const p = part + 8 * (c * TPR + t);
        if (WHOLE ? len[c] > 0 : len[c] == 8) {
            typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<f4_any *>(p) = (f4_any){dw[c][0], dw[c][1], dw[c][2], dw[c][3]};
            *reinterpret_cast<f4_any *>(p + 4) = (f4_any){dw[c][4], dw[c][5], dw[c][6], dw[c][7]};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < len[c]) p[j] = dw[c][j];
        }
    }
}

// The weight's gradient from the work-groups' sums: one column per lane, 16
// lanes along the parts, added in a fixed order.
template <typename T>
__global__ __launch_bounds__(kSumThreads) void rms_parts_kernel(const float *partial, int parts,
                                                                int hidden, void *dweight,
                                                                int params_f32) {
    constexpr int kLanes = kSumThreads / kWave;
    __shared__ float sums[kLanes][kWave];
    const int col = blockIdx.x * kWave + (threadIdx.x & (kWave - 1));
    const int lane = threadIdx.x / kWave;
    float s = 0.0f;
    if (col < hidden) {
        const float *p = partial + col;
#pragma unroll 8
        for (int i = lane; i < parts; i += kLanes) s += p[(int64_t)i * hidden];
    }
    sums[lane][threadIdx.x & (kWave - 1)] = s;
    __syncthreads();
    if (lane == 0 && col < hidden) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kLanes; ++i) s += sums[i][threadIdx.x];
        store_param<T>(dweight, params_f32, col, s);
    }
}

// ---------------------------------------------------------- wide rows -----

// One work-group per row, which is re-read for each pass over it.
template <typename T, bool RES, bool MX>
__global__ __launch_bounds__(kWideThreads) void rms_forward_wide_kernel(RmsForward a) {
    __shared__ float lds[kWideThreads / kWave];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.ldx;
        const T *res = static_cast<const T *>(a.residual) + row * a.ldr;
        auto value = [&](int i) { return RES ? (float)x[i] + (float)res[i] : (float)x[i]; };
        float s = 0.0f;
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads) {
            const float v = value(i);
            s = __builtin_fmaf(v, v, s);
        }
        const float rstd = 1.0f / sqrtf(group_sum(s, lds) / (float)a.hidden + a.eps);
        if (!MX && threadIdx.x == 0 && a.rstd) a.rstd[row] = rstd;
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads) {
            const float v = value(i);
            // (each element is read, then written, by one thread: total may be x or residual)
            if (RES && a.total) static_cast<T *>(a.total)[row * a.ldt + i] = (T)v;
            const float o = v * rstd * param<T>(a.weight, a.params_f32, i, 1.0f);
            if constexpr (MX) {
                // 32 neighbouring lanes hold a block, all of it.
                uint32_t m = __float_as_uint(o) & 0x7FFFFFFFu;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t other = (uint32_t)__shfl_xor((int)m, d);
                    m = other > m ? other : m;
                }
                const uint32_t byte = taco_mx::scale_byte(m);
                const float all[8] = {o, o, o, o, o, o, o, o};
                a.codes[row * a.hidden + i] = (uint8_t)taco_mx::codes8(all, byte).x;
                if ((i & 31) == 0) a.scales[row * (a.hidden / 32) + i / 32] = (uint8_t)byte;
            } else {
                static_cast<T *>(a.y)[row * a.ldy + i] = (T)o;
            }
        }
    }
}

template <typename T, bool RES>
__global__ __launch_bounds__(kWideThreads) void rms_backward_wide_kernel(RmsBackward a) {
    __shared__ float lds[kWideThreads / kWave];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *dy = static_cast<const T *>(a.dy) + row * a.lddy;
        const T *x = static_cast<const T *>(a.x) + row * a.ldx;
        const T *dt = static_cast<const T *>(a.dtotal) + row * a.lddt;
        T *dx = static_cast<T *>(a.dx) + row * a.lddx;
        const float q = a.rstd[row];
        float dot = 0.0f;
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads)
            dot = __builtin_fmaf((float)dy[i] * param<T>(a.weight, a.params_f32, i, 1.0f), (float)x[i] * q, dot);
        const float c2 = group_sum(dot, lds) / (float)a.hidden;
        for (int i = threadIdx.x; i < a.hidden; i += kWideThreads) {
            const float g = (float)dy[i] * param<T>(a.weight, a.params_f32, i, 1.0f);
            float o = q * __builtin_fmaf(-(float)x[i] * q, c2, g);
            if (RES) o += (float)dt[i];
            dx[i] = (T)o;
        }
    }
}

// The weight's gradient of wide rows: a column per thread, rows blockIdx.y,
// blockIdx.y + gridDim.y, ...  Runs before rms_backward_wide_kernel, which may
// overwrite dy with dx.
template <typename T>
__global__ __launch_bounds__(256) void rms_weight_wide_kernel(RmsBackward a) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= a.hidden) return;
    float dw = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
        dw = __builtin_fmaf((float)static_cast<const T *>(a.dy)[row * a.lddy + i],
                            (float)static_cast<const T *>(a.x)[row * a.ldx + i] * a.rstd[row], dw);
    a.partial[(int64_t)blockIdx.y * a.hidden + i] = dw;
}

// ---------------------------------------------------------------- host ----

template <typename T>
struct RmsForwardLaunch {
    static constexpr int size = sizeof(T);
    RmsForward a;
    hipStream_t stream;
    bool whole;
    template <int TPR, int NV, bool WHOLE> taco_status go() const {
        constexpr int threads = block_threads<TPR>();
        constexpr int per_cu = 2048 / NV < 512 ? 512 : 2048 / NV;
        const unsigned grid = grid_rows(a.rows, threads / TPR, 256 * (per_cu / threads));
        const void *fn = nullptr;
        if (a.codes)
            fn = a.residual ? reinterpret_cast<const void *>(&rms_forward_kernel<T, TPR, NV, WHOLE, true, true>)
                            : reinterpret_cast<const void *>(&rms_forward_kernel<T, TPR, NV, WHOLE, false, true>);
        else
            fn = a.residual ? reinterpret_cast<const void *>(&rms_forward_kernel<T, TPR, NV, WHOLE, true, false>)
                            : reinterpret_cast<const void *>(&rms_forward_kernel<T, TPR, NV, WHOLE, false, false>);
        return launch(fn, dim3(grid), threads, stream, a);
    }
    template <int TPR, int NV> taco_status run() const {
        return whole ? go<TPR, NV, true>() : go<TPR, NV, false>();
    }
};

template <typename T>
struct RmsBackwardLaunch {
    static constexpr int kMaxHeld = sizeof(T) == 4 ? 512 * 24 : 512 * 32;
    RmsBackward a;
    hipStream_t stream;
    bool whole, apart;
    template <int TPR, int NV, bool WHOLE, bool APART>
    taco_status go(const RmsBackward &a, int64_t grid) const {
        const void *fn =
            a.dtotal ? reinterpret_cast<const void *>(&rms_backward_kernel<T, TPR, NV, WHOLE, true, APART>)
                     : reinterpret_cast<const void *>(&rms_backward_kernel<T, TPR, NV, WHOLE, false, APART>);
        return launch(fn, dim3((unsigned)grid), block_threads<TPR>(), stream, a);
    }
    template <int TPR, int NV> taco_status run() const {
        if (!apart)
            return whole ? go<TPR, NV, true, false>(a, a.row_groups) : go<TPR, NV, false, false>(a, a.row_groups);
        // (The loads of whole chunks are not to be kept; these are read twice.)
        const int64_t columns = (a.hidden + 63) / 64 * a.segments;
        if (a.dx != a.dy) return go<TPR, NV, false, true>(a, a.row_groups + columns);
        // dx in dy's place: after those who read dy.
        RmsBackward first = a;
        first.row_groups = 0;
        const taco_status st = go<TPR, NV, false, true>(first, columns);
        return st != TACO_OK ? st : go<TPR, NV, false, true>(a, a.row_groups);
    }
};

}  // namespace

template <typename K>
taco_status Rms<K>::forward(const RmsForward &a, hipStream_t stream) {
    using T = typename K::type;
    if (a.hidden > kMaxHeld) {
        const void *fn = nullptr;
        if (a.codes)
            fn = a.residual ? reinterpret_cast<const void *>(&rms_forward_wide_kernel<T, true, true>)
                            : reinterpret_cast<const void *>(&rms_forward_wide_kernel<T, false, true>);
        else
            fn = a.residual ? reinterpret_cast<const void *>(&rms_forward_wide_kernel<T, true, false>)
                            : reinterpret_cast<const void *>(&rms_forward_wide_kernel<T, false, false>);
        return launch(fn, dim3(grid_rows(a.rows, 1, 512)), kWideThreads, stream, a);
    }
    const bool whole = a.hidden % 8 == 0 && on16(a.x, a.ldx, sizeof(T)) &&
                       (!a.residual || on16(a.residual, a.ldr, sizeof(T))) &&
                       (!a.total || on16(a.total, a.ldt, sizeof(T))) &&
                       (a.codes ? (reinterpret_cast<uintptr_t>(a.codes) & 7u) == 0
                                : on16(a.y, a.ldy, sizeof(T)));
    return for_forward_width(a.rows, a.hidden, RmsForwardLaunch<T>{a, stream, whole});
}

template <typename K>
taco_status Rms<K>::backward(const RmsBackward &args, hipStream_t stream) {
    using T = typename K::type;
    RmsBackward a = args;
    const int64_t parts = rms_parts(a.rows, a.hidden);
    a.row_groups = (int32_t)parts;
    taco_status st;
    if (a.hidden > RmsBackwardLaunch<T>::kMaxHeld) {
        if (a.partial) {
            st = launch(reinterpret_cast<const void *>(&rms_weight_wide_kernel<T>),
                        dim3((unsigned)((a.hidden + 255) / 256), (unsigned)parts), 256, stream, a);
            if (st != TACO_OK) return st;
        }
        st = launch(a.dtotal ? reinterpret_cast<const void *>(&rms_backward_wide_kernel<T, true>)
                             : reinterpret_cast<const void *>(&rms_backward_wide_kernel<T, false>),
                    dim3(grid_rows(a.rows, 1, 512)), kWideThreads, stream, a);
    } else {
        a.segments = rms_segments(a.rows, a.hidden);
        const bool apart = a.partial && a.segments > 0;
        if (apart) a.row_groups = (int32_t)grid_rows(a.rows, rows_per_group(a.hidden), 2048);
        const bool whole = a.hidden % 8 == 0 && on16(a.dy, a.lddy, sizeof(T)) &&
                           on16(a.x, a.ldx, sizeof(T)) && on16(a.dx, a.lddx, sizeof(T)) &&
                           (!a.dtotal || on16(a.dtotal, a.lddt, sizeof(T)));
        st = for_backward_width(a.hidden, RmsBackwardLaunch<T>{a, stream, whole, apart});
        if (apart && a.segments == 1) return st;
    }
    if (st != TACO_OK || !a.partial) return st;
    return launch(reinterpret_cast<const void *>(&rms_parts_kernel<T>),
                  dim3((unsigned)((a.hidden + kWave - 1) / kWave)), kSumThreads, stream,
                  static_cast<const float *>(a.partial), (int)(a.segments > 0 ? a.segments : parts), a.hidden,
                  a.dweight, a.params_f32);
}

}  // namespace taco_norm
