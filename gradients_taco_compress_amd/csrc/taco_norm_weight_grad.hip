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
//  * Global loads go straight to LDS (16 bytes per lane, no registers) into a
//    ring of tiles; rows past the last are out of the loads' bounds and
//    arrive as zeros.  Fragments are read a few products ahead of their use,
//    and one barrier per tile serves both ends of the ring: the next tile has
//    arrived, and the one before the current has been read, by all waves.
//    Operands whose rows do not start on 16-byte boundaries are first copied
//    to where they do (measured at 8191 x 2555x2559: 145 us in all, of which the
//    copies take 25 us; loading such rows through registers instead took 220 us).
//  * db, the column sums of dY, comes from the same fragments (dot products
//    with ones), so dY is read by one kernel only.
//  * Tiles beyond a whole number per CU are split along t, evenly or into one
//    share for each CU, and their partial sums joined, in order, by a second
//    kernel.
//
// Measured, bf16, by card and run: 32768 x 1536x12288 958-1073 us (1150-1290
// TFLOP/s), 8192 x 10240x2560 386-420 us (1020-1110), 2048 x 1024x1024 20-21 us.
// Large products are bound by the matrix cores and the power they draw: 57 % of
// the cycles busy at a clock of 1.7 GHz.  Small ones are bound by the latency of
// a tile's loads: one work-group to a CU asks for a tile two steps before it
// needs it, and a step then takes 0.335 us, its products about 0.11 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <numeric>

#include "taco_norm.h"
#include "taco_norm_internal.hpp"
#include "taco_norm_device.hpp"

namespace taco_norm {
namespace {

typedef float f4v __attribute__((ext_vector_type(4)));
typedef int i2v __attribute__((ext_vector_type(2)));
typedef short s4v __attribute__((ext_vector_type(4)));

constexpr int kDepth = 32;             // t per tile: one matrix instruction's

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
    // c + a[0] + a[1]
    static __device__ __forceinline__ float add2(v2 a, float c) {
        return __builtin_amdgcn_fdot2_f32_bf16(a, (v2){1.0f, 1.0f}, c, false);
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
    static __device__ __forceinline__ float add2(v2 a, float c) {
        return __builtin_amdgcn_fdot2(a, (v2){1.0f, 1.0f}, c, false);
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

// Which output tile and which rows a work-group takes.  The first `whole`
// work-groups take a tile each.  The steps (kDepth rows) of the remaining
// tiles stand behind one another, `pitch` for each tile, and are cut every
// `share` steps; where a share goes over into the next tile, its two pieces are
// work-groups of their own.
struct Schedule {
    int32_t tiles_n, tiles_k;
    int32_t whole;
    int32_t uneven;            // pitch is not a multiple of share
    int64_t share, pitch;      // pitch >= share
    // Where the piece of share q in tile t (from the first split one) keeps
    // its sums.  Consecutive pieces have different q + t.
    __host__ __device__ __forceinline__ int64_t slab(int64_t t, int64_t q) const {
        return q + (uneven ? t : 0);
    }
};
// Of uneven pieces, the order in which they start, longest first: a CU that
// is done early takes a short one next.  An entry is the share, and in the top
// bit whether it is the share's second piece.  (Small tiles have no uneven
// plans: the longer arguments alone cost their short launches 0.4 us.)
template <bool LARGE>
struct Order {
    static constexpr int kMost = LARGE ? 512 : 1;
    uint16_t at[kMost];
};

struct Tile { int n, k; };

// f(Int<0>{}), ..., f(Int<N - 1>{}): loop bodies that need their index constant.
template <int I>
struct Int { static constexpr int value = I; };
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_each(F &&f) {
    if constexpr (I < N) {
        f(Int<I>{});
        for_each<N, I + 1>(f);
    }
}

// Tile number t of an order in which neighbours share operands: strips of
// four tile rows, each walked column by column.
__device__ __forceinline__ Tile tile_at(const Schedule &s, int t) {
    constexpr int kStrip = 4;
    const int strip = t / (kStrip * s.tiles_k), in = t - strip * kStrip * s.tiles_k;
    const int left = s.tiles_n - strip * kStrip, rows = left < kStrip ? left : kStrip;
    return {strip * kStrip + in % rows, in / rows};
}

// The finished gradient of four neighbours of a row: (w_k / S) sum + b_k db_n.
// Rows of dW, and the parameters, need no alignment beyond their elements': four
// neighbours are one load or store all the same (999 x 1030x1111: one by one,
// 25.4 us instead of 22.7).
template <typename E>
struct Finish {
    const WeightGrad &a;
    typedef E e4v __attribute__((ext_vector_type(4)));
    typedef E e4v_any __attribute__((ext_vector_type(4), aligned(sizeof(E))));
    typedef float f4v_any __attribute__((ext_vector_type(4), aligned(4)));
    __device__ __forceinline__ explicit Finish(const WeightGrad &args) : a(args) {}
    __device__ __forceinline__ f4v param4(const void *p, int k, float missing) const {
        if (!p) return (f4v){missing, missing, missing, missing};
        const float *const f = static_cast<const float *>(p);
        const E *const e = static_cast<const E *>(p);
        if (k + 4 <= a.hidden) {
            if (a.params_f32) return *reinterpret_cast<const f4v_any *>(f + k);
            return __builtin_convertvector((e4v)*reinterpret_cast<const e4v_any *>(e + k), f4v);
        }
        f4v v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = k + i < a.hidden ? k + i : a.hidden - 1;
            v[i] = a.params_f32 ? f[at] : (float)e[at];
        }
        return v;
    }
    __device__ __forceinline__ f4v scale(int k) const {
        return param4(a.weight, k, 1.0f) * a.inv_scale;
    }
    __device__ __forceinline__ f4v bias(int k) const { return param4(a.bias, k, 0.0f); }
    __device__ __forceinline__ void store(int n, int k, f4v sum, f4v sc, f4v b, float db) const {
        f4v v = sum * sc;
        if (a.bias) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(b[e], db, v[e]);
        }
        const int64_t at = (int64_t)n * a.hidden + k;
        if (k + 4 <= a.hidden) {
            if (a.dw_f32) {
                f4v_any *p = reinterpret_cast<f4v_any *>(static_cast<float *>(a.dw) + at);
                *p = a.accumulate ? *p + v : v;
            } else {
                *reinterpret_cast<e4v_any *>(static_cast<E *>(a.dw) + at) =
                    __builtin_convertvector(v, e4v);
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k + e >= a.hidden) break;
            if (a.dw_f32) {
                float *p = static_cast<float *>(a.dw) + at + e;
                *p = a.accumulate ? *p + v[e] : v[e];
            } else {
                static_cast<E *>(a.dw)[at + e] = (E)v[e];
            }
        }
    }
};

// Shape of a work-group's tile: BN x BK outputs by WN x WK waves, RING tiles
// of both operands in LDS.
template <int BN_, int BK_, int WN_, int WK_, int RING_>
struct Shape {
    static constexpr int BN = BN_, BK = BK_, WN = WN_, WK = WK_, RING = RING_;
    static_assert(RING % 2 == 0 && RING >= 4, "fragments alternate between two sets");
    static constexpr int THREADS = WN * WK * kWave;
    static constexpr int NI = BN / WN / 16, KI = BK / WK / 16;    // fragments of a wave
    // The waves that share columns of dY share their column sums: each adds up
    // its first NB fragments, which differ (Place::n).
    static constexpr int NB = NI / WK;
    static_assert((NI & (NI - 1)) == 0 && (KI & (KI - 1)) == 0 && (NB & (NB - 1)) == 0 && NB > 0,
                  "units of a wave");
    // A split's partial sums: every thread's, then the columns' sums.
    static constexpr int SLAB = BN * BK + BN;
};

// Lane (g, r) = (lane / 16, lane % 16) of wave (wn, wk) holds, in fragment
// (j, i), output row n = r and columns k = 4 g + (0..3) of that fragment.
template <typename S>
struct Place {
    int g, r, wn, wk;
    __device__ __forceinline__ explicit Place(int tid)
        : g((tid >> 4) & 3), r(tid & 15),
          wn(__builtin_amdgcn_readfirstlane(tid / kWave) % S::WN),
          wk(__builtin_amdgcn_readfirstlane(tid / kWave) / S::WN) {}
    __device__ __forceinline__ int n(int i) const {
        return (wn * S::NI + (i ^ (wk * S::NB))) * 16 + r;
    }
    __device__ __forceinline__ int k(int j) const { return (wk * S::KI + j) * 16 + 4 * g; }
};

template <typename E, typename S>
__global__ __launch_bounds__(S::THREADS) void grad_kernel(WeightGrad a, Schedule plan,
                                                          float *slabs, Order<S::BN == 256> order) {
    constexpr int BN = S::BN, BK = S::BK, NI = S::NI, KI = S::KI, THREADS = S::THREADS;
    constexpr int DY_BYTES = kDepth * BN * 2, CODE_BYTES = kDepth * BK;
    constexpr int DY_LOADS = DY_BYTES / 16 / THREADS, CODE_LOADS = CODE_BYTES / 16 / THREADS;
    constexpr int LOADS = DY_LOADS + CODE_LOADS;
    constexpr int DY_CHUNKS = BN / 8, CODE_CHUNKS = BK / 16;      // 16-byte chunks of a row
    using M = Mfma<E>;
    // A variable for each tile of the ring, not one for all: the compiler then
    // knows that a load into one does not touch the fragments being read from
    // another, and does not wait for it.
    constexpr int TILE = DY_BYTES + CODE_BYTES, RING = S::RING;
    __shared__ __align__(1024) uint8_t lds0[TILE], lds1[TILE], lds2[TILE], lds3[TILE],
        lds4[RING > 4 ? TILE : 1], lds5[RING > 5 ? TILE : 1];
    auto ring = [&](auto index) -> uint8_t * {
        constexpr int i = decltype(index)::value % RING;
        if constexpr (i == 0) return lds0;
        else if constexpr (i == 1) return lds1;
        else if constexpr (i == 2) return lds2;
        else if constexpr (i == 3) return lds3;
        else if constexpr (i == 4) return lds4;
        else return lds5;
    };

    const int tid = threadIdx.x;
    [[maybe_unused]] const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const Place<S> place(tid);

    // Consecutive work-groups go to the 8 XCDs in turn; each XCD gets a
    // contiguous range of the whole tiles, whose operands meet in its L2.
    int t_index, part = -1;
    int64_t t0 = 0, t1 = a.rows;
    if ((int)blockIdx.x < plan.whole) {
        const int xcd = blockIdx.x % 8, q = plan.whole / 8, rem = plan.whole % 8;
        t_index = xcd * q + (xcd < rem ? xcd : rem) + blockIdx.x / 8;
    } else {
        int64_t q = blockIdx.x - plan.whole;
        int second = 0;
        if (BN == 256 && plan.uneven) {
            const int piece = order.at[q];
            second = piece >> 15;
            q = piece & 0x7FFF;
        }
        const int64_t begin = q * plan.share, t = begin / plan.pitch + second;
        const int64_t from = t * plan.pitch, end = begin + plan.share;
        t0 = (begin > from ? begin - from : 0) * kDepth;
        t1 = (end < from + plan.pitch ? end - from : plan.pitch) * kDepth;
        if (t1 > a.rows) t1 = a.rows;
        part = (int)plan.slab(t, q);
        t_index = plan.whole + (int)t;
    }
    const Tile tile = tile_at(plan, t_index);
    const int n0 = tile.n * BN, k0 = tile.k * BK;
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

    // Loads go straight to LDS: rows past t1 are out of the resource's bounds, which
    // makes them zero; a chunk past the last column reads the tile's first one
    // instead (its sums are never stored).  A tile's offsets from its first
    // element fit 31 bits (the launcher sees to it).  (What only the loads use is
    // unused in the host pass.)
    static_assert(DY_LOADS == 2 && CODE_LOADS == 1, "loads of a tile");
    [[maybe_unused]] uint32_t dy_off[2], code_off;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = dy_col(i);
        dy_off[i] = (uint32_t)(dy_row(i) * (int)a.lddy + (n0 + col < a.out_features ? col : 0)) * 2u;
    }
    code_off = (uint32_t)(code_row(0) * (int)a.ldcodes + (k0 + code_col(0) < a.hidden ? code_col(0) : 0));
    // The next tile to load: its first elements, and how many tiles remain, the
    // last of them with fewer rows.
    [[maybe_unused]] const char *next_dy = dy + (t0 * a.lddy + n0) * 2;
    [[maybe_unused]] const char *next_codes = codes + t0 * a.ldcodes + k0;
    // (readfirstlane: these are the same for all lanes, and have to be kept so)
    const int steps = __builtin_amdgcn_readfirstlane((int)((t1 - t0 + kDepth - 1) / kDepth));
    [[maybe_unused]] int tiles_left = steps;
    [[maybe_unused]] const int last_rows =
        __builtin_amdgcn_readfirstlane((int)(t1 - t0 - (int64_t)(steps - 1) * kDepth));
    [[maybe_unused]] const int dy_pitch = (int)a.lddy * 2;
    auto load_tile = [&](uint8_t *buf) {
#if defined(__HIP_DEVICE_COMPILE__)      // the host pass does not know the resource type
        // Rows of this tile (none past the last tile).  Every column read exists,
        // so the bounds need to be right for whole rows only.
        const int two = tiles_left < 2 ? tiles_left : 2, sum_rows = (two - 1) * kDepth + last_rows;
        const int rows = __builtin_amdgcn_readfirstlane(
            sum_rows < 0 ? 0 : sum_rows < kDepth ? sum_rows : kDepth);
        // 0x00020000: raw 32-bit data.
        const auto rd = __builtin_amdgcn_make_buffer_rsrc((void *)next_dy, 0, rows * dy_pitch, 0x00020000);
        const auto rc = __builtin_amdgcn_make_buffer_rsrc((void *)next_codes, 0, rows * (int)a.ldcodes, 0x00020000);
#pragma unroll
        for (int i = 0; i < DY_LOADS; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rd,
                (__attribute__((address_space(3))) void *)(buf + (i * THREADS + wave * kWave) * 16),
                16, dy_off[i], 0, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rc,
            (__attribute__((address_space(3))) void *)(buf + DY_BYTES + wave * kWave * 16), 16,
            code_off, 0, 0, 0);
        next_dy += (int64_t)kDepth * dy_pitch;
        next_codes += (int64_t)kDepth * a.ldcodes;
        --tiles_left;
#endif
    };
    // Fragment addresses: lane (g, r) reads 8 bytes of row 8 g + r / 4 (dY;
    // then + 4) or 8 g + r / 2 (codes); the read hands it column r of them.
    // A wave's units differ in their low bits only, so fragment i's unit is
    // the first one's XOR i.
    int dy_at, code_at;
    {
        const int t = 8 * place.g + (place.r >> 2);
        dy_at = t * BN * 2 + (((place.wn * NI + place.wk * S::NB) ^ turn_dy<BN>(t)) * 32) + (place.r & 3) * 8;
    }
    {
        const int t = 8 * place.g + (place.r >> 1);
        code_at = DY_BYTES + t * BK + (((place.wk * KI) ^ turn_codes<BK>(t)) * 16) +
                  (place.r & 1) * 8;
    }

    // (The addresses are opaque at each use, so that they are formed again for
    // each tile: kept, those of the whole ring would not fit the registers.)
    auto read_dy = [&](uint8_t *buf, int i) {
        uint8_t *p = buf + (dy_at ^ (i * 32));
        union { s4v s[2]; typename M::v8 v; } u;
        u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v *)p);
        u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4v *)(p + 4 * BN * 2));
        return u.v;
    };
    auto read_codes = [&](uint8_t *buf, int j) {
        return __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i2v *)(buf + (code_at ^ (j * 16))));
    };
    auto convert = [&](i2v c) {
        union { typename M::v2 h[4]; typename M::v8 v; } u;
        u.h[0] = M::template codes<false>((uint32_t)c[0]);
        u.h[1] = M::template codes<true>((uint32_t)c[0]);
        u.h[2] = M::template codes<false>((uint32_t)c[1]);
        u.h[3] = M::template codes<true>((uint32_t)c[1]);
        return u.v;
    };

    constexpr int NB = S::NB;
    f4v sum[KI][NI];
    float db[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) db[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int j = 0; j < KI; ++j) sum[j][i] = (f4v){0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto add_columns = [&](const typename M::v8 &v, int i, int e) {
        union { typename M::v8 v; typename M::v2 h[4]; } u;
        u.v = v;
        db[i] = M::add2(u.h[e], db[i]);
    };

    // Two sets of dY fragments (this tile's and the next's), a queue of code
    // fragments read three products ahead, and two converted ones.
    typename M::v8 fd[2][NI], fc[2];
    i2v queue[4];
    for_each<RING - 1>([&](auto i) { load_tile(ring(i)); });
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((RING - 2) * LOADS) : "memory");
#pragma unroll
    for (int i = 0; i < NI; ++i) fd[0][i] = read_dy(lds0, i);
#pragma unroll
    for (int j = 0; j < 3; ++j) queue[j] = read_codes(lds0, j);
    fc[0] = convert(queue[0]);
    auto step = [&](auto index) {
        constexpr int s = decltype(index)::value;
        uint8_t *const cur = ring(Int<s>{}), *const next = ring(Int<s + 1>{});
        constexpr int kTurn = KI / 2 - 1;        // the block with the barrier
        constexpr int kReads = NI / (KI / 2);    // dY fragments read in each of those after
        for_each<KI>([&](auto block) {
            constexpr int j = decltype(block)::value;
            if constexpr (j == kTurn) {
                // The next tile has arrived (those after it may be on their way)
                // and the previous one has been read; after the barrier, for all.
                asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((RING - 3) * LOADS)
                             : "memory");
                load_tile(ring(Int<s + RING - 1>{}));
            }
            asm volatile("" : "+v"(dy_at), "+v"(code_at));
            constexpr int ahead = j + 3;
            queue[ahead & 3] = ahead < KI ? read_codes(cur, ahead) : read_codes(next, ahead - KI);
            if constexpr (j >= kTurn && j < kTurn + KI / 2) {
#pragma unroll
                for (int i = 0; i < kReads; ++i)
                    fd[(s + 1) & 1][(j - kTurn) * kReads + i] =
                        read_dy(next, (j - kTurn) * kReads + i);
            }
            __builtin_amdgcn_sched_barrier(0);
            fc[(j + 1) & 1] = convert(queue[(j + 1) & 3]);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                sum[j][i] = M::run(fc[j & 1], fd[s & 1][i], sum[j][i]);
#pragma unroll
            for (int e = j * 4 * NB / KI; e < (j + 1) * 4 * NB / KI; ++e)
                add_columns(fd[s & 1][e / 4], e / 4, e & 3);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // MFMA
                __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);      // VALU
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // A whole ring at a time, so that every LDS address is a constant; the
    // tiles past the last row are zero.
    for (int s = 0; s < steps; s += RING) for_each<RING>(step);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // Column sums: a lane holds those of its rows' group g.
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        db[i] += __shfl_xor(db[i], 16);
        db[i] += __shfl_xor(db[i], 32);
    }
    if (part >= 0) {
        float *const slab = slabs + (int64_t)part * S::SLAB;
#pragma unroll
        for (int j = 0; j < KI; ++j)
#pragma unroll
            for (int i = 0; i < NI; ++i)
                *reinterpret_cast<f4v *>(slab + ((j * NI + i) * THREADS + tid) * 4) = sum[j][i];
        if (place.g == 0) {
#pragma unroll
            for (int i = 0; i < NB; ++i) slab[BN * BK + place.n(i)] = db[i];
        }
        return;
    }
    // Every wave needs those of all its columns.
    float *const shared_db = reinterpret_cast<float *>(lds0);
    __syncthreads();
    if (place.g == 0) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            shared_db[place.n(i)] = db[i];
            if (a.dbias && tile.k == 0 && n0 + place.n(i) < a.out_features)
                a.dbias[n0 + place.n(i)] = db[i];
        }
    }
    __syncthreads();
    const Finish<E> finish(a);
#pragma unroll
    for (int j = 0; j < KI; ++j) {
        const int k = k0 + place.k(j);
        if (k >= a.hidden) continue;
        const f4v sc = finish.scale(k), b = finish.bias(k);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int n = n0 + place.n(i);
            if (n < a.out_features) finish.store(n, k, sum[j][i], sc, b, shared_db[place.n(i)]);
        }
    }
}

// Adds the parts of a split tile in order and finishes it: blockIdx.x is the
// tile after the whole ones, blockIdx.y its fragment.
template <typename E, typename S>
__global__ __launch_bounds__(S::THREADS) void join_kernel(WeightGrad a, Schedule plan,
                                                          const float *slabs) {
    const int j = blockIdx.y / S::NI, i = blockIdx.y % S::NI;
    const Place<S> place(threadIdx.x);
    const Tile tile = tile_at(plan, plan.whole + blockIdx.x);
    const int n = tile.n * S::BN + place.n(i), k = tile.k * S::BK + place.k(j);
    if (n >= a.out_features || k >= a.hidden) return;
    // The tile's pieces: the shares from the one that its first step is in to
    // the one that its last is in.
    const int64_t from = blockIdx.x * plan.pitch;
    const int64_t first = from / plan.share, last = (from + plan.pitch - 1) / plan.share;
    const float *p = slabs + plan.slab(blockIdx.x, first) * S::SLAB;
    f4v sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float db = 0.0f;
    for (int64_t q = first; q <= last; ++q, p += S::SLAB) {
        sum += *reinterpret_cast<const f4v *>(p + (blockIdx.y * S::THREADS + threadIdx.x) * 4);
        db += p[S::BN * S::BK + place.n(i)];
    }
    const Finish<E> finish(a);
    finish.store(n, k, sum, finish.scale(k), finish.bias(k), db);
    if (a.dbias && tile.k == 0 && j == 0 && place.wk == 0 && place.g == 0) a.dbias[n] = db;
}

// Rows of `width` bytes, `from_pitch` apart at any address, to rows `to_pitch`
// apart that start on 16-byte boundaries (bytes past the width: zero).
struct Repack {
    const char *from;
    char *to;
    int64_t from_pitch, to_pitch;
    int32_t width;
    int32_t lanes_log2;            // threads to a row
};
__global__ __launch_bounds__(256) void repack_kernel(Repack one, Repack two, int64_t rows) {
    const Repack r = blockIdx.y ? two : one;
    if (!r.from) return;
    const int lanes = 1 << r.lanes_log2, lane = threadIdx.x & (lanes - 1);
    const int per = 256 >> r.lanes_log2;
    for (int64_t row = (int64_t)blockIdx.x * per + (threadIdx.x >> r.lanes_log2); row < rows;
         row += (int64_t)gridDim.x * per) {
        const char *from = r.from + row * r.from_pitch;
        char *to = r.to + row * r.to_pitch;
        for (int at = lane * 16; at < r.to_pitch; at += lanes * 16) {
            const int n = r.width - at;
            *reinterpret_cast<u4v *>(to + at) = load_tail<true>(from + at, from, n < 16 ? n : 16);
        }
    }
}

// ---------------------------------------------------------------- host ----

using Large = Shape<256, 256, 4, 2, 6>;
using Small = Shape<128, 128, 2, 2, 4>;

struct Plan {
    bool large;
    Schedule schedule;
    int64_t split_tiles, pieces, slabs;
};

int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

// What a plan's parts cost in microseconds, as measured on an MI355X: a
// work-group's beginning and end, a step (kDepth rows) of a tile while every
// place of the GPU has one and where there are no more work-groups than CUs,
// and a part's sums, written, read and joined.
struct Cost {
    int places;            // work-groups that run at once
    double fixed, step, alone, part;
};
// A large tile's ring fills a CU's LDS (8192 x 8192x8192: 1024 tiles of 256
// steps in 875 us; 16384 x 3584x3584: 196 tiles of 512 in 390 us).  Two small ones
// keep a CU busy (2048 x 2560x2560: 400 tiles of 64 steps in 39 us; one to a CU,
// 8192 x 512x512: 16 tiles of 256 steps in 91 us).
constexpr Cost kLargeCost = {256, 8.0, 0.82, 0.74, 0.11};
constexpr Cost kSmallCost = {512, 5.5, 0.56, 0.335, 0.01};
// The second launch, and each part that a thread of it adds up.
constexpr double kJoinUs = 5.0, kJoinPartUs = 0.3;

template <typename S>
double groups_us(const Cost &c, int64_t groups, int64_t steps) {
    steps = up(steps, S::RING) * S::RING;
    const int64_t left = groups % c.places;
    return (double)(groups / c.places) * (c.fixed + (double)steps * c.step) +
           (left == 0 ? 0.0 : c.fixed + (double)steps * (left <= 256 ? c.alone : c.step));
}

// The tiles left over after a whole number for each place are split along the
// rows: each into the same number of parts, or all of them into one share for
// each place, whichever takes least time.  Shares against the best equal parts:
// 8192 x 5120x5120 (144 tiles left) 415 against 431 us, 16384 x 4096x1536 (96
// tiles) 212 against 228 us, 20000 x 1700x5000 (140) 445 against 462 us; at 196
// tiles they gain nothing over leaving 60 CUs idle (417 against 400 us), whose
// power the other CUs turn into clock: Cost::alone.
template <typename S>
Plan plan_for(int64_t rows, int64_t n, int64_t k, const Cost &cost, double *us) {
    Plan p = {};
    p.large = S::BN == 256;
    const int64_t tn = up(n, S::BN), tk = up(k, S::BK), tiles = tn * tk;
    const int64_t steps = up(rows, kDepth), left = tiles % cost.places;
    double best = groups_us<S>(cost, tiles, steps);
    Schedule &s = p.schedule;
    s.tiles_n = (int32_t)tn;
    s.tiles_k = (int32_t)tk;
    auto take = [&](double parts_us, int64_t parts, int64_t share, int64_t pitch, int64_t slabs) {
        const double t = groups_us<S>(cost, tiles - left, steps) + parts_us +
                         (double)parts * cost.part + kJoinUs +
                         (double)up(steps, share) * kJoinPartUs;
        if (t >= best) return;
        best = t;
        s.share = share;
        s.pitch = pitch;
        s.uneven = pitch % share != 0;
        p.split_tiles = left;
        p.pieces = parts;
        p.slabs = slabs;
    };
    for (int64_t split : {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128}) {
        if (left == 0 || split * 4 > steps) break;
        const int64_t share = up(steps, split), parts = up(steps, share);
        take(groups_us<S>(cost, left * parts, share), left * parts, share, parts * share,
             left * parts);
    }
    const int64_t share = up(left * steps, cost.places);
    if (p.large && share >= 4 && share < steps && steps % share != 0) {
        // A tile's end inside a share makes two pieces of it.
        const int64_t shares = up(left * steps, share);
        const int64_t cuts = left - 1 - (left - 1) / (share / std::gcd(share, steps));
        take(2 * cost.fixed + (double)(share + S::RING) * cost.step, shares + cuts, share, steps,
             shares + left);
    }
    s.whole = (int32_t)(tiles - p.split_tiles);
    *us = best;
    return p;
}

// The pieces of an uneven plan, about longest first (by sixty-fourths of a share).
Order<true> order_of(const Plan &p) {
    Order<true> order;
    const Schedule &s = p.schedule;
    const int64_t total = p.split_tiles * s.pitch;
    int32_t at[65] = {};
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t q = 0; q * s.share < total; ++q) {
            const int64_t begin = q * s.share;
            const int64_t end = begin + s.share < total ? begin + s.share : total;
            const int64_t cut = (begin / s.pitch + 1) * s.pitch;
            const int64_t length[2] = {(cut < end ? cut : end) - begin, cut < end ? end - cut : 0};
            for (int second = 0; second < 2; ++second) {
                if (length[second] == 0) continue;
                int32_t &place = at[64 - length[second] * 64 / s.share];
                if (pass == 0) ++place;
                else order.at[place++] = (uint16_t)(q | second << 15);
            }
        }
        if (pass == 0)
            for (int32_t i = 0, sum = 0; i < 65; ++i) {
                const int32_t count = at[i];
                at[i] = sum;
                sum += count;
            }
    }
    return order;
}

Plan plan(int64_t rows, int64_t n, int64_t k) {
    double large_us, small_us;
    const Plan large = plan_for<Large>(rows, n, k, kLargeCost, &large_us);
    const Plan small = plan_for<Small>(rows, n, k, kSmallCost, &small_us);
    return large_us <= small_us ? large : small;
}

// Bytes of the parts' sums, and of the operands' copies (0 where the operand
// can be read as it is), each a multiple of 16.
struct Workspace {
    int64_t slabs, dy, codes;
    int64_t dy_pitch, code_pitch;          // bytes between the copies' rows
};
Workspace workspace(const Plan &p, const WeightGrad &a) {
    Workspace w = {};
    w.slabs = p.slabs * (int64_t)(p.large ? Large::SLAB : Small::SLAB) * (int64_t)sizeof(float);
    // 16-byte loads of whole chunks of a row, 31-bit offsets inside a tile.
    const bool dy_direct =
        ((reinterpret_cast<uintptr_t>(a.dy) | (uintptr_t)(a.lddy * 2)) & 15u) == 0 &&
        a.out_features % 8 == 0 && a.lddy < (INT64_C(1) << 24);
    const bool codes_direct = ((reinterpret_cast<uintptr_t>(a.codes) | (uintptr_t)a.hidden) & 15u) == 0;
    if (!dy_direct) {
        w.dy_pitch = up((int64_t)a.out_features * 2, 16) * 16;
        w.dy = a.rows * w.dy_pitch;
    }
    if (!codes_direct) {
        w.code_pitch = up(a.hidden, 16) * 16;
        w.codes = a.rows * w.code_pitch;
    }
    return w;
}

template <typename E, typename S>
taco_status launch_grad(const WeightGrad &a, const Plan &p, hipStream_t stream) {
    static_assert(2 * kLargeCost.places <= Order<true>::kMost, "two pieces of every share");
    const int64_t groups = p.schedule.whole + p.pieces;
    Order<S::BN == 256> order = {};
    if constexpr (S::BN == 256)
        if (p.schedule.uneven) order = order_of(p);
    const taco_status st = launch(reinterpret_cast<const void *>(&grad_kernel<E, S>),
                                  dim3((unsigned)groups), S::THREADS, stream, a, p.schedule,
                                  a.workspace, order);
    if (st != TACO_OK || p.split_tiles == 0) return st;
    return launch(reinterpret_cast<const void *>(&join_kernel<E, S>),
                  dim3((unsigned)p.split_tiles, S::NI * S::KI), S::THREADS, stream, a, p.schedule,
                  static_cast<const float *>(a.workspace));
}

template <typename E>
taco_status run(WeightGrad a, hipStream_t stream) {
    const Plan p = plan(a.rows, a.out_features, a.hidden);
    const Workspace w = workspace(p, a);
    a.ldcodes = a.hidden;
    if (w.dy || w.codes) {
        char *const copies = reinterpret_cast<char *>(a.workspace) + w.slabs;
        auto repack = [&](const void *from, int64_t from_pitch, char *to, int64_t to_pitch,
                          int32_t width) {
            int32_t log2 = 0;
            while (log2 < 8 && (INT64_C(16) << log2) < to_pitch) ++log2;
            return Repack{static_cast<const char *>(from), to, from_pitch, to_pitch, width, log2};
        };
        Repack dy = {}, codes = {};
        if (w.dy) {
            dy = repack(a.dy, a.lddy * 2, copies, w.dy_pitch, a.out_features * 2);
            a.dy = dy.to;
            a.lddy = w.dy_pitch / 2;
        }
        if (w.codes) {
            codes = repack(a.codes, a.hidden, copies + w.dy, w.code_pitch, a.hidden);
            a.codes = reinterpret_cast<const uint8_t *>(codes.to);
            a.ldcodes = w.code_pitch;
        }
        const int64_t groups = up((w.dy > w.codes ? w.dy : w.codes) / 16, 256);
        const taco_status st = launch(reinterpret_cast<const void *>(&repack_kernel),
                                      dim3((unsigned)(groups < 2048 ? groups : 2048), 2), 256, stream,
                                      dy, codes, a.rows);
        if (st != TACO_OK) return st;
    }
    return p.large ? launch_grad<E, Large>(a, p, stream) : launch_grad<E, Small>(a, p, stream);
}

}  // namespace

int64_t weight_grad_workspace(const WeightGrad &a) {
    const Workspace w = workspace(plan(a.rows, a.out_features, a.hidden), a);
    return w.slabs + w.dy + w.codes;
}

taco_status weight_grad(const WeightGrad &a, taco_norm_dtype dtype, hipStream_t stream) {
    return dtype == TACO_NORM_BF16 ? run<__bf16>(a, stream) : run<_Float16>(a, stream);
}

}  // namespace taco_norm
