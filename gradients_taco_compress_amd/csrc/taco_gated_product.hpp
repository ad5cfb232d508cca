// The three matrix products of the gated feed-forward block (formulas in
// taco_gated.h) for gfx950, templated on the operands' type and on the kind of
// product.
//
//  * A work-group makes BM x BN outputs from K-tiles of 128 bytes of summed length
//    (64 elements, or 128 codes).  Both operands of a K-tile are kept in LDS as two
//    halves each (A0, A1, B0, B1), two K-tiles at a time (four where tiles are few),
//    and a K-tile is worked off in four phases, the quadrants (A0, F), (A0, S),
//    (A1, S), (A1, F) of the output.  F and S are
//    B0 and B1, the other way round in every second K-tile: so the half of B
//    that is done with first is the one that is needed first next.
//  * The forward pass takes gate features as B0 and the same up features as
//    B1, so that G and U of an element meet in one lane and A is formed from
//    the float32 sums: G and U are not written unless training asks for them.
//  * Registers hold one half of A and both of B.  Where a half of A is used for
//    the last time, each of its fragments is replaced as its products have
//    been issued, so the LDS reads run beside the products without a second set
//    of registers.
//  * Each phase loads one half of a later K-tile straight to LDS (16 bytes a
//    lane, no registers); three to five halves are on their way at any time.  Two
//    barriers a K-tile serve all of it: after (A0, F), A1 has arrived and A0 and F have
//    been read, by all waves; after (A1, S), the next A0, F and S have arrived
//    and this S and A1 have been read.
//  * Operands whose summed index is contiguous (X and the weights, forward)
//    lie in LDS as rows of 128 bytes, 16-byte chunk c of row R at chunk
//    c ^ f(R); those whose summed index is the slow one lie as they do in memory
//    and are turned by the transposing LDS reads, 32-byte units of row t at
//    unit u ^ turn(t).  f and turn put what is read together on different banks.
//  * Rows and columns outside the matrices are out of the loads' bounds and
//    arrive as zeros, so ragged edges cost no instructions in the products.
//  * Tiles beyond a whole number per CU are split along the summed index, and
//    a second kernel adds the parts in order and finishes them.
//  * Codes go through the scaled matrix instruction (16x16x128).  Its scale
//    operand of lane (g, r) is the one of 32-block g of row r, while the lane's
//    data are the 16-byte chunks g and 4 + g of the row: the same reads as for
//    16-bit elements.  Of each eight neighbouring codes it adds the products with 12
//    bits below the largest one's exponent (measured), which is about 1e-4 of a
//    result.
//
// Bound by the matrix cores, busy 63 to 70 % of the cycles, and by power, at 1.85 to 1.9
// GHz.  8192 x 10240x2560 bf16: forward with G and U 660 to 685 us (1255 to 1300 TFLOP/s),
// dX 605 us and the weights' gradients 652 us (1420 and 1320).  Codes 16384 x
// 14336x3584: 1240 to 1300 us (2590 to 2720 TFLOP/s).  No bank conflicts, no scratch.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "taco_gated_internal.hpp"
#include "taco_gated_device.hpp"

namespace taco_gated {
namespace {

typedef int i8v __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));

constexpr int kDeep = 128;          // bytes of summed length in a K-tile

// A fragment: 16 rows (or columns) of a K-tile.  Lane (g, r) holds of row r the
// elements 8 g .. 8 g + 7 of each half of the K-tile (codes: 16 g ..).
struct Fragment {
    u4v v[2];
};

template <typename E>
struct Element;
template <>
struct Element<BF16> {
    typedef __bf16 type;
    static constexpr int SIZE = 2;
    static constexpr bool SCALED = false;
    template <int, int>
    static __device__ __forceinline__ f4v run(const Fragment &a, const Fragment &b, f4v c, int, int) {
        typedef __bf16 v8 __attribute__((ext_vector_type(8)));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a.v[i]),
                                                        __builtin_bit_cast(v8, b.v[i]), c, 0, 0, 0);
        return c;
    }
};
template <>
struct Element<F16> {
    typedef _Float16 type;
    static constexpr int SIZE = 2;
    static constexpr bool SCALED = false;
    template <int, int>
    static __device__ __forceinline__ f4v run(const Fragment &a, const Fragment &b, f4v c, int, int) {
        typedef _Float16 v8 __attribute__((ext_vector_type(8)));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a.v[i]),
                                                       __builtin_bit_cast(v8, b.v[i]), c, 0, 0, 0);
        return c;
    }
};
template <>
struct Element<Codes> {
    typedef uint8_t type;
    static constexpr int SIZE = 1;
    static constexpr bool SCALED = true;
    // BA, BB: which byte of the registers holds the scale.
    template <int BA, int BB>
    static __device__ __forceinline__ f4v run(const Fragment &a, const Fragment &b, f4v c, int sa,
                                              int sb) {
        // 0, 0: both operands E4M3.
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            __builtin_bit_cast(i8v, a), __builtin_bit_cast(i8v, b), c, 0, 0, BA, sa, BB, sb);
    }
};

// Shape of a work-group: BM x BN outputs by WM x WN waves.  (Forward: BN / 2
// features.)
template <int BM_, int BN_, int WM_, int WN_, int RING_>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int RING = RING_;                                 // K-tiles in LDS
    static_assert(RING == 2 || RING == 4, "F and S change places with every K-tile");
    static constexpr int THREADS = WM * WN * kWave;
    static constexpr int HM = BM / 2, HN = BN / 2;                     // a half's rows
    static constexpr int MF = HM / WM / 16, NF = HN / WN / 16;         // a wave's fragments of it
    static constexpr int A_HALF = HM * kDeep, B_HALF = HN * kDeep;     // its bytes
    static_assert(HM == HN, "halves alike: one load count for all");
    static constexpr int LOADS = A_HALF / 16 / THREADS;                // a thread's loads of it
    static_assert(LOADS == 2 && NF == 2, "loads and pairs of column fragments");
    // Register sets for the halves of A: large tiles have none to spare, the others
    // read a half in one go (1 to 2 % less time).
    static constexpr int SETS = BM == 256 ? 1 : 2;
    // A split's partial sums.
    static constexpr int64_t SLAB = (int64_t)BM * BN;
};
using Large = Shape<256, 256, 2, 4, 2>;
using Small = Shape<128, 128, 2, 2, 2>;
// One to a CU, for few tiles: its loads are asked for three K-tiles ahead.
using Deep = Shape<128, 128, 2, 2, 4>;

// The items of work, one to a work-group: the first `whole` are a tile each; the
// remaining tiles are cut into `parts` parts of `share` K-tiles.  (Work-groups that
// stay and walk over items, the next one's loads going out before the current
// one's outputs are formed, took as long forward and 5 % longer backward, 8192 x
// 10240x2560 1577 instead of 1507 us: items handed out one by one even out what CUs
// take.)
struct Plan {
    int32_t tiles_m, tiles_n;
    int32_t whole, parts, share;
    int32_t depth;                 // K-tiles of a tile
    int32_t items;
};

struct Tile { int m, n; };

// Tile number t of an order in which neighbours share operands: strips of
// four tile rows, each walked column by column.
__device__ __forceinline__ Tile tile_at(const Plan &s, int t) {
    constexpr int kStrip = 4;
    const int strip = t / (kStrip * s.tiles_n), in = t - strip * kStrip * s.tiles_n;
    const int left = s.tiles_m - strip * kStrip, rows = left < kStrip ? left : kStrip;
    return {strip * kStrip + in % rows, in / rows};
}

__device__ __forceinline__ int clamp(int64_t v, int most) {
    return v < 0 ? 0 : v < most ? (int)v : most;
}

// Lane (g, r) = (lane / 16, lane % 16) of wave (wm, wn) holds, in fragments
// (i, j) of a quadrant, row m = r and columns 4 g + (0..3).
template <typename S>
struct Place {
    int g, r, wm, wn;
    __device__ __forceinline__ explicit Place(int tid)
        : g((tid >> 4) & 3), r(tid & 15),
          wm(__builtin_amdgcn_readfirstlane(tid / kWave) % S::WM),
          wn(__builtin_amdgcn_readfirstlane(tid / kWave) / S::WM) {}
};

// Writes one row fragment of a tile's outputs: v[qb][j], quadrant column qb and
// column fragment j.
template <typename E, Kind K, typename S>
struct Finish {
    const Product &p;
    const Place<S> &place;
    Tile tile;

    template <typename T>
    __device__ __forceinline__ void forward(int64_t m, const f4v (&v)[2][2]) const {
        const int64_t f = (int64_t)tile.n * S::HN + place.wn * 32 + 8 * place.g;
        const int64_t left = p.n - f;
        if (left <= 0) return;
        float gate[8], up[8], out[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            gate[e] = v[0][e >> 2][e & 3];
            up[e] = v[1][e >> 2][e & 3];
        }
        with_activation(p.activation, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                out[e] = gate[e] * gate_share<decltype(act)::value>(gate[e]) * up[e];
        });
        store_row<T, 8>(static_cast<T *>(p.out[0]) + m * p.out_pitch[0] + f, out, left);
        if (p.out[1]) {
            store_row<T, 8>(static_cast<T *>(p.out[1]) + m * p.out_pitch[1] + f, gate, left);
            store_row<T, 8>(static_cast<T *>(p.out[2]) + m * p.out_pitch[2] + f, up, left);
        }
    }

    __device__ __forceinline__ void operator()(int qa, int i, const f4v (&v)[2][2]) const {
        int tm = tile.m, which = 0;
        if constexpr (K == Kind::kWeight) {
            // The tiles of dWg, then those of dWu.
            const int per = (int)((p.m + S::BM - 1) / S::BM);
            which = tm >= per;
            tm -= which * per;
        }
        const int64_t m = (int64_t)tm * S::BM + qa * S::HM + place.wm * (S::HM / S::WM) + 16 * i + place.r;
        if (m >= p.m) return;
        if constexpr (K == Kind::kForward) {
            if constexpr (Element<E>::SCALED) {
                if (p.out_f16) forward<_Float16>(m, v);
                else forward<__bf16>(m, v);
            } else {
                forward<typename Element<E>::type>(m, v);
            }
        } else {
            using T = typename Element<E>::type;
            T *const row = static_cast<T *>(p.out[which]) + m * p.out_pitch[which];
#pragma unroll
            for (int qb = 0; qb < 2; ++qb)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int64_t n = (int64_t)tile.n * S::BN + qb * S::HN + place.wn * 32 + 16 * j + 4 * place.g;
                    if (n >= p.n) continue;
                    const float out[4] = {v[qb][j][0], v[qb][j][1], v[qb][j][2], v[qb][j][3]};
                    store_row<T, 4>(row + n, out, p.n - n);
                }
        }
    }
};

// A work-group's LDS.  Several variables, not one for all: the compiler then knows
// that a load into one does not touch the fragments being read from another, and
// does not wait for it.  It tells few of them apart, so what is never loaded and
// read at the same time shares one: the halves of B and the scales, and in a ring
// of four K-tiles (whose loads into a variable follow the reads from it) all of a
// K-tile.
template <typename E, typename S>
struct Lds {
    static constexpr bool APART = S::RING == 2;                // halves of A have their own
    static constexpr int SCALES = Element<E>::SCALED ? S::THREADS * 4 : 0;     // [A0 | A1 | B0 | B1]
    static constexpr int B_AT = APART ? 0 : 2 * S::A_HALF, S_AT = B_AT + 2 * S::B_HALF;
    static constexpr int HALF = APART ? S::A_HALF : 1, REST = S_AT + SCALES;
    static constexpr int MORE = APART ? 1 : REST;
    uint8_t *a[4], *rest[4];
};

// Item j of a product.
template <typename E, Kind K, typename S>
__device__ __forceinline__ void multiply_item(const Product &p, const Plan &plan, int j,
                                              const Lds<E, S> &mem) {
    using El = Element<E>;
    constexpr int HM = S::HM, HN = S::HN, MF = S::MF, NF = S::NF, THREADS = S::THREADS;
    constexpr int SIZE = El::SIZE, KT = kDeep / SIZE;          // summed elements of a K-tile
    constexpr bool A_TURNED = K == Kind::kWeight, B_TURNED = K != Kind::kForward;
    constexpr bool SCALED = El::SCALED, APART = Lds<E, S>::APART;
    constexpr int B_AT = Lds<E, S>::B_AT, S_AT = Lds<E, S>::S_AT;
    auto lds = [&](auto stage) -> uint8_t * { return mem.rest[decltype(stage)::value % S::RING]; };
    auto lds_a = [&](auto stage, auto half) -> uint8_t * {
        constexpr int s = decltype(stage)::value % S::RING, h = decltype(half)::value;
        if constexpr (!APART) return lds(stage) + h * S::A_HALF;
        else return mem.a[2 * s + h];
    };
    auto lds_b = [&](auto stage, auto half) -> uint8_t * {
        return lds(stage) + B_AT + decltype(half)::value * S::B_HALF;
    };
    [[maybe_unused]] auto lds_s = [&](auto stage) -> uint8_t * { return lds(stage) + S_AT; };   // scales

    const int tid = threadIdx.x;
    [[maybe_unused]] const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const Place<S> place(tid);

    // Chunk i of this thread is LDS chunk i * THREADS + tid of a half: its row
    // there, the chunk of the source row it comes from, and its offset there.
    auto f_of = [](int R) { return (R >> 1) & 7; };
    auto turn_of = [](int t) {
        return HM == 128 ? ((t & 3) | (((t >> 3) & 1) << 2)) : (((t >> 1) & 1) | (((t >> 3) & 1) << 1));
    };
    constexpr int TURNED_CHUNKS = HM / 8;                       // 16-byte chunks of a turned row
    auto chunk_of = [&](bool turned, int i, int *row) {
        const int q = i * THREADS + tid;
        if (!turned) {
            *row = q / 8;
            return (q % 8) ^ f_of(*row);
        }
        *row = q / TURNED_CHUNKS;
        const int c = q % TURNED_CHUNKS;
        return (((c >> 1) ^ turn_of(*row)) << 1) | (c & 1);
    };
    [[maybe_unused]] uint32_t off_a[2], off_b[2];
    [[maybe_unused]] int chunk_a, chunk_b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        // (the same chunk for both: their rows differ by a multiple of 16)
        int row;
        chunk_a = chunk_of(A_TURNED, i, &row);
        off_a[i] = (uint32_t)(row * (int)p.a[0].pitch + chunk_a * 16);
        chunk_b = chunk_of(B_TURNED, i, &row);
        if (K == Kind::kForward) row = feature_of_row(row);
        off_b[i] = (uint32_t)(row * (int)p.b[0].pitch + chunk_b * 16);
    }

    const int pitch_a = (int)p.a[0].pitch, pitch_b = (int)p.b[0].pitch;
    const int per_m = (int)((p.m + S::BM - 1) / S::BM);
    // Along the summed index: whole K-tiles (of a segment), elements of the one
    // after them, 16-byte chunks; kInput's second segment (dU, Wu) begins at K-tile
    // seg_depth.
    [[maybe_unused]] const int k_whole = (int)(p.k / KT), k_rest = (int)(p.k % KT);
    [[maybe_unused]] const int k_chunks = (int)((p.k * SIZE + 15) / 16);
    [[maybe_unused]] const int seg_depth = plan.depth / 2;
    // From one K-tile to the next, and from an operand to its second matrix (kInput:
    // as if it followed the first).
    const int64_t step_a = A_TURNED ? (int64_t)KT * pitch_a : kDeep;
    const int64_t step_b = B_TURNED ? (int64_t)KT * pitch_b : kDeep;
    [[maybe_unused]] const int64_t second_a =
        static_cast<const char *>(p.a[1].p) - static_cast<const char *>(p.a[0].p) - seg_depth * step_a;
    [[maybe_unused]] const int64_t second_b =
        static_cast<const char *>(p.b[1].p) - static_cast<const char *>(p.b[0].p) -
        (K == Kind::kInput ? seg_depth * step_b : 0);

    // The item: its K-tiles kt0 .. kt0 + count - 1, where they begin in both operands,
    // the rows (or columns) that exist in the halves, and for codes the scales of
    // the quarter of them that this wave loads.
    int part = -1, kt0 = 0, count = plan.depth, t;             // part: of a split tile, else -1
    if (j < plan.whole) {
        // Consecutive work-groups go to the 8 XCDs in turn; each XCD gets a
        // contiguous range of the whole tiles, whose operands meet in its L2.
        const int xcd = j % 8, q = plan.whole / 8, rem = plan.whole % 8;
        t = xcd * q + (xcd < rem ? xcd : rem) + j / 8;
    } else {
        part = j - plan.whole;
        const int in = part % plan.parts;
        t = plan.whole + part / plan.parts;
        kt0 = in * plan.share;
        const int left = plan.depth - kt0;
        count = left < plan.share ? left : plan.share;
    }
    const Tile tile = tile_at(plan, t);
    const int which = K == Kind::kWeight && tile.m >= per_m;
    const int64_t m0 = (int64_t)(tile.m - which * per_m) * S::BM;
    const int64_t n0 = (int64_t)tile.n * (K == Kind::kForward ? HN : S::BN);
    const char *const item_a =
        static_cast<const char *>(p.a[which].p) + m0 * (A_TURNED ? SIZE : pitch_a) + kt0 * step_a;
    const char *const item_b =
        static_cast<const char *>(p.b[0].p) + n0 * (B_TURNED ? SIZE : pitch_b) + kt0 * step_b;
    int here_a[2], here_b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        here_a[h] = clamp(p.m - m0 - h * HM, HM);
        here_b[h] = clamp(p.n - n0 - (K == Kind::kForward ? 0 : h * HN), HN);
    }
    [[maybe_unused]] const char *item_scale = nullptr;
    [[maybe_unused]] int here_scale = 0;
    [[maybe_unused]] int64_t scale_pitch = 0;
    if constexpr (SCALED) {
        const int quarter = __builtin_amdgcn_readfirstlane(tid / HM);
        const Matrix &scales = quarter >= 2 ? p.b_scale[quarter & 1] : p.a_scale;
        const int64_t first = quarter >= 2 ? n0 : m0 + quarter * HM;
        scale_pitch = scales.pitch;
        item_scale = static_cast<const char *>(scales.p) + first * 4 + kt0 * scale_pitch;
        here_scale = clamp(scale_pitch / 4 - first, HM) * 4;
    }

    // Loads; K-tile kt counts from the item's first, and those past its last are zeros.
    // All of this is the same for every lane but the offset, which is out of bounds
    // for chunks past a row's end, and all choices are selects: a branch here would
    // part the products from what is to run beside them.
    auto load = [&](uint8_t *buf, const char *base, int records, const uint32_t (&off)[2], bool in) {
#if defined(__HIP_DEVICE_COMPILE__)      // the host pass does not know the resource type
        // 0x00020000: raw 32-bit data.
        const auto r = __builtin_amdgcn_make_buffer_rsrc((void *)base, 0, records, 0x00020000);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (__attribute__((address_space(3))) void *)(buf + (i * THREADS + wave * kWave) * 16),
                16, in ? off[i] : 0x80000000u, 0, 0, 0);
#endif
    };
    // A half of an operand, `more` bytes from the first one.
    auto load_half = [&](auto turned, uint8_t *buf, const char *base, int64_t step, int64_t second,
                         int64_t more, int here, int pitch, const uint32_t (&off)[2], int chunk, int kt) {
        int in_seg = kt0 + kt;
        if constexpr (K == Kind::kInput) {
            const bool seg = in_seg >= seg_depth;
            in_seg -= seg ? seg_depth : 0;
            more += seg ? second : 0;
        }
        base += kt * step + more;
        int records;
        bool in;
        if constexpr (decltype(turned)::value != 0) {
            records = (in_seg < k_whole ? KT : in_seg == k_whole ? k_rest : 0) * pitch;
            in = chunk < (here + 7) / 8;
        } else {
            records = here * pitch;
            in = chunk + in_seg * 8 < k_chunks;
        }
        load(buf, base, kt < count ? records : 0, off, in);
    };
    auto load_a = [&](auto stage, auto half, int kt) {
        constexpr int h = decltype(half)::value;
        load_half(Int<A_TURNED>{}, lds_a(stage, half), item_a, step_a, second_a,
                  (int64_t)(h * HM) * (A_TURNED ? SIZE : pitch_a), here_a[h], pitch_a, off_a, chunk_a, kt);
    };
    auto load_b = [&](auto stage, auto half, int kt) {
        constexpr int h = decltype(half)::value;
        // (forward: the second half is the same rows of the other weight)
        load_half(Int<B_TURNED>{}, lds_b(stage, half), item_b, step_b, second_b,
                  h == 0 ? 0 : K == Kind::kForward ? second_b : (int64_t)HN * SIZE, here_b[h], pitch_b,
                  off_b, chunk_b, kt);
    };
    // Scales of a K-tile: one 4-byte load a thread.
    [[maybe_unused]] const uint32_t scale_off = tid % HM * 4;
    auto load_scales = [&](auto stage, int kt) {
#if defined(__HIP_DEVICE_COMPILE__)
        if constexpr (SCALED) {
            const auto r = __builtin_amdgcn_make_buffer_rsrc(
                (void *)(item_scale + kt * scale_pitch), 0, kt < count ? here_scale : 0, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (__attribute__((address_space(3))) void *)(lds_s(stage) + wave * kWave * 4), 4,
                scale_off, 0, 0, 0);
        }
#endif
    };

    // Fragment addresses.  Rows of 128 bytes: lane (g, r) reads chunk g (then
    // 4 + g) of row r.  Turned: 8 bytes of row 8 g + r / 4 (then + 4), which
    // the read hands out as column r of them; a wave's units differ in their
    // low bits only, so fragment i's unit is the first one's XOR i.
    auto first_of = [&](bool turned, int row) {
        if (!turned) return (row + place.r) * kDeep + ((place.g ^ f_of(row + place.r)) * 16);
        const int t = 8 * place.g + (place.r >> 2);
        return t * HM * 2 + (((row / 16) ^ turn_of(t)) * 32) + (place.r & 3) * 8;
    };
    int at_a = first_of(A_TURNED, place.wm * (HM / S::WM));
    int at_b = first_of(B_TURNED, place.wn * (HN / S::WN));
    auto read = [&](auto turned, uint8_t *buf, int at, int i) {
        Fragment f;
        if constexpr (decltype(turned)::value != 0) {
            uint8_t *q = buf + (at ^ (i * 32));
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                union { s4v s[2]; u4v v; } u;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    u.s[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) s4v *)(q + (32 * kk + 4 * e) * HM * 2));
                f.v[kk] = u.v;
            }
        } else {
            f.v[0] = *reinterpret_cast<const u4v *>(buf + at + i * 16 * kDeep);
            f.v[1] = *reinterpret_cast<const u4v *>(buf + (at ^ 64) + i * 16 * kDeep);
        }
        return f;
    };
    // The scales of a wave's fragments of a half share a register, a byte each.
    Fragment fa[S::SETS][MF], fb[2][NF];
    int sa[2] = {}, sb[2] = {};
    // Where they are among those of a K-tile (see ScaleTiles), from the first
    // fragment's row on.  (Opaque: a sum taken apart into several additions to the
    // pointer hides from the compiler which variable is read.)
    auto scales_at = [&](int row) {
        int at = S_AT + (row / 64 * 64 + place.g * 16 + place.r) * 4 + row % 64 / 16;
        asm volatile("" : "+v"(at));
        return at;
    };
    [[maybe_unused]] int at_sa = 0, at_sb = 0;
    if constexpr (SCALED) {
        at_sa = scales_at(place.wm * (HM / S::WM));
        at_sb = scales_at(2 * HM + place.wn * (HN / S::WN));
    }
    auto read_scales = [&](auto stage, int at, auto count) {
        [[maybe_unused]] const uint8_t *const q = lds(stage) + at;
        if constexpr (decltype(count)::value == 4) return *reinterpret_cast<const int *>(q);
        else return (int)*reinterpret_cast<const uint16_t *>(q);
    };
    auto read_a_scales = [&](auto stage, auto half) {
        constexpr int h = decltype(half)::value;
        if constexpr (SCALED) sa[h] = read_scales(stage, at_sa + h * HM * 4, Int<MF>{});
    };
    auto read_a = [&](auto stage, auto half, auto index) {
        constexpr int i = decltype(index)::value;
        fa[decltype(half)::value % S::SETS][i] = read(Int<A_TURNED>{}, lds_a(stage, half), at_a, i);
    };
    auto read_b = [&](auto stage, auto half) {
        constexpr int h = decltype(half)::value;
#pragma unroll
        for (int j = 0; j < NF; ++j) fb[h][j] = read(Int<B_TURNED>{}, lds_b(stage, half), at_b, j);
        if constexpr (SCALED)
            sb[h] = read_scales(stage, at_sb + h * HM * 4, Int<NF>{});
    };
    f4v sum[2][2][MF][NF];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int e = 0; e < NF; ++e) sum[q >> 1][q & 1][i][e] = (f4v){0.0f, 0.0f, 0.0f, 0.0f};
    // Products of a row fragment with a half of B.
    auto multiply = [&](auto qa, auto qb, auto fi) {
        constexpr int a = decltype(qa)::value, b = decltype(qb)::value, i = decltype(fi)::value;
        for_each<NF>([&](auto fj) {
            constexpr int j = decltype(fj)::value;
            sum[a][b][i][j] =
                El::template run<j, i>(fb[b][j], fa[a % S::SETS][i], sum[a][b][i][j], sb[b], sa[a]);
        });
    };

    // K-tile t lies in stage t % RING.  (An item takes whole rings of them: an exit in
    // between would make the compiler wait for all loads at its target.)
    // Loads are in the order A0, F, scales, S, A1 of each K-tile, so "the half has
    // arrived" is a count of those after it.
    using C0 = Int<0>;
    using C1 = Int<1>;
    constexpr int L = S::LOADS, SL = SCALED ? 1 : 0, RING = S::RING;
    for_each<RING>([&](auto stage) {
        constexpr int t = decltype(stage)::value;
        load_a(stage, C0{}, t);
        load_b(stage, Int<t & 1>{}, t);
        load_scales(stage, t);
        load_b(stage, Int<1 - (t & 1)>{}, t);
        if constexpr (t + 1 < RING) load_a(stage, C1{}, t);
    });
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((RING - 1) * (4 * L + SL)) : "memory");
    read_a_scales(C0{}, C0{});
    for_each<MF>([&](auto i) { read_a(C0{}, C0{}, i); });
    read_b(C0{}, C0{});

    auto pin = [] { __builtin_amdgcn_sched_barrier(0); };
    auto barrier = [&](auto later) {
        pin();
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(decltype(later)::value) : "memory");
        pin();
    };
    // The products of a half of A that is used for the last time with half b of B, and
    // the reads of the half that follows it.
    auto last_use = [&](auto qa, auto qb, auto stage, auto half) {
        read_a_scales(stage, half);
        if constexpr (S::SETS == 2) for_each<MF>([&](auto i) { read_a(stage, half, i); });
        for_each<MF>([&](auto i) {
            multiply(qa, qb, i);
            if constexpr (S::SETS == 1) {
                pin();
                read_a(stage, half, i);
            }
        });
        pin();
    };
    auto k_tile = [&](auto stage, int kt) {
        using Now = decltype(stage);
        using Next = Int<(Now::value + 1) % RING>;
        using Before = Int<(Now::value + RING - 1) % RING>;
        using F = Int<Now::value & 1>;
        using G = Int<1 - F::value>;                 // S above
        // (A0, F)
        if constexpr (APART) load_a(Before{}, C1{}, kt + RING - 1);
        read_b(Now{}, G{});
        if constexpr (!APART) load_a(Before{}, C1{}, kt + RING - 1);
        for_each<MF>([&](auto i) { multiply(C0{}, F{}, i); });
        barrier(Int<(RING - 1) * (4 * L + SL)>{});
        // (A0, S), A1 read.  (A load into the variable that is read follows the reads.)
        if constexpr (APART) load_a(Now{}, C0{}, kt + RING);
        last_use(C0{}, G{}, Now{}, C1{});
        if constexpr (!APART) load_a(Now{}, C0{}, kt + RING);
        // (A1, S)
        load_b(Now{}, F{}, kt + RING);
        for_each<MF>([&](auto i) { multiply(C1{}, G{}, i); });
        barrier(Int<3 * L + (RING - 2) * (4 * L + SL)>{});
        // (A1, F), the next A0 and F read
        load_scales(Now{}, kt + RING);
        load_b(Now{}, G{}, kt + RING);
        read_b(Next{}, G{});
        last_use(C1{}, F{}, Next{}, C0{});
    };
    for (int kt = 0; kt < count; kt += RING)
        for_each<RING>([&](auto stage) { k_tile(stage, kt + decltype(stage)::value); });
    // (loads of nothing may still be on their way to LDS)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    if (part >= 0) {
        float *const slab = p.slabs + (int64_t)part * S::SLAB;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int e = 0; e < NF; ++e) {
                    const int at = ((q >> 1) * MF + i) * 4 + (q & 1) * 2 + e;
                    *reinterpret_cast<f4v *>(slab + (int64_t)(at * THREADS + tid) * 4) =
                        sum[q >> 1][q & 1][i][e];
                }
        return;
    }
    const Finish<E, K, S> finish{p, place, tile};
#pragma unroll
    for (int qa = 0; qa < 2; ++qa)
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const f4v v[2][2] = {{sum[qa][0][i][0], sum[qa][0][i][1]},
                                 {sum[qa][1][i][0], sum[qa][1][i][1]}};
            finish(qa, i, v);
        }
}

template <typename E, Kind K, typename S>
__global__ __launch_bounds__(S::THREADS) void product_kernel(Product p, Plan plan) {
    using M = Lds<E, S>;
    __shared__ __align__(1024) uint8_t a00[M::HALF], a01[M::HALF], a10[M::HALF], a11[M::HALF],
        b0[M::REST], b1[M::REST], b2[M::MORE], b3[M::MORE];
    multiply_item<E, K, S>(p, plan, blockIdx.x, M{{a00, a01, a10, a11}, {b0, b1, b2, b3}});
}

// Both products of a small backward pass in one launch: neither fills the GPU.
template <typename E, typename S>
__global__ __launch_bounds__(S::THREADS) void both_kernel(Product input, Plan input_plan, Product weight,
                                                          Plan weight_plan) {
    using M = Lds<E, S>;
    __shared__ __align__(1024) uint8_t a00[M::HALF], a01[M::HALF], a10[M::HALF], a11[M::HALF],
        b0[M::REST], b1[M::REST], b2[M::MORE], b3[M::MORE];
    const M mem = {{a00, a01, a10, a11}, {b0, b1, b2, b3}};
    const int j = (int)blockIdx.x;
    if (j < input_plan.items)
        multiply_item<E, Kind::kInput, S>(input, input_plan, j, mem);
    else
        multiply_item<E, Kind::kWeight, S>(weight, weight_plan, j - input_plan.items, mem);
}

// Adds the parts of split tile `split` in order and finishes row fragment `part` of it.
// (64 tiles of 256x256 in four parts, 67 MB: 13.7 us, 4.9 TB/s.)
template <typename E, Kind K, typename S>
__device__ __forceinline__ void join_parts(const Product &p, const Plan &plan, int split, int part) {
    const Place<S> place(threadIdx.x);
    const Tile tile = tile_at(plan, plan.whole + split);
    const float *at = p.slabs + (int64_t)split * plan.parts * S::SLAB +
                      ((int64_t)part * 4 * S::THREADS + threadIdx.x) * 4;
    f4v v[2][2] = {};
    for (int q = 0; q < plan.parts; ++q, at += S::SLAB)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e >> 1][e & 1] += *reinterpret_cast<const f4v *>(at + (int64_t)e * S::THREADS * 4);
    Finish<E, K, S>{p, place, tile}(part / S::MF, part % S::MF, v);
}
template <typename E, Kind K, typename S>
__global__ __launch_bounds__(S::THREADS) void join_kernel(Product p, Plan plan) {
    join_parts<E, K, S>(p, plan, blockIdx.x, blockIdx.y);
}
template <typename E, typename S>
__global__ __launch_bounds__(S::THREADS) void join_both_kernel(Product input, Plan input_plan, int splits,
                                                               Product weight, Plan weight_plan) {
    const int j = (int)blockIdx.x;
    if (j < splits) join_parts<E, Kind::kInput, S>(input, input_plan, j, blockIdx.y);
    else join_parts<E, Kind::kWeight, S>(weight, weight_plan, j - splits, blockIdx.y);
}

// ---------------------------------------------------------------- host ----

inline int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

enum class Size { kLarge, kSmall, kDeep };
struct Choice {
    Size size;
    Plan plan;
    int64_t split_tiles, slab_floats;
};

// What a plan's parts cost in microseconds, as measured on an MI355X: a round of
// tiles' beginning and end, a K-tile while every place of the GPU has a tile and
// while half of them or fewer have one (between, the share that is taken counts),
// and a part's sums, written and read.  Measured forward without G and U, at
// 16, 32 and 64 K-tiles in us:
//     large, 256 / 512 / 768 tiles    33, 57, 104 / 63, 113, 205 / 91, 165, 307
//     large, 32 / 128 tiles           25, 42, 76 / 28, 45, 78
//     small, 512 / 1024 / 2048 tiles  25, 37, 69 / 39, 71, 133 / 74, 137, 259
//     small, 128 / 256 tiles          15, 23, 38 / 15, 23, 41
//     deep, 128 / 256 / 512 tiles     15, 21, 34 / 15, 21, 38 / 24, 40, 74
// (64x64 outputs a wave read twice as much LDS for a product as 128x64: small tiles
// are bound by that, at 0.35 us a K-tile.)  The backward products take the same or
// up to a fifth more: turned fragments are twice as many reads.  A K-tile of codes
// takes the same time as one of 16-bit elements.
struct Cost {
    int places;            // work-groups that run at once
    double fixed, step, alone, part;
};
constexpr Cost kLargeCost = {256, 8.0, 1.48, 1.06, 0.08};
constexpr Cost kSmallCost = {512, 6.5, 0.95, 0.55, 0.015};
constexpr Cost kDeepCost = {256, 8.0, 0.50, 0.45, 0.015};
constexpr double kJoinUs = 5.0;

inline double groups_us(const Cost &c, int64_t groups, int64_t steps) {
    const int64_t left = groups % c.places;
    const double more = 2.0 * (double)left / c.places - 1.0;
    const double step = c.alone + (c.step - c.alone) * (more > 0.0 ? more : 0.0);
    return (double)(groups / c.places) * (c.fixed + (double)steps * c.step) +
           (left == 0 ? 0.0 : c.fixed + (double)steps * step);
}

template <typename S>
Choice choice_for(Kind kind, const Product &p, int size, const Cost &c, double *us) {
    Choice r = {};
    const int64_t kt = kDeep / size;
    const int64_t depth = up(p.k, kt) * (kind == Kind::kInput ? 2 : 1);
    const int64_t tm = up(p.m, S::BM) * (kind == Kind::kWeight ? 2 : 1);
    const int64_t tn = up(p.n, kind == Kind::kForward ? S::HN : S::BN), tiles = tm * tn;
    const int64_t left = tiles % c.places;
    auto rounds_us = [&](int64_t groups, int64_t steps) {
        return groups_us(c, groups, up(steps, S::RING) * S::RING);
    };
    double best = rounds_us(tiles, depth);
    r.plan = {(int32_t)tm, (int32_t)tn, (int32_t)tiles, 1, (int32_t)depth, (int32_t)depth, (int32_t)tiles};
    for (int64_t split : {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
        if (left == 0 || split * 4 > depth) break;
        const int64_t share = up(depth, split), parts = up(depth, share);
        const double t = rounds_us(tiles - left, depth) + rounds_us(left * parts, share) +
                         (double)(left * parts) * c.part + kJoinUs;
        if (t >= best) continue;
        best = t;
        r.plan.whole = (int32_t)(tiles - left);
        r.plan.parts = (int32_t)parts;
        r.plan.share = (int32_t)share;
        r.plan.items = (int32_t)(tiles - left + left * parts);
        r.split_tiles = left;
        r.slab_floats = left * parts * S::SLAB;
    }
    r.size = S::BM == 256 ? Size::kLarge : S::RING == 2 ? Size::kSmall : Size::kDeep;
    *us = best;
    return r;
}

inline Choice choose(Kind kind, const Product &p, int size, double *us = nullptr) {
    double large_us, small_us, deep_us;
    const Choice large = choice_for<Large>(kind, p, size, kLargeCost, &large_us);
    const Choice small = choice_for<Small>(kind, p, size, kSmallCost, &small_us);
    const Choice deep = choice_for<Deep>(kind, p, size, kDeepCost, &deep_us);
    const double other_us = large_us <= small_us ? large_us : small_us;
    if (us) *us = deep_us <= other_us ? deep_us : other_us;
    if (deep_us <= other_us) return deep;
    return large_us <= small_us ? large : small;
}

template <typename E, Kind K, typename S>
taco_status launch_product(const Product &p, const Choice &c, hipStream_t stream) {
    const taco_status st = launch(reinterpret_cast<const void *>(&product_kernel<E, K, S>),
                                  dim3((unsigned)c.plan.items), S::THREADS, stream, p, c.plan);
    if (st != TACO_OK || c.split_tiles == 0) return st;
    return launch(reinterpret_cast<const void *>(&join_kernel<E, K, S>),
                  dim3((unsigned)c.split_tiles, 2 * S::MF), S::THREADS, stream, p, c.plan);
}

template <typename E, Kind K>
taco_status run_kind(const Product &p, hipStream_t stream) {
    const Choice c = choose(K, p, Element<E>::SIZE);
    switch (c.size) {
        case Size::kLarge: return launch_product<E, K, Large>(p, c, stream);
        case Size::kSmall: return launch_product<E, K, Small>(p, c, stream);
        default: return launch_product<E, K, Deep>(p, c, stream);
    }
}

// A backward pass that wants both products.  Where neither takes large tiles they are
// one launch of small ones, each with half of the places (999 x 1030x1111: 24 us,
// one after the other 14 and 18, and one join).
struct Pair {
    bool together;
    Choice input, weight;
};
inline Pair pair_of(const Product &input, const Product &weight, int size) {
    Pair r = {};
    r.together = choose(Kind::kInput, input, size).size != Size::kLarge &&
                 choose(Kind::kWeight, weight, size).size != Size::kLarge;
    if (!r.together) return r;
    Cost half = kSmallCost;
    half.places /= 2;
    double us;
    r.input = choice_for<Small>(Kind::kInput, input, size, half, &us);
    r.weight = choice_for<Small>(Kind::kWeight, weight, size, half, &us);
    return r;
}

}  // namespace

template <typename E>
int64_t Products<E>::workspace(Kind kind, const Product &p) {
    return choose(kind, p, Element<E>::SIZE).slab_floats * (int64_t)sizeof(float);
}

template <typename E>
taco_status Products<E>::run(Kind kind, const Product &p, hipStream_t stream) {
    if constexpr (Element<E>::SCALED) {
        return run_kind<E, Kind::kForward>(p, stream);
    } else {
        switch (kind) {
            case Kind::kForward: return run_kind<E, Kind::kForward>(p, stream);
            case Kind::kInput: return run_kind<E, Kind::kInput>(p, stream);
            default: return run_kind<E, Kind::kWeight>(p, stream);
        }
    }
}

template <typename E>
int64_t Products<E>::pair_workspace(const Product &input, const Product &weight) {
    const Pair c = pair_of(input, weight, Element<E>::SIZE);
    if (c.together) return (c.input.slab_floats + c.weight.slab_floats) * (int64_t)sizeof(float);
    // One after the other, in the same place.
    const int64_t i = workspace(Kind::kInput, input), w = workspace(Kind::kWeight, weight);
    return i > w ? i : w;
}

template <typename E>
taco_status Products<E>::run_pair(const Product &input, Product weight, hipStream_t stream) {
    if constexpr (Element<E>::SCALED) {
        return TACO_ERR_FORMAT;            // codes have no backward pass
    } else {
        const Pair c = pair_of(input, weight, Element<E>::SIZE);
        if (!c.together) {
            const taco_status st = run(Kind::kInput, input, stream);
            return st != TACO_OK ? st : run(Kind::kWeight, weight, stream);
        }
        weight.slabs += c.input.slab_floats;
        const taco_status st =
            launch(reinterpret_cast<const void *>(&both_kernel<E, Small>),
                   dim3((unsigned)(c.input.plan.items + c.weight.plan.items)), Small::THREADS, stream,
                   input, c.input.plan, weight, c.weight.plan);
        const int64_t splits = c.input.split_tiles + c.weight.split_tiles;
        if (st != TACO_OK || splits == 0) return st;
        return launch(reinterpret_cast<const void *>(&join_both_kernel<E, Small>),
                      dim3((unsigned)splits, 2 * Small::MF), Small::THREADS, stream, input,
                      c.input.plan, (int)c.input.split_tiles, weight, c.weight.plan);
    }
}

}  // namespace taco_gated
