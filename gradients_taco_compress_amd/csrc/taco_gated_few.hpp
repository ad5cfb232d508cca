// Forward pass of the gated block for few rows (the tokens that a serving step
// adds): both weights are read once, which is nearly all the time it takes, so
// they go from memory to the matrix instructions' registers without LDS in
// between.
//
//  * A wave multiplies RF fragments of 16 rows by 16 gate and the 16 same up
//    features.  Lane (g, r) reads chunks of feature r (and of row r of X, which
//    stays in cache); the waves of a work-group share the summed length, and
//    their sums are added in LDS, in order.
//  * A wave's turn takes 128 bytes of each feature.  All its loads are issued before
//    they are waited for; where turns are held ahead, the next round's go out
//    between the products of this one.
//
// Bound by HBM: 1 x 10240x2560 bf16 20.6 to 23.3 us (5.1 to 4.5 TB/s), 4 x 14336x3584
// codes 23.2 to 25.1 us (4.6 to 4.2); else by what a CU takes in, X's rows among it:
// 34 GB/s a CU (codes 25).  Few features fill few CUs (1 x 256x8192: bf16 18.7 us,
// codes 14.1).
#pragma once

#include <type_traits>

#include "taco_gated_product.hpp"

namespace taco_gated {
namespace {

template <typename E, int WAVES, int AHEAD, int RF>
__global__ __launch_bounds__(WAVES * kWave) void few_kernel(Product p) {
    using El = Element<E>;
    constexpr int SIZE = El::SIZE;
    constexpr bool SCALED = El::SCALED;
    constexpr int N = 2 + RF;                               // row fragments: gate, up, X
    static_assert(RF <= WAVES, "a wave to a fragment of X at the end");
    __shared__ f4v sums[WAVES][2 * RF][kWave];
    const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, r = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    const int64_t f = f0 + r < p.n ? f0 + r : p.n - 1;
    // Rows of gate, up and X; those past the last are repeated and not stored.
    const char *rows[N] = {static_cast<const char *>(p.b[0].p) + f * p.b[0].pitch,
                           static_cast<const char *>(p.b[1].p) + f * p.b[1].pitch};
    [[maybe_unused]] const uint8_t *scales[N] = {};
    if constexpr (SCALED) {
        scales[0] = static_cast<const uint8_t *>(p.b_scale[0].p) + f * p.b_scale[0].pitch;
        scales[1] = static_cast<const uint8_t *>(p.b_scale[1].p) + f * p.b_scale[1].pitch;
    }
#pragma unroll
    for (int i = 0; i < RF; ++i) {
        const int64_t m = 16 * i + r < p.m ? 16 * i + r : p.m - 1;
        rows[2 + i] = static_cast<const char *>(p.a[0].p) + m * p.a[0].pitch;
        if constexpr (SCALED)
            scales[2 + i] = static_cast<const uint8_t *>(p.a_scale.p) + m * p.a_scale.pitch;
    }
    const int64_t bytes = p.k * SIZE;
    // A K-tile of 128 bytes of each row.
    struct Turn {
        Fragment v[N];
        int scale[N];
    };
    Turn held[AHEAD];
    auto load = [&](int64_t turn, Turn &to) {
        const int64_t at = turn * kDeep;
#pragma unroll
        for (int s = 0; s < N; ++s) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                to.v[s].v[h] = *reinterpret_cast<const u4v_any *>(rows[s] + at + h * 64 + g * 16);
            if constexpr (SCALED) to.scale[s] = scales[s][at / 32 + g];
        }
    };
    // What is left of each row: past its end is zero.
    auto load_rest = [&](int64_t turn, Turn &to) {
        const int64_t at = turn * kDeep;
#pragma unroll
        for (int s = 0; s < N; ++s) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t c = at + h * 64 + g * 16, left = bytes - c;
                to.v[s].v[h] = (u4v){0u, 0u, 0u, 0u};
                if (left > 0)
                    to.v[s].v[h] = load_tail<true>(rows[s] + c, rows[s], left < 16 ? (int)left : 16);
            }
            if constexpr (SCALED) {
                const int64_t block = at / 32 + g;
                to.scale[s] = block < p.k / 32 ? scales[s][block] : 0;
            }
        }
    };
    f4v gate[RF], up[RF];
#pragma unroll
    for (int i = 0; i < RF; ++i) gate[i] = up[i] = (f4v){0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Turn &in) {
#pragma unroll
        for (int i = 0; i < RF; ++i) {
            gate[i] = El::template run<0, 0>(in.v[0], in.v[2 + i], gate[i], in.scale[0], in.scale[2 + i]);
            up[i] = El::template run<0, 0>(in.v[1], in.v[2 + i], up[i], in.scale[1], in.scale[2 + i]);
        }
    };
    const int64_t turns = bytes / kDeep;
    int64_t turn = wave;
    // Whole rounds of AHEAD turns, the next round's loads between the products.
    if (turn + (AHEAD - 1) * WAVES < turns) {
        for_each<AHEAD>([&](auto i) { load(turn + decltype(i)::value * WAVES, held[decltype(i)::value]); });
        for (turn += AHEAD * WAVES; turn + (AHEAD - 1) * WAVES < turns; turn += AHEAD * WAVES)
            for_each<AHEAD>([&](auto i) {
                constexpr int n = decltype(i)::value;
                multiply(held[n]);
                load(turn + n * WAVES, held[n]);
            });
        for_each<AHEAD>([&](auto i) { multiply(held[decltype(i)::value]); });
    }
    // Fewer than AHEAD turns, together.
    for_each<AHEAD - 1>([&](auto i) {
        constexpr int n = decltype(i)::value;
        if (turn + n * WAVES < turns) load(turn + n * WAVES, held[n]);
    });
    for_each<AHEAD - 1>([&](auto i) {
        constexpr int n = decltype(i)::value;
        if (turn + n * WAVES < turns) multiply(held[n]);
    });
    if (turns * kDeep < bytes && turns % WAVES == wave) {
        load_rest(turns, held[0]);
        multiply(held[0]);
    }
    // Wave i adds and finishes fragment i of X.
#pragma unroll
    for (int i = 0; i < RF; ++i) {
        sums[wave][2 * i][lane] = gate[i];
        sums[wave][2 * i + 1][lane] = up[i];
    }
    __syncthreads();
    if (wave >= RF) return;
    f4v all_gate = sums[0][2 * wave][lane], all_up = sums[0][2 * wave + 1][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        all_gate += sums[w][2 * wave][lane];
        all_up += sums[w][2 * wave + 1][lane];
    }
    // Lane (g, r): features 4 g + (0..3) of row r.
    const int64_t first = f0 + 4 * g, left = p.n - first, m = 16 * wave + r;
    if (m >= p.m || left <= 0) return;
    float vg[4], vu[4], out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        vg[e] = all_gate[e];
        vu[e] = all_up[e];
    }
    with_activation(p.activation, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = vg[e] * gate_share<decltype(act)::value>(vg[e]) * vu[e];
    });
    auto store = [&](auto *kind) {
        using T = typename std::remove_pointer<decltype(kind)>::type;
        store_row<T, 4>(static_cast<T *>(p.out[0]) + m * p.out_pitch[0] + first, out, left);
        if (p.out[1]) {
            store_row<T, 4>(static_cast<T *>(p.out[1]) + m * p.out_pitch[1] + first, vg, left);
            store_row<T, 4>(static_cast<T *>(p.out[2]) + m * p.out_pitch[2] + first, vu, left);
        }
    };
    if constexpr (SCALED) {
        if (p.out_f16) store(static_cast<_Float16 *>(nullptr));
        else store(static_cast<__bf16 *>(nullptr));
    } else {
        store(static_cast<typename El::type *>(nullptr));
    }
}

}  // namespace

// The products of up to 16 rows; of up to kFewRows where these few columns a
// work-group are estimated to take less than tiles and what tiles need: copies of
// operands that are not on 16-byte rows, scales by K-tile.  In us, this and tiles:
//     bf16    17 / 32 x 4096x4096     15.9, 18.3 and 23.5, 23.4
//     bf16    17 / 32 x 10240x2560    30.3, 35.8 and 28.1, 29.0
//     bf16    64 x 1024x1024          8.6 and 11.6
//     codes   17 / 64 x 4096x4096     12.2, 19.7 and 22.1, 21.9
//     codes   64 x 2048x512           4.7 and 8.8
// Up to 16 rows no estimate is made, so that such a call needs no workspace, whatever
// its operands' alignment.  That is the faster side nearly everywhere, not where few
// CUs have features or where 16-bit weights are large (1, 8 and 16 rows, this and tiles):
//     bf16    256x8192                18.7, 21.3, 23.9 and 22.1, 22.1, 22.1
//     bf16    768x2048                7.2, 7.8, 8.5 and 13.6, 13.5, 13.5
//     bf16    2048x7168               18.3, 20.3, 22.7 and 22.7, 22.4, 22.8
//     bf16    4096x4096               15.8, 15.5, 16.4 and 23.2, 23.5, 23.4
//     bf16    10240x2560              23.3, 24.2, 26.9 and 27.1, 27.3, 27.6
//     bf16    14336x3584              40.2, 40.3, 44.2 and 37.9, 37.6, 37.8
//     codes   256x8192                14.1, 16.7, 18.5 and 18.6, 18.3, 18.4
//     codes   4096x4096               9.9, 11.0, 11.7 and 22.7, 22.7, 22.5
//     codes   14336x3584              24.2, 25.2, 28.9 and 29.8, 29.6, 29.8
//     codes   14336x4096              30.1, 32.9, 36.3 and 34.8, 34.2, 34.3
template <typename E>
bool Products<E>::few_takes(const Product &p, int64_t copy_bytes) {
    constexpr int SIZE = Element<E>::SIZE;
    if (p.m <= 16) return true;
    if (p.m > kFewRows) return false;
    // Bytes of a CU's work-groups; rows that are read again and again count half.
    const int64_t fragments = p.m <= 32 ? 32 : 64, rounds = up(up(p.n, 16), 256);
    const double in = (double)rounds * (32.0 + 0.5 * (double)(p.m + fragments)) * (double)(p.k * SIZE);
    const double weights = 2.0 * (double)p.n * (double)(p.k * SIZE) / 5.0e6;
    const double cu = in / (SIZE == 1 ? 25.0e3 : 34.0e3);
    const double few_us = 3.0 + (cu > weights ? cu : weights);
    double tiles_us;
    const Choice c = choose(Kind::kForward, p, SIZE, &tiles_us);
    const double join = c.split_tiles ? kJoinUs + 0.015 * (c.plan.items - c.plan.whole) : 0.0;
    const double read = 4.0 + weights + 0.8 * join;
    if (read > tiles_us) tiles_us = read;
    if (SIZE == 1) tiles_us += 4.0;
    if (copy_bytes) tiles_us += 3.0 + (double)copy_bytes / 2.0e6;
    return few_us < tiles_us;
}

template <typename E>
taco_status Products<E>::few(const Product &p, hipStream_t stream) {
    const dim3 grid((unsigned)up(p.n, 16));
    // Turns held at once: 1, 3 and 4 of 16-bit elements take 22.9, 22.4 and 22.0 us at
    // 1 x 10240x2560, and of codes, whose turn is twice as long in summed elements,
    // 13.5, 16.5 and 16.5 us.  (Four waves 22.2 and 14.1 at their best, sixteen 24.0
    // and 15.5.)  More rows hold one (32 and 64 x 10240x2560: 35.8, 48.1 us; two 35.9, 53.2).
    constexpr int kAhead = Element<E>::SCALED ? 1 : 4;
    const void *fn = p.m <= 16   ? reinterpret_cast<const void *>(&few_kernel<E, 8, kAhead, 1>)
                     : p.m <= 32 ? reinterpret_cast<const void *>(&few_kernel<E, 8, 1, 2>)
                                 : reinterpret_cast<const void *>(&few_kernel<E, 8, 1, 4>);
    return launch(fn, grid, 8 * kWave, stream, p);
}

}  // namespace taco_gated
