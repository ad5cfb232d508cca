// Declarations shared by the translation units of libtaco_gated: the matrix
// products (taco_gated_product.hpp, compiled once per operand type), the
// products of few rows (taco_gated_few.hpp), the element-wise kernels
// (taco_gated_rows.hip) and the C ABI (taco_gated_abi.hip).
#pragma once

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "taco_gated.h"

namespace taco_gated {

struct BF16 { typedef __bf16 type; };
struct F16 { typedef _Float16 type; };

// A matrix in memory: rows `pitch` bytes apart.
struct Matrix {
    const void *p;
    int64_t pitch;
};

// One product.  Operands may be read 16 bytes at a time from 16-byte
// boundaries, with pitches below kMaxPitch; `contiguous` counts below are the
// operands' own lengths along their contiguous dimension.
//
//   kForward   out[t][f]: G = X Wg^T, U = X Wu^T, then act(G) U (and G, U)
//   kInput     out[t][h] = dG Wg + dU Wu
//   kWeight    out[f][h] = dG^T X and dU^T X
enum class Kind { kForward, kInput, kWeight };

constexpr int64_t kMaxPitch = INT64_C(1) << 23;

struct Product {
    // kForward: a = X, b = Wg, Wu.  kInput: a = dG, dU, b = Wg, Wu.
    // kWeight: a = dG, dU, b = X (twice).
    Matrix a[2], b[2];
    // kForward of codes, E8M0 bytes.  few(): rows as they are; run(): by K-tile, as
    // tile_scales() lays them out (pitch: bytes of a K-tile).
    Matrix a_scale, b_scale[2];
    void *out[3];                      // kForward: A, G, U (the last two may be null)
    int64_t out_pitch[3];              // in elements
    int64_t m, n, k;                   // rows, columns and summed length of one out
    int32_t activation;
    int32_t out_f16;                   // kForward of codes: type of A
    float *slabs;                      // partial sums of a split
};

// Bytes of slabs that a product needs, and the product.
template <typename E> struct Products {
    static int64_t workspace(Kind kind, const Product &p);
    static taco_status run(Kind kind, const Product &p, hipStream_t stream);
    // kInput and kWeight of one backward pass; slabs are input's.
    static int64_t pair_workspace(const Product &input, const Product &weight);
    static taco_status run_pair(const Product &input, Product weight, hipStream_t stream);
    // Whether few() is to make kForward (p: the sizes), and not run() after copies of
    // so many bytes.
    static bool few_takes(const Product &p, int64_t copy_bytes);
    // kForward of at most kFewRows rows; operands at any 2-byte (codes:
    // 16-byte) boundary.
    static taco_status few(const Product &p, hipStream_t stream);
};
struct Codes {};
extern template struct Products<BF16>;
extern template struct Products<F16>;
extern template struct Products<Codes>;

constexpr int64_t kFewRows = 64;

// dG = dA U act'(G), dU = dA act(G) into rows of `to_pitch` elements (a
// multiple of 8; elements past the last are zero).
struct ActivationGrad {
    const void *da, *gate, *up;
    void *dgate, *dup;
    int64_t ldda, ldgu, to_pitch, rows;
    int32_t features, activation;
};
// Rows of `width` bytes to rows `to_pitch` bytes apart (a multiple of 16) on
// 16-byte boundaries, with zeros behind them.
struct Repack {
    const void *from;
    void *to;
    int64_t from_pitch, to_pitch, rows;
    int64_t width;
};
taco_status repack(const Repack *r, int count, hipStream_t stream);      // count <= 3
// (with the copies in the same launch)
taco_status activation_grad(const ActivationGrad &a, bool f16, const Repack *r, int count,
                            hipStream_t stream);

// Feature of LDS row R of a forward B half: of each 32 features, column fragment
// j takes 8 q + 4 j + (0..3), so that a lane's two fragments are eight
// neighbours.
__host__ __device__ constexpr int feature_of_row(int R) {
    return (R & ~31) | (((R >> 2) & 3) << 3) | (((R >> 4) & 1) << 2) | (R & 3);
}

// Rows of `width` scale bytes (one a block of 32) to where a K-tile of 128 codes
// finds its own together, in the order in which lanes take them:
// [K-tile][64 rows][block g][row r of 16][rows r, 16 + r, 32 + r, 48 + r], zeros
// where there is no row or block.  features: rows in the order of feature_of_row.
struct ScaleTiles {
    const uint8_t *from;
    uint32_t *to;
    int64_t rows;
    int32_t width, features;
};
inline int64_t scale_tile_pitch(int64_t rows) { return (rows + 63) / 64 * 256; }
inline int64_t scale_tile_bytes(int64_t rows, int64_t width) {
    return (width + 3) / 4 * scale_tile_pitch(rows);
}
taco_status tile_scales(const ScaleTiles *s, int count, hipStream_t stream);      // count <= 3

taco_status fill_zero(void *p, int64_t n16, hipStream_t stream);         // n16 16-bit zeros

struct Encode {
    const void *x;
    uint8_t *codes, *scales;
    int64_t ldx, rows, hidden;
};
taco_status encode(const Encode &e, taco_norm_dtype dtype, hipStream_t stream);

// The status is the launch's own (not an earlier error left in the runtime).
template <typename... Args>
taco_status launch(const void *fn, dim3 grid, int threads, hipStream_t stream, Args... args) {
    void *ptrs[] = {static_cast<void *>(&args)...};
    const hipError_t err = hipLaunchKernel(fn, grid, dim3((unsigned)threads), ptrs, 0, stream);
    return err == hipSuccess ? TACO_OK : TACO_ERR_HIP;
}

}  // namespace taco_gated
