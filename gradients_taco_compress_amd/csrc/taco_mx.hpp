// The block-scaled 8-bit form that libtaco_norm writes and libtaco_gated reads
// (taco_gated.h): 32 neighbours of a row share a scale 2^e, e the least integer
// >= -127 with max|y| <= 448 2^e; a code is E4M3(y / 2^e).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace taco_mx {
namespace {

typedef unsigned int u2 __attribute__((ext_vector_type(2)));

// Scale byte e + 127 of a block from the bits of max|y| as float32 (the larger
// of a NaN and a number is the NaN, by their bits): 448 = 1.75 2^8, so e is the
// exponent of the maximum less 8, and one more where its fraction passes 1.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
    if (max_bits >= 0x7F800000u) return 255u;
    const int byte = (int)((max_bits + 0x1FFFFFu) >> 23) - 8;
    return byte < 0 ? 0u : (uint32_t)byte;
}

// Codes of eight values of a block.  1 / scale is a power of two from 2^-120 to
// 2^127, so the quotient is exact (or far below the smallest code); the +0 turns
// -0 into +0.  |y / scale| <= 448: nothing saturates.
__device__ __forceinline__ u2 codes8(const float *y, uint32_t byte) {
    if (byte == 255u) return (u2){0x7F7F7F7Fu, 0x7F7F7F7Fu};
    const float inv = __uint_as_float((254u - byte) << 23);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float v = __builtin_fmaf(y[j], inv, 0.0f);
        q[j] = v;
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    return (u2){(uint32_t)lo, (uint32_t)hi};
}

__device__ __forceinline__ uint32_t abs_max8(const float *y) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t b = __float_as_uint(y[j]) & 0x7FFFFFFFu;
        m = b > m ? b : m;
    }
    return m;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}

// Maximum over four neighbouring lanes (4 q .. 4 q + 3).
__device__ __forceinline__ uint32_t max_of_four(uint32_t v) {
    return dpp_max<0x4E>(dpp_max<0xB1>(v));
}

}  // namespace
}  // namespace taco_mx
