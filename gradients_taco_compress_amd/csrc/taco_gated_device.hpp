// Device code that the kernels of libtaco_gated share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "taco_gated.h"
#include "taco_norm_device.hpp"

namespace taco_gated {
namespace {

using taco_norm::kWave;
using taco_norm::load_tail;
using taco_norm::u2v;
using taco_norm::u2v_any;
using taco_norm::u4v;
using taco_norm::u4v_any;

typedef float f2v __attribute__((ext_vector_type(2)));
typedef float f4v __attribute__((ext_vector_type(4)));

// f(Int<0>{}), ..., f(Int<N - 1>{}): bodies that need their index constant.
template <int I>
struct Int { static constexpr int value = I; };
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_each(F &&f) {
    if constexpr (I < N) {
        f(Int<I>{});
        for_each<N, I + 1>(f);
    }
}

// 1 / (1 + e^-z), accurate to a few float32 steps on both sides (0 where it is below
// 2^-126: z < -87.3).
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

constexpr float kRootEightOverPi = 1.5957691216057308f;

// act(g) / g, the factor between 0 and 1 that all three activations are made of.
template <int ACT>
__device__ __forceinline__ float gate_share(float g) {
    if constexpr (ACT == TACO_GATED_SILU) return sigmoid(g);
    // (erfc keeps the small values of the negative side)
    if constexpr (ACT == TACO_GATED_GELU) return 0.5f * erfcf(g * -0.70710678118654752f);
    // (1 + tanh z) / 2 = sigmoid(2 z)
    return sigmoid(kRootEightOverPi * g * __builtin_fmaf(0.044715f * g, g, 1.0f));
}

// act'(g) from the share.  Where |g| is large the share's own slope is zero in
// float32; the clamp keeps its factor finite there.
template <int ACT>
__device__ __forceinline__ float gate_slope(float g, float share) {
    const float t = __builtin_amdgcn_fmed3f(g, -64.0f, 64.0f);
    if constexpr (ACT == TACO_GATED_SILU) return share * __builtin_fmaf(t, 1.0f - share, 1.0f);
    if constexpr (ACT == TACO_GATED_GELU)
        return __builtin_fmaf(t * 0.39894228040143268f, __expf(-0.5f * t * t), share);
    const float inner = kRootEightOverPi * __builtin_fmaf(0.134145f * t, t, 1.0f);
    return __builtin_fmaf(t * share * (1.0f - share), inner, share);
}

// f with the activation as a constant.
template <typename F>
__device__ __forceinline__ void with_activation(int activation, F &&f) {
    if (activation == TACO_GATED_SILU) f(Int<TACO_GATED_SILU>{});
    else if (activation == TACO_GATED_GELU) f(Int<TACO_GATED_GELU>{});
    else f(Int<TACO_GATED_GELU_TANH>{});
}

// N neighbours of a row, of which `left` exist, rounded to T.
template <typename T, int N>
__device__ __forceinline__ void store_row(T *p, const float *v, int64_t left) {
    typedef T tn __attribute__((ext_vector_type(N)));
    typedef T tn_any __attribute__((ext_vector_type(N), aligned(sizeof(T))));
    typedef float fn __attribute__((ext_vector_type(N)));
    if (left >= N) {
        fn f;
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = v[i];
        *reinterpret_cast<tn_any *>(p) = __builtin_convertvector(f, tn);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left) p[i] = (T)v[i];
}

}  // namespace
}  // namespace taco_gated
