// activation.cuh -- the activations of the linear layer's epilogue and their
// derivatives, in binary32.
//
// With s(x) = 1 / (1 + exp(-x)) and P the normal distribution function:
//   silu       z s(z)            slope  s + z s (1 - s)
//   gelu       z P(z)            slope  P + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z s(2 u), u = sqrt(2/pi) (z + 0.044715 z^3), which is
//              z (1 + tanh u) / 2: one exponential instead of a tanh
//              slope  s + z s (1 - s) 2 u'
// The logistic uses the fast exponential and division (each good to a few
// binary32 steps, 2^-21 relative): far below the bf16 step of the results and
// the same order as the rounding of the sums they are applied to.
#pragma once

#include <cuda_runtime.h>

namespace nvfp4 {

enum Activation { ACT_NONE = 0, ACT_RELU = 1, ACT_RELU2 = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_SILU = 5 };
constexpr int kNumActivations = 6;

// exp(-x) overflows to infinity below x = -88, where the quotient is 0.
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }
// __fdividef(1, y) is 0 for y in (2^126, 2^128) and for infinite y: the true
// quotient is below 2^-126 there.

constexpr float kTanhScale2 = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == ACT_RELU) return fmaxf(z, 0.0f);
    if constexpr (ACT == ACT_RELU2) {
        const float r = fmaxf(z, 0.0f);
        return r * r;
    }
    if constexpr (ACT == ACT_GELU) return z * normcdff(z);
    if constexpr (ACT == ACT_GELU_TANH) return z * logistic(kTanhScale2 * z * fmaf(kTanhCubic * z, z, 1.0f));
    if constexpr (ACT == ACT_SILU) return z * logistic(z);
    return z;
}

template <int ACT>   // not for NONE and RELU2, see act_grad_value
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == ACT_GELU) return fmaf(z * 0.3989422804014327f, __expf(-0.5f * z * z), normcdff(z));
    if constexpr (ACT == ACT_GELU_TANH) {
        const float zz = z * z;
        const float s = logistic(kTanhScale2 * z * fmaf(kTanhCubic, zz, 1.0f));
        const float d = s * (1.0f - s);   // 0 far out, where the other factor may overflow
        return d == 0.0f ? s : fmaf(d, kTanhScale2 * z * fmaf(3.0f * kTanhCubic, zz, 1.0f), s);
    }
    if constexpr (ACT == ACT_SILU) {
        const float s = logistic(z);
        return fmaf(z, s * (1.0f - s), s);
    }
}

// g * slope(z); relu2's factor 2 comes last, so that nothing overflows on the
// way to a product that does not.
template <int ACT>
__device__ __forceinline__ float act_grad_value(float g, float z) {
    if constexpr (ACT == ACT_NONE) return g;
    else if constexpr (ACT == ACT_RELU2) return 2.0f * (g * fmaxf(z, 0.0f));
    else return g * act_slope<ACT>(z);
}

// The activation applied to n values; the choice is uniform over the grid, so
// it is made once per group of values and not once per value.
template <int N>
__device__ __forceinline__ void apply_act(int act, float (&v)[N]) {
    switch (act) {
        case ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<ACT_RELU>(v[i]);
            break;
        case ACT_RELU2:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<ACT_RELU2>(v[i]);
            break;
        case ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<ACT_GELU>(v[i]);
            break;
        case ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<ACT_GELU_TANH>(v[i]);
            break;
        case ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = act_value<ACT_SILU>(v[i]);
            break;
        default: break;
    }
}

}  // namespace nvfp4
