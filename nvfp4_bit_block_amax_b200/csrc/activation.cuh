// activation.cuh -- the activations of the linear layer's epilogue and their
// derivatives, in binary32.
//
// With s(x) = 1 / (1 + exp(-x)) and P the normal distribution function:
//   silu       z s(z)            slope  s + z s (1 - s)
//   gelu       z P(z)            slope  P + z exp(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z s(2 u), u = sqrt(2/pi) (z + 0.044715 z^3), which is
//              z (1 + tanh u) / 2: one exponential instead of a tanh
//              slope  s + z s (1 - s) 2 u'
// The exponentials and the logistic use the hardware's exponential (2^-22) and
// reciprocal (2^-23).  Rounding the exponent's argument counts for more: an
// exponential of q is off by |q| 2^-22 at most, so s(x) by 2^-20 + |x| 2^-22
// relative, 2e-5 at x = -80; below x = -87 it is 0 (a subnormal).  bf16's half
// step is 4e-3, and binary32 sums of K products are no better near a z whose
// activation is that small, so no more is spent on it for binary32 outputs.
#pragma once

#include <cuda_runtime.h>

namespace nvfp4 {

enum Activation { ACT_NONE = 0, ACT_RELU = 1, ACT_RELU2 = 2, ACT_GELU = 3, ACT_GELU_TANH = 4, ACT_SILU = 5 };
constexpr int kNumActivations = 6;

// 2^x and 1/x, the hardware's approximations (2 and 1 units in the last place)
// with subnormals as zeros: one instruction each, where exp and the division
// with subnormals kept take four or five.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Maxima that leave NaN as it is (fmaxf gives the other operand): a step that
// has diverged shows in the layer's results.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max0(float x) { return max_nan(x, 0.0f); }

// exp(-x) overflows to infinity below x = -88, where the quotient is 0.
__device__ __forceinline__ float logistic(float x) { return rcp_fast(1.0f + exp2_fast(-kLog2e * x)); }

// The normal distribution function's tail, P(-x) = exp(-x^2 / 2) R(x) for x >= 0:
// R falls smoothly from 1/2 to 1 / (x sqrt(2 pi)), so with t = 1 / (1 + p x) it is
// close to a polynomial in t without a constant term.  The seven coefficients
// are a minimax fit made for this file (p chosen with them) to the smaller of
// two bounds, 1e-7 absolute in P and 5e-5 relative; it reaches 0.3 of both.  In
// binary32 P(-x) is off by at most 1.7e-7, and relative to itself by 1.6e-5 plus
// x^2 2^-23 from the rounded exponent, down to where it leaves the normal range
// at x = 13: a hundredth of bf16's half step, so a stored gelu is right far
// out too, where a fit with an absolute bound alone (five terms) was off by
// 0.4 % at 6 and 1.5 % at 9.  One exponential and one reciprocal serve
// function and density.
constexpr float kTailP = 0.2609f;
constexpr float kTail1 = 0.10401621460914612f, kTail2 = 0.10570815950632095f, kTail3 = 0.08265645802021027f,
                kTail4 = 0.14435040950775146f, kTail5 = -0.07746347039937973f, kTail6 = 0.20951735973358154f,
                kTail7 = -0.068785160779953f;
// exp(-x^2 / 2) and R(x), x = |z|.
struct Tail {
    float2 e, r;
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ Tail tail2(float2 z) {
    const float2 q = __fmul2_rn(__fmul2_rn(z, z), both(-0.5f * kLog2e));
    const float2 d = __ffma2_rn(make_float2(fabsf(z.x), fabsf(z.y)), both(kTailP), both(1.0f));
    const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    float2 r = __ffma2_rn(t, both(kTail7), both(kTail6));
    r = __ffma2_rn(t, r, both(kTail5));
    r = __ffma2_rn(t, r, both(kTail4));
    r = __ffma2_rn(t, r, both(kTail3));
    r = __ffma2_rn(t, r, both(kTail2));
    r = __ffma2_rn(t, r, both(kTail1));
    return Tail{make_float2(exp2_fast(q.x), exp2_fast(q.y)), __fmul2_rn(t, r)};
}
struct Normal {
    float cdf, pdf;
};
__device__ __forceinline__ Normal normal(float z) {
    const Tail w = tail2(both(z));
    const float tail = w.e.x * w.r.x;
    return Normal{z > 0.0f ? 1.0f - tail : tail, 0.3989422804f * w.e.x};
}

// z P(z) = max(z, 0) - |z| P(-|z|); the product takes z no further than the
// largest number, so that infinity less a tail of zero stays infinity.
__device__ __forceinline__ float gelu_value(float z, float tail) {
    return fmaf(-fabsf(fminf(z, 0x1.fffffep127f)), tail, fmaxf(z, 0.0f));
}

constexpr float kTanhScale2 = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == ACT_RELU) return max0(z);
    if constexpr (ACT == ACT_RELU2) {
        const float r = max0(z);
        return r * r;
    }
    if constexpr (ACT == ACT_GELU) {
        const Normal n = normal(-fabsf(z));
        return gelu_value(z, n.cdf);
    }
    if constexpr (ACT == ACT_GELU_TANH) return z * logistic(kTanhScale2 * z * fmaf(kTanhCubic * z, z, 1.0f));
    if constexpr (ACT == ACT_SILU) return z * logistic(z);
    return z;
}

template <int ACT>   // not for NONE and RELU2, see act_grad_value
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;   // NaN's slope is NaN
    if constexpr (ACT == ACT_GELU) {
        const Normal n = normal(z);
        return n.pdf == 0.0f ? n.cdf : fmaf(z, n.pdf, n.cdf);   // 0 far out, where z may be anything
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const float zz = z * z;
        const float s = logistic(kTanhScale2 * z * fmaf(kTanhCubic, zz, 1.0f));
        const float d = s * (1.0f - s);   // 0 far out, where the other factor may overflow
        return d == 0.0f ? s : fmaf(d, kTanhScale2 * z * fmaf(3.0f * kTanhCubic, zz, 1.0f), s);
    }
    if constexpr (ACT == ACT_SILU) {
        const float s = logistic(z), d = s * (1.0f - s);   // 0 far out, where z may be infinite
        return d == 0.0f ? s : fmaf(z, d, s);
    }
}

// g * slope(z); relu2's factor 2 comes last, so that nothing overflows on the
// way to a product that does not.
template <int ACT>
__device__ __forceinline__ float act_grad_value(float g, float z) {
    if constexpr (ACT == ACT_NONE) return g;
    else if constexpr (ACT == ACT_RELU2) return 2.0f * (g * max0(z));
    else return g * act_slope<ACT>(z);
}

// The activation of two values at once, through the two-wide multiply and add
// where the formula is made of them.
__device__ __forceinline__ float2 logistic2(float2 x_log2e_neg) {   // of -x log2(e)
    const float2 d = __fadd2_rn(make_float2(exp2_fast(x_log2e_neg.x), exp2_fast(x_log2e_neg.y)), both(1.0f));
    return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}
template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 z) {
    if constexpr (ACT == ACT_SILU) return __fmul2_rn(z, logistic2(__fmul2_rn(z, both(-kLog2e))));
    else if constexpr (ACT == ACT_GELU_TANH) {
        const float2 zz = __fmul2_rn(z, z);
        const float2 u = __ffma2_rn(zz, both(-kLog2e * kTanhScale2 * kTanhCubic), both(-kLog2e * kTanhScale2));
        return __fmul2_rn(z, logistic2(__fmul2_rn(z, u)));
    } else if constexpr (ACT == ACT_GELU) {
        const Tail w = tail2(z);
        const float2 tail = __fmul2_rn(w.r, w.e);
        return make_float2(gelu_value(z.x, tail.x), gelu_value(z.y, tail.y));
    } else return make_float2(act_value<ACT>(z.x), act_value<ACT>(z.y));
}

// act_grad_value of two values at once.
template <int ACT>
__device__ __forceinline__ float2 act_grad_value2(float2 g, float2 z) {
    if constexpr (ACT == ACT_SILU || ACT == ACT_GELU_TANH) {
        float2 x = z, dx = both(1.0f);   // s(x); slope s + z s (1 - s) x'
        if constexpr (ACT == ACT_GELU_TANH) {
            const float2 zz = __fmul2_rn(z, z);
            x = __fmul2_rn(z, __ffma2_rn(zz, both(kTanhScale2 * kTanhCubic), both(kTanhScale2)));
            dx = __ffma2_rn(zz, both(3.0f * kTanhScale2 * kTanhCubic), both(kTanhScale2));
        }
        const float2 s = logistic2(__fmul2_rn(x, both(-kLog2e)));
        const float2 d = __fmul2_rn(s, __ffma2_rn(s, both(-1.0f), both(1.0f)));   // 0 far out, where z x' may overflow
        const float2 q = __fmul2_rn(z, dx);
        return __fmul2_rn(g, make_float2(d.x == 0.0f ? s.x : fmaf(d.x, q.x, s.x), d.y == 0.0f ? s.y : fmaf(d.y, q.y, s.y)));
    } else if constexpr (ACT == ACT_GELU) {
        const Tail w = tail2(z);
        const float2 density = w.e, tail = __fmul2_rn(w.r, density);
        const float2 cdf = make_float2(z.x > 0.0f ? 1.0f - tail.x : tail.x, z.y > 0.0f ? 1.0f - tail.y : tail.y);
        const float2 q = __fmul2_rn(z, both(0.3989422804f));
        return __fmul2_rn(g, make_float2(density.x == 0.0f ? cdf.x : fmaf(density.x, q.x, cdf.x),
                                         density.y == 0.0f ? cdf.y : fmaf(density.y, q.y, cdf.y)));
    } else return make_float2(act_grad_value<ACT>(g.x, z.x), act_grad_value<ACT>(g.y, z.y));
}

}  // namespace nvfp4
