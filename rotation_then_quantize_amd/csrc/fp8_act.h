// fp8_act.h -- activation functions and their slopes, in fp32.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/rtq.h"

namespace rtq {
namespace fp8 {

// Sigmoid through the hardware's exp2 and reciprocal (1 ulp each); 0 and 1 at its ends.
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * z));
}

constexpr float kGeluC = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// The normal distribution's tail q = erfc(|h| / sqrt 2) / 2 = e g(|h|), e = exp(-h^2 / 2), in relative terms: 1 + erf
// cancels below zero (4% off at h = -5, no digit left at -5.5).  g(a) is smooth and falls as 1 / a: a polynomial in
// t = 1 / (1 + 0.35 a) without a constant term, fitted to a <= 14.5, where e ends, with its relative error levelled
// out (3.2e-8; 3e-7 as evaluated).  The error of e is that of its exponent's rounding, h^2 2^-23.
__device__ __forceinline__ float normal_tail(float h, float* e) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, __builtin_fabsf(h), 1.0f));
    float g = -2.915787697e-02f;
    g = __builtin_fmaf(g, t, 1.440308839e-01f);
    g = __builtin_fmaf(g, t, -2.558389306e-01f);
    g = __builtin_fmaf(g, t, 1.593196094e-01f);
    g = __builtin_fmaf(g, t, -2.321229503e-02f);
    g = __builtin_fmaf(g, t, 1.055524796e-01f);
    g = __builtin_fmaf(g, t, 1.198212951e-01f);
    g = __builtin_fmaf(g, t, 1.398635209e-01f);
    g = __builtin_fmaf(g, t, 1.396213025e-01f);
    *e = __builtin_amdgcn_exp2f(-0.72134752044448170f * h * h);
    return *e * (g * t);
}

// f(h).  GELU's tanh form is h * sigmoid(2 u), u = sqrt(2/pi) (h + 0.044715 h^3): (1 + tanh u) / 2 =
// sigmoid(2 u), without the cancellation of 1 + tanh u for negative u.
template <int kAct>
__device__ __forceinline__ float act_value(float h) {
    if constexpr (kAct == RTQ_ACT_GELU_TANH) return h * sigmoid(2.0f * kGeluC * h * (1.0f + kGeluA * h * h));
    if constexpr (kAct == RTQ_ACT_GELU) {
        float e;
        const float q = normal_tail(h, &e);
        return h * (h < 0.0f ? q : 1.0f - q);
    }
    if constexpr (kAct == RTQ_ACT_SILU) return h * sigmoid(h);
    return h;
}

// f'(h).  |h| is cut at 128, where every slope has long reached 0 or 1 in fp32, so that no product
// below meets 0 * infinity; the comparisons keep a NaN.
template <int kAct>
__device__ __forceinline__ float act_slope(float h) {
    h = h > 128.0f ? 128.0f : (h < -128.0f ? -128.0f : h);
    if constexpr (kAct == RTQ_ACT_GELU_TANH) {
        const float p = sigmoid(2.0f * kGeluC * h * (1.0f + kGeluA * h * h));
        return p + h * p * (1.0f - p) * (2.0f * kGeluC) * (1.0f + 3.0f * kGeluA * h * h);
    }
    if constexpr (kAct == RTQ_ACT_GELU) {
        float e;
        const float q = normal_tail(h, &e);
        return (h < 0.0f ? q : 1.0f - q) + h * 0.39894228040143268f * e;
    }
    if constexpr (kAct == RTQ_ACT_SILU) {
        const float p = sigmoid(h);
        return p * (1.0f + h * (1.0f - p));
    }
    return 1.0f;
}

}  // namespace fp8
}  // namespace rtq
