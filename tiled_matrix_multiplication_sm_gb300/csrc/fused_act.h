// Activations and their slopes, in FP32.
#pragma once

#include "fused_internal.h"

namespace tgemm {
namespace fused_act {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float ROOT_2_PI = 0.79788456080286536f;       // sqrt(2 / pi)
constexpr float INV_ROOT_2PI = 0.39894228040143268f;    // 1 / sqrt(2 pi)

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Of denormal results: 0. (__fdividef's care for large divisors costs as much as the
// rest of a sigmoid.)
__device__ __forceinline__ float inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-v)): off by 2^-21 of itself and, below zero, by 2^-24 |v| more, the rounding
// of v log2(e) (2^-18 at -64), where it is not near FP32's smallest numbers: far below
// BF16's rounding.
__device__ __forceinline__ float sigmoid(float v) { return inverse(1.0f + exp2_fast(v * -LOG2E)); }

// tanh's form of GELU is z sigmoid(2 u), without the cancellation of 1 + tanh
// for negative z.
__device__ __forceinline__ float tanh_arg(float z) { return 2.0f * ROOT_2_PI * z * fmaf(0.044715f * z, z, 1.0f); }

// Phi(z) of the normal distribution; e = exp(-z^2 / 2). For z <= 0 it is half of
// erfc(-z / sqrt 2) = half of erfcx(x) e, x = |z| / sqrt 2, and erfcx(x) = t p(t) with t =
// 1 / (1 + 0.44 x) and p of degree 7 fitted to it over 0 <= x <= 10: 1.9e-7 of the
// value at most (coefficients times a half). Evaluated, it is off by 5e-7 up to |z| = 1 and by
// the roundings of z^2 / 2 in the tail, 2^-23 of that (2e-6 at -6, 7e-6 at -12). A third of erfcf's
// instructions: 3000 x 5001 x 1537 with R and Z spent more on it than on the product.
__device__ __forceinline__ float phi(float z, float& e) {
    e = exp2_fast(z * z * (-0.5f * LOG2E));
    const float t = inverse(fmaf(0.31112698372208f, fabsf(z), 1.0f));
    float p = 0.035613206675f;
    p = fmaf(p, t, -0.138980170652f);
    p = fmaf(p, t, 0.148354368869f);
    p = fmaf(p, t, -0.010100093198f);
    p = fmaf(p, t, 0.107911232036f);
    p = fmaf(p, t, 0.108655253647f);
    p = fmaf(p, t, 0.124435826964f);
    p = fmaf(p, t, 0.124110462029f);
    const float h = p * t * e;
    return z > 0.0f ? 1.0f - h : h;
}

template <int ACT>
__device__ __forceinline__ float value(float z) {
    if constexpr (ACT == TGEMM_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
    if constexpr (ACT == TGEMM_ACT_GELU) {
        float e;
        return z * phi(z, e);
    }
    if constexpr (ACT == TGEMM_ACT_GELU_TANH) return z * sigmoid(tanh_arg(z));
    if constexpr (ACT == TGEMM_ACT_SILU) return z * sigmoid(z);
    return z;
}

// act(z) and act'(z).
template <int ACT>
__device__ __forceinline__ void value_slope(float z, float& v, float& d) {
    if constexpr (ACT == TGEMM_ACT_RELU) {
        v = value<ACT>(z);
        d = z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == TGEMM_ACT_GELU) {
        float e;
        const float s = phi(z, e);
        v = z * s;
        d = fmaf(z * INV_ROOT_2PI, e, s);
    } else if constexpr (ACT == TGEMM_ACT_GELU_TANH) {
        const float s = sigmoid(tanh_arg(z));
        v = z * s;
        // (A square past FP32's range, from |z| of 4e19 on, would be an infinity times 0: s or 1 - s
        // is 0 long before.)
        const float a = fminf(fabsf(z), 1e18f);
        d = fmaf(v * (1.0f - s), 2.0f * ROOT_2_PI * fmaf(3.0f * 0.044715f * a, a, 1.0f), s);
    } else if constexpr (ACT == TGEMM_ACT_SILU) {
        const float s = sigmoid(z);
        v = z * s;
        d = fmaf(v, 1.0f - s, s);
    } else {
        v = z;
        d = 1.0f;
    }
}

template <int N>
__device__ __forceinline__ void apply(int act, float (&v)[N]) {
#define TGEMM_EACH(ACT)                                       \
    case ACT:                                                 \
        _Pragma("unroll") for (int j = 0; j < N; ++j) v[j] = value<ACT>(v[j]); \
        break
    switch (act) {
        TGEMM_EACH(TGEMM_ACT_RELU);
        TGEMM_EACH(TGEMM_ACT_GELU);
        TGEMM_EACH(TGEMM_ACT_GELU_TANH);
        TGEMM_EACH(TGEMM_ACT_SILU);
        default: break;
    }
#undef TGEMM_EACH
}
// d *= act'(z).
template <int N>
__device__ __forceinline__ void times_slope(int act, float (&d)[N], const float (&z)[N]) {
#define TGEMM_EACH(ACT)                                       \
    case ACT:                                                 \
        _Pragma("unroll") for (int j = 0; j < N; ++j) {       \
            float v, slope;                                   \
            value_slope<ACT>(z[j], v, slope);                 \
            d[j] *= slope;                                    \
        }                                                     \
        break
    switch (act) {
        TGEMM_EACH(TGEMM_ACT_RELU);
        TGEMM_EACH(TGEMM_ACT_GELU);
        TGEMM_EACH(TGEMM_ACT_GELU_TANH);
        TGEMM_EACH(TGEMM_ACT_SILU);
        default: break;
    }
#undef TGEMM_EACH
}
// Gated: g, u become d u act'(g), d act(g).
template <int N>
__device__ __forceinline__ void gated_grad(int act, const float (&d)[N], float (&g)[N], float (&u)[N]) {
#define TGEMM_EACH(ACT)                                       \
    case ACT:                                                 \
        _Pragma("unroll") for (int j = 0; j < N; ++j) {       \
            float v, slope;                                   \
            value_slope<ACT>(g[j], v, slope);                 \
            g[j] = d[j] * u[j] * slope;                       \
            u[j] = d[j] * v;                                  \
        }                                                     \
        break
    switch (act) {
        TGEMM_EACH(TGEMM_ACT_RELU);
        TGEMM_EACH(TGEMM_ACT_GELU);
        TGEMM_EACH(TGEMM_ACT_GELU_TANH);
        TGEMM_EACH(TGEMM_ACT_SILU);
        default:
            TGEMM_EACH(TGEMM_ACT_NONE);
    }
#undef TGEMM_EACH
}

}  // namespace fused_act
}  // namespace tgemm
