// The gated activations and their slopes with relative accuracy over their whole range (moe_act values 1..5).
// EXACT: expf, erfcf and divisions, for fp32 results; else the hardware exp2 and reciprocal, for results of 16 bits
// or fewer.
#pragma once

#include "device.h"

namespace moe {

// 1 / (1 + e^-g): to a 16-bit result from the hardware exp2 and reciprocal, to fp32 from expf and a division.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float g) {
    if constexpr (EXACT) return 1.0f / (1.0f + expf(-g));
    else return fast_sigmoid(g);
}

// The sigmoid and its slope r (1 - r), both from t = e^-|g|: with q = 1 / (1 + t) they are q or t q, and t q^2 on either
// side of 0.  No step subtracts, so the slope keeps its relative accuracy (1 - r loses 6 % of it at g = 16 and all at 17).
template <bool EXACT>
__device__ __forceinline__ void sigmoid_and_slope(float g, float& f, float& d) {
    const float z = __builtin_fabsf(g);
    const float t = EXACT ? expf(-z) : __builtin_amdgcn_exp2f(-z * 1.44269504088896341f);
    const float q = EXACT ? 1.0f / (1.0f + t) : __builtin_amdgcn_rcpf(1.0f + t);
    f = g < 0.0f ? t * q : q;
    d = t * q * q;
}

// R(z) of Phi(-z) = e^(-z^2/2) R(z): it falls smoothly from 1/2 like 1/z and is t P(t), t = 1 / (1 + 0.345 z), with P of
// degree 8 fitted for the least relative error over 0 <= z <= 14.5, where the exponential passes 2^-126 (2.4e-8 in exact
// arithmetic, 3.5e-7 in fp32).
__device__ __forceinline__ float tail_ratio(float z) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.345f, z, 1.0f));
    float r = -0.0281518046f;
    r = __builtin_fmaf(r, t, 0.144233614f);
    r = __builtin_fmaf(r, t, -0.269153595f);
    r = __builtin_fmaf(r, t, 0.18505466f);
    r = __builtin_fmaf(r, t, -0.0362379402f);
    r = __builtin_fmaf(r, t, 0.111267723f);
    r = __builtin_fmaf(r, t, 0.117361993f);
    r = __builtin_fmaf(r, t, 0.138005242f);
    r = __builtin_fmaf(r, t, 0.137620106f);
    return r * t;
}

// The normal distribution's Phi(g) and density.  Phi(-z) = (1 + erf(-z / sqrt 2)) / 2 cancels (4 % off at z = 5, 0 from
// 6 on), so the lower tail is formed as itself.  fp32: erfcf.  16 bits: Phi(-z) = e^(-z^2/2) R(z) with the density's
// exponential.  The backward of 24576 x 1024 fp16 rows takes 42.5 us a call so, 55 with erfcf and expf, 46 to 49 with erff and
// expf.
template <bool EXACT>
__device__ __forceinline__ void normal_and_density(float g, float& p, float& density) {
    constexpr float kRootHalf = 0.70710678118654752f, kDensity0 = 0.39894228040143268f;
    if constexpr (EXACT) {
        p = 0.5f * erfcf(-g * kRootHalf);
        density = kDensity0 * expf(-0.5f * g * g);
    } else {
        const float z = __builtin_fminf(__builtin_fabsf(g), 16.0f);
        const float e = __builtin_amdgcn_exp2f(z * z * (-0.5f * 1.44269504088896341f));
        const float tail = e * tail_ratio(z);
        p = g < 0.0f ? tail : 1.0f - tail;
        density = kDensity0 * e;
    }
}

// act(g) and act'(g) (moe_act values 1..5).
template <int ACT, bool EXACT>
__device__ __forceinline__ void gate_and_slope(float g, float& f, float& d) {
    if constexpr (ACT == 1) {
        const float r = sigmoid<EXACT>(g);
        f = g * r;
        d = r + f * (1.0f - r);
    } else if constexpr (ACT == 2) {
        float p, density;
        normal_and_density<EXACT>(g, p, density);
        f = g * p;
        d = p + g * density;
    } else if constexpr (ACT == 3) {
        f = g <= 0.0f ? 0.0f : g;                // a NaN stays one, in the slope too
        d = g > 0.0f ? 1.0f : f;
    } else if constexpr (ACT == 4) {
        sigmoid_and_slope<EXACT>(g, f, d);
    } else {
        f = g;
        d = 1.0f;
    }
}

}  // namespace moe
