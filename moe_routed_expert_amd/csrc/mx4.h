// MXFP4 (OCP microscaling): E2M1 elements, +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, two a byte with the even element in the low
// nibble, and one E8M0 scale byte, 2^(byte - 127) or NaN for 255, per 32 consecutive elements.
#pragma once

#include "device.h"
#include "gates.h"

namespace moe {
namespace mx4 {

constexpr int kGroup = 32;                    // elements of a scale

// The scale byte of a group whose largest magnitude has the fp32 bits `top` (|v| as integers order like the values, with
// infinities and NaN above them).  floor: 2^(floor(log2 amax) - 2), the format's own rule, under which values above
// 6 * 2^e saturate; ceil: the least power of two with amax <= 6 * 2^e, 6 = 1.5 * 2^2.  Not below 2^-127, byte 0, which
// a group of zeros takes too; an infinity or NaN makes the whole group NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top, bool ceil) {
    if (top >= 0x7F800000u) return 255u;
    const int e = (int)(top >> 23) - (ceil && (top & 0x7FFFFFu) > 0x400000u ? 1 : 2);
    return (uint32_t)(e < 0 ? 0 : e);
}

// The scale as a float: 2^-127 is a subnormal.  (The conversions below read the exponent field alone, so byte 255 needs
// no value of its own.)
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// Eight values of one group to eight codes, element i in bits 4i..4i+3: round to nearest even of v / scale, the quotient
// exact, saturating at 6 (v_cvt_scalef32_pk_fp4_f32, checked on the device at every tie, its neighbours and every scale).
// A group with scale byte 255 takes codes 0.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t byte) {
    const float s = scale_value(byte);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
    return byte == 255u ? 0u : w;
}

__device__ __forceinline__ uint32_t max_bits8(const float (&v)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        top = top > b ? top : b;
    }
    return top;
}

// act(g) * u of moe_act `ACT`, in one form whatever the type, so that the products' epilogue and the pass over stored
// rows give the same codes.  The exponentials of |g| are formed as squares and their factors multiplied one by one, so that
// every gate whose value fp32 holds comes out with it: e^-89 alone is below 2^-126, -89 e^-89 is not, and a group of such gates
// has scales of its own.  In units of 2^-24 SiLU and the sigmoid are off by 1.22 |g| (the exponent |g| log2 e's constant and
// rounding) and 13 at most (two hardware exponentials 2 each, 1 + t and its reciprocal 6, three products), GELU by 1.11 g^2 (g^2 / 2
// log2 e's two roundings and constant) and 13 (the same, with tail_ratio's 6); a gate below 2^-126 by half a step of 2^-149 more.
// (The fma's are written out: whether the compiler makes them must not depend on the kernel.)  Four instructions more than
// g / (1 + e^-g) u, which is -0 from g = -89 on: 8 x 2048 rows to 2 x 2048 columns of 2048 with their requant take 85.6 us so and
// 83.6 without the tail, of 8192 262 and 259; the pass over stored rows is HBM's either way.
template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
    constexpr float kHalfLog2e = 0.5f * 1.44269504088896341f;
    const float z = __builtin_fabsf(g);
    if constexpr (ACT == 0) {
        return g;
    } else if constexpr (ACT == 1 || ACT == 4) {         // h = e^(-z/2), sigmoid = 1 / (1 + h^2), or h^2 times that
        const float h = __builtin_amdgcn_exp2f(z * -kHalfLog2e), q = __builtin_amdgcn_rcpf(__builtin_fmaf(h, h, 1.0f));
        const float a = g < 0.0f ? h : 1.0f, aq = a * q;
        return (ACT == 1 ? (g * a) * aq : a * aq) * u;
    } else if constexpr (ACT == 2) {                     // h = e^(-z^2/4), Phi(-z) = h^2 R(z)
        const float h = __builtin_amdgcn_exp2f(z * z * (-0.5f * kHalfLog2e)), r = tail_ratio(z);
        return (g < 0.0f ? (g * h) * (h * r) : g * __builtin_fmaf(-(h * h), r, 1.0f)) * u;
    } else {
        float f, d;
        gate_and_slope<ACT, false>(g, f, d);
        return f * u;
    }
}

}  // namespace mx4
}  // namespace moe
