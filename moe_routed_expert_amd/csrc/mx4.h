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
// rows give the same codes.
template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
    if constexpr (ACT == 0) {
        return g;
    } else {
        float f, d;
        gate_and_slope<ACT, false>(g, f, d);
        return f * u;
    }
}

}  // namespace mx4
}  // namespace moe
