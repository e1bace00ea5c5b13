// Eight consecutive columns of a row per lane, as fp32: 16-byte accesses of 2-byte types (two of fp32) where the
// caller's rows allow it (VEC), else one element at a time below `valid`.  The vector stores bypass the caches' usual
// order: the activation backward of 24576 x 1024 took 43.8 us with them and 46.7 without, and a reader of its output
// right after it 34 us and 39.
#pragma once

#include "device.h"

namespace moe {

constexpr int kCols = 8;

template <int DT, bool VEC>
__device__ __forceinline__ void load_cols(const void* __restrict__ base, int64_t off, int valid, float (&v)[kCols]) {
    if constexpr (VEC && DT == kF32) {
        const v4f a = *reinterpret_cast<const v4f*>((const float*)base + off);
        const v4f b = *reinterpret_cast<const v4f*>((const float*)base + off + 4);
#pragma unroll
        for (int i = 0; i < 4; i++) { v[i] = a[i]; v[4 + i] = b[i]; }
    } else if constexpr (VEC) {
        const uint4 r = *reinterpret_cast<const uint4*>((const uint16_t*)base + off);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint16_t lo = (uint16_t)(w[i] & 0xFFFFu), hi = (uint16_t)(w[i] >> 16);
            v[2 * i] = DT == kBF16 ? bf16_to_f32(lo) : f16_to_f32(lo);
            v[2 * i + 1] = DT == kBF16 ? bf16_to_f32(hi) : f16_to_f32(hi);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kCols; i++) v[i] = i < valid ? load_as_f32<DT>(base, off + i) : 0.0f;
    }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store_cols(void* __restrict__ base, int64_t off, int valid, const float (&v)[kCols]) {
    if constexpr (VEC && DT == kF32) {
        __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, reinterpret_cast<v4f*>((float*)base + off));
        __builtin_nontemporal_store(v4f{v[4], v[5], v[6], v[7]}, reinterpret_cast<v4f*>((float*)base + off + 4));
    } else if constexpr (VEC) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = pk16<DT>(v[2 * i], v[2 * i + 1]);
        __builtin_nontemporal_store(v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]}, reinterpret_cast<v4i*>((uint16_t*)base + off));
    } else {
#pragma unroll
        for (int i = 0; i < kCols; i++)
            if (i < valid) store_from_f32<DT>(base, off + i, v[i]);
    }
}

}  // namespace moe
