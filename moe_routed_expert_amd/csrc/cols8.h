// Eight consecutive columns of a row per lane, as fp32: 16-byte accesses of 2-byte types (two of fp32) where the
// caller's rows allow it (VEC), else one element at a time below `valid`.  The vector stores bypass the caches' usual
// order: the activation backward of 24576 x 1024 took 43.8 us with them and 46.7 without, and a reader of its output
// right after it 34 us and 39.
#pragma once

#include "device.h"

namespace moe {

constexpr int kCols = 8;

// The eight columns as loaded, so that several rows can be asked for before the first is used.
template <int DT>
struct RawCols8 {
    uint4 w[DT == kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* __restrict__ base, int64_t off) {
        const uint4* p = reinterpret_cast<const uint4*>((const char*)base + off * (DT == kF32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (DT == kF32 ? 2 : 1); i++) w[i] = p[i];
    }
    __device__ __forceinline__ void get(float (&v)[kCols]) const {
        const uint32_t a[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
        if constexpr (DT == kF32) {
            const uint32_t b[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                v[i] = __uint_as_float(a[i]);
                v[4 + i] = __uint_as_float(b[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint16_t lo = (uint16_t)(a[i] & 0xFFFFu), hi = (uint16_t)(a[i] >> 16);
                v[2 * i] = DT == kBF16 ? bf16_to_f32(lo) : f16_to_f32(lo);
                v[2 * i + 1] = DT == kBF16 ? bf16_to_f32(hi) : f16_to_f32(hi);
            }
        }
    }
};

template <int DT, bool VEC>
__device__ __forceinline__ void load_cols(const void* __restrict__ base, int64_t off, int valid, float (&v)[kCols]) {
    if constexpr (VEC) {
        RawCols8<DT> r;
        r.load(base, off);
        r.get(v);
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
