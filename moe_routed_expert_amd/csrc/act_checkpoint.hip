// Activations kept in 8 bits for the backward pass, and the gated activation's backward from them.
//
// moe_act_checkpoint saves rows as e4m3 codes with one scale per 1 x 128 group, as moe_act_quant does, but the
// scale is a power of two: the smallest s with amax / s <= 448.  A division by s and a product with s are then
// exact, so a value has one rounding (3 mantissa bits) and code * s is a bf16 value (from s = 2^-124 on), which the
// weight gradient takes as an operand without a second rounding.  The cost is at most one bit of range at a group's
// small end.
// The gated forms save [gate | up] of the gate/up product and write h = act(gate) * up beside it, in one pass.
// moe_gated_act_backward reads dh and the saved gate and up, and forms d gate = dh up act'(gate),
// d up = dh act(gate) and, for the down projection's weight gradient, h again, so the forward keeps no h.
//
// MI355X design: HBM-bound elementwise passes, one wave per (row, 512 columns); a lane owns 8 consecutive
// columns (16-byte loads and stores of 16-bit types, 8 bytes of codes), 16 lanes share a 128-column group and
// its maximum, taken over the bits of |v| with DPP moves: as integers they order like the values, with
// infinities and NaN on top, so a group that holds one keeps it (the NaN code) instead of losing it.
#include "cols8.h"
#include "gates.h"
#include "host.h"

namespace moe {
namespace {

constexpr int kWaveCols = kWave * kCols;        // 8 columns a lane: 512, 4 groups
constexpr int kWavesPerBlock = 4;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}

// Codes (two words) and scale of this lane's 8 columns; the 16 lanes of a row of lanes share a group.
// amax = m 2^e with m in [1, 2) and 448 = 1.75 * 2^8, so s = 2^(e - 8), or 2^(e - 7) for m > 1.75; not below
// 2^-126, so that 1 / s is a normal number (amax below 2^-118 then has fewer bits, or code 0).
__device__ __forceinline__ void quant_pow2(const float (&v)[kCols], uint2& code, float& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kCols; i++) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        top = top > b ? top : b;
    }
    top = dpp_max<0xB1>(top);                   // lanes 1 apart, 2 apart, then mirrored halves and rows
    top = dpp_max<0x4E>(top);
    top = dpp_max<0x141>(top);
    top = dpp_max<0x140>(top);
    int e = (int)(top >> 23) - ((top & 0x7FFFFFu) > 0x600000u ? 7 : 8);     // exponent of s, biased by 127
    e = e < 1 ? 1 : e;
    scale = top == 0 ? 0.0f : __uint_as_float((uint32_t)e << 23);
    const float inv = top == 0 ? 0.0f : __uint_as_float((uint32_t)(254 - e) << 23);
    float q[kCols];
#pragma unroll
    for (int i = 0; i < kCols; i++) q[i] = v[i] * inv;                      // exact, or far below the least code
    // |q| <= 448 needs no clamp; an infinity or NaN becomes the NaN code
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    code = top == 0 ? make_uint2(0u, 0u) : make_uint2((uint32_t)lo, (uint32_t)hi);
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* __restrict__ p, int valid, uint2 c) {
    if constexpr (VEC) {
        *reinterpret_cast<uint2*>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < kCols; i++)
            if (i < valid) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

template <bool VEC>
__device__ __forceinline__ void load_codes(const uint8_t* __restrict__ p, int valid, float s, float (&v)[kCols]) {
    uint2 c = make_uint2(0u, 0u);
    if constexpr (VEC) {
        c = *reinterpret_cast<const uint2*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < kCols; i++) {
            const uint32_t b = i < valid ? p[i] : 0u;
            if (i < 4) c.x |= b << (8 * i);
            else c.y |= b << (8 * (i - 4));
        }
    }
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
    const v2f d = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), f = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
    v[0] = a[0] * s; v[1] = a[1] * s; v[2] = b[0] * s; v[3] = b[1] * s;
    v[4] = d[0] * s; v[5] = d[1] * s; v[6] = f[0] * s; v[7] = f[1] * s;
}

struct SaveArgs {
    const void* in;
    int64_t in_stride, rows, n;
    uint8_t* q;
    int64_t q_stride;
    float* s;
    int64_t s_stride;
    void* h;
    int64_t h_stride;
};

// grid: (512-column segments, rows / waves per block); a wave takes rows blockIdx.y * 4 + wave, then on in strides.
template <int DT, int ACT, bool VEC>
__global__ void __launch_bounds__(64 * kWavesPerBlock) act_checkpoint_kernel(const SaveArgs a) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWaveCols + lane * kCols;
    const int valid = (int)(a.n - c < 0 ? 0 : (a.n - c < kCols ? a.n - c : kCols));
    const int64_t groups = ceil_div(a.n, 128);
    for (int64_t r = (int64_t)blockIdx.y * kWavesPerBlock + wave; r < a.rows; r += (int64_t)gridDim.y * kWavesPerBlock) {
        float v[kCols] = {}, u[kCols] = {};
        if (valid > 0) {
            load_cols<DT, VEC>(a.in, r * a.in_stride + c, valid, v);
            if constexpr (ACT != 0) load_cols<DT, VEC>(a.in, r * a.in_stride + a.n + c, valid, u);
        }
        uint2 code;
        float s;
        quant_pow2(v, code, s);                          // every lane takes part in the group's maximum
        if (valid > 0) {
            store_codes<VEC>(a.q + r * a.q_stride + c, valid, code);
            if ((lane & 15) == 0) a.s[r * a.s_stride + c / 128] = s;
        }
        if constexpr (ACT != 0) {
            quant_pow2(u, code, s);
            if (valid > 0) {
                store_codes<VEC>(a.q + r * a.q_stride + a.n + c, valid, code);
                if ((lane & 15) == 0) a.s[r * a.s_stride + groups + c / 128] = s;
                if (a.h) {
                    float h[kCols];
#pragma unroll
                    for (int i = 0; i < kCols; i++) {
                        float f, d;
                        gate_and_slope<ACT, DT == kF32>(v[i], f, d);
                        h[i] = f * u[i];
                    }
                    store_cols<DT, VEC>(a.h, r * a.h_stride + c, valid, h);
                }
            }
        }
    }
}

struct UseArgs {
    const void* dh;
    int64_t dh_stride, rows, n;
    const uint8_t* q;
    int64_t q_stride;
    const float* s;
    int64_t s_stride;
    void* dx;
    int64_t dx_stride;
    void* h;
    int64_t h_stride;
};

template <int DT, int ACT, bool VEC>
__global__ void __launch_bounds__(64 * kWavesPerBlock) gated_act_backward_kernel(const UseArgs a) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWaveCols + lane * kCols;
    if (c >= a.n) return;
    const int valid = (int)(a.n - c < kCols ? a.n - c : kCols);
    const int64_t groups = ceil_div(a.n, 128);
    for (int64_t r = (int64_t)blockIdx.y * kWavesPerBlock + wave; r < a.rows; r += (int64_t)gridDim.y * kWavesPerBlock) {
        float dh[kCols], g[kCols], u[kCols];
        load_cols<DT, VEC>(a.dh, r * a.dh_stride + c, valid, dh);
        const float* s = a.s + r * a.s_stride + c / 128;
        load_codes<VEC>(a.q + r * a.q_stride + c, valid, s[0], g);
        load_codes<VEC>(a.q + r * a.q_stride + a.n + c, valid, s[groups], u);
        float dg[kCols], du[kCols], h[kCols];
#pragma unroll
        for (int i = 0; i < kCols; i++) {
            float f, d;
            gate_and_slope<ACT, DT == kF32>(g[i], f, d);
            dg[i] = dh[i] * u[i] * d;
            du[i] = dh[i] * f;
            h[i] = f * u[i];
        }
        store_cols<DT, VEC>(a.dx, r * a.dx_stride + c, valid, dg);
        store_cols<DT, VEC>(a.dx, r * a.dx_stride + a.n + c, valid, du);
        if (a.h) store_cols<DT, VEC>(a.h, r * a.h_stride + c, valid, h);
    }
}

template <int DT, int ACT>
void launch_save_act(hipStream_t st, dim3 grid, bool vec, const SaveArgs& a) {
    const dim3 block(64 * kWavesPerBlock);
    if (vec) hipLaunchKernelGGL((act_checkpoint_kernel<DT, ACT, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((act_checkpoint_kernel<DT, ACT, false>), grid, block, 0, st, a);
}

template <int DT, int ACT>
void launch_use_act(hipStream_t st, dim3 grid, bool vec, const UseArgs& a) {
    const dim3 block(64 * kWavesPerBlock);
    if (vec) hipLaunchKernelGGL((gated_act_backward_kernel<DT, ACT, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((gated_act_backward_kernel<DT, ACT, false>), grid, block, 0, st, a);
}

template <int DT>
void launch_save(hipStream_t st, dim3 grid, int act, bool vec, const SaveArgs& a) {
    switch (act) {
        case 0: return launch_save_act<DT, 0>(st, grid, vec, a);
        case 1: return launch_save_act<DT, 1>(st, grid, vec, a);
        case 2: return launch_save_act<DT, 2>(st, grid, vec, a);
        case 3: return launch_save_act<DT, 3>(st, grid, vec, a);
        case 4: return launch_save_act<DT, 4>(st, grid, vec, a);
        default: return launch_save_act<DT, 5>(st, grid, vec, a);
    }
}

template <int DT>
void launch_use(hipStream_t st, dim3 grid, int act, bool vec, const UseArgs& a) {
    switch (act) {
        case 1: return launch_use_act<DT, 1>(st, grid, vec, a);
        case 2: return launch_use_act<DT, 2>(st, grid, vec, a);
        case 3: return launch_use_act<DT, 3>(st, grid, vec, a);
        case 4: return launch_use_act<DT, 4>(st, grid, vec, a);
        default: return launch_use_act<DT, 5>(st, grid, vec, a);
    }
}

constexpr int64_t kMaxCols = (int64_t)1 << 30;

int64_t elem_size(int dt) { return dt == MOE_F32 ? 4 : 2; }

bool natural(const void* p, int dt) { return reinterpret_cast<uintptr_t>(p) % elem_size(dt) == 0; }

// Rows of 16-byte loads and stores: base 16-byte aligned, stride a multiple of 8 elements.
bool vec_rows(const void* p, int64_t stride) { return aligned16(p) && stride % 8 == 0; }

bool vec_codes(const uint8_t* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && stride % 8 == 0; }

dim3 rows_grid(int64_t rows, int64_t n) {
    const int64_t blocks = ceil_div(rows, kWavesPerBlock);
    return dim3((unsigned)ceil_div(n, kWaveCols), (unsigned)(blocks < 65535 ? blocks : 65535));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_act_checkpoint(const void* in, int dt, int64_t in_stride, int64_t rows, int64_t n, int act,
                                  uint8_t* out_q, int64_t q_stride, float* out_s, int64_t s_stride, void* h,
                                  int64_t h_stride, void* stream) {
    if (!dtype_ok(dt)) return MOE_ERR_DTYPE;
    if (act < MOE_ACT_IDENTITY || act > MOE_ACT_MUL) return MOE_ERR_SHAPE;
    if (rows < 0 || n < 0 || n > kMaxCols) return MOE_ERR_SHAPE;
    if (act == MOE_ACT_IDENTITY && h) return MOE_ERR_SHAPE;
    if (rows == 0 || n == 0) return MOE_OK;
    if (!in || !out_q || !out_s) return MOE_ERR_NULL;
    const int64_t both = act == MOE_ACT_IDENTITY ? 1 : 2;
    if (in_stride < both * n || q_stride < both * n || s_stride < both * ceil_div(n, 128) || (h && h_stride < n))
        return MOE_ERR_SHAPE;
    if (!natural(in, dt) || !natural(out_s, MOE_F32) || (h && !natural(h, dt))) return MOE_ERR_ALIGN;
    const bool vec = n % 8 == 0 && vec_rows(in, in_stride) && vec_codes(out_q, q_stride) && (!h || vec_rows(h, h_stride));
    const SaveArgs a{in, in_stride, rows, n, out_q, q_stride, out_s, s_stride, h, h_stride};
    const dim3 grid = rows_grid(rows, n);
    if (dt == MOE_F32) launch_save<kF32>(as_stream(stream), grid, act, vec, a);
    else if (dt == MOE_BF16) launch_save<kBF16>(as_stream(stream), grid, act, vec, a);
    else launch_save<kF16>(as_stream(stream), grid, act, vec, a);
    return launch_status();
}

extern "C" int moe_gated_act_backward(const void* dh, int dt, int64_t dh_stride, const uint8_t* q, int64_t q_stride,
                                      const float* s, int64_t s_stride, int64_t rows, int64_t n, int act, void* dx,
                                      int64_t dx_stride, void* h, int64_t h_stride, void* stream) {
    if (!dtype_ok(dt)) return MOE_ERR_DTYPE;
    if (act < MOE_ACT_SILU_MUL || act > MOE_ACT_MUL) return MOE_ERR_SHAPE;
    if (rows < 0 || n < 0 || n > kMaxCols) return MOE_ERR_SHAPE;
    if (rows == 0 || n == 0) return MOE_OK;
    if (!dh || !q || !s || !dx) return MOE_ERR_NULL;
    if (dh_stride < n || q_stride < 2 * n || s_stride < 2 * ceil_div(n, 128) || dx_stride < 2 * n || (h && h_stride < n))
        return MOE_ERR_SHAPE;
    if (!natural(dh, dt) || !natural(s, MOE_F32) || !natural(dx, dt) || (h && !natural(h, dt))) return MOE_ERR_ALIGN;
    const bool vec = n % 8 == 0 && vec_rows(dh, dh_stride) && vec_codes(q, q_stride) && vec_rows(dx, dx_stride) &&
                     (!h || vec_rows(h, h_stride));
    const UseArgs a{dh, dh_stride, rows, n, q, q_stride, s, s_stride, dx, dx_stride, h, h_stride};
    const dim3 grid = rows_grid(rows, n);
    if (dt == MOE_F32) launch_use<kF32>(as_stream(stream), grid, act, vec, a);
    else if (dt == MOE_BF16) launch_use<kBF16>(as_stream(stream), grid, act, vec, a);
    else launch_use<kF16>(as_stream(stream), grid, act, vec, a);
    return launch_status();
}
