// Rows quantised to MXFP4, optionally of a gated activation, and read back.
//
// MI355X design: HBM-bound passes.  A lane owns 8 consecutive columns (16-byte loads of 2-byte types, 4 bytes of codes), 4
// lanes share a group of 32 and its maximum (two DPP moves over the bits of |v|), and a wave covers 512 columns of a row.
// The conversions to and from E2M1 are gfx950's, two elements an instruction with the scale applied inside.  24576 x 4096 bf16
// take 48 us (5.3 TB/s; a copy reaches 4.6) and back 40 (6.4); fp32 10000 x 4096 34 and 29 (back 60 by eight columns a lane,
// whose stores fill half a line each).
#include <algorithm>

#include "cols8.h"
#include "host.h"
#include "mx4.h"

namespace moe {
namespace mx4 {
namespace {

constexpr int kWaveCols = kWave * kCols;        // 512
constexpr int kWavesPerBlock = 4;
constexpr int64_t kMaxCols = (int64_t)1 << 30;

struct QuantArgs {
    const void* in;
    int64_t in_stride, rows, n;
    uint8_t* q;
    int64_t q_stride;
    uint8_t* s;
    int64_t s_stride;
    int ceil;
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}

// Whole pieces of eight columns in rows that begin anywhere: the same wide accesses, which the memory takes at any byte; an
// element at a time is left for a row's last piece.  (23977 rows of 1924 fp16 there and back: 130 us by elements, 80 so.)
typedef uint32_t words4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t word_any __attribute__((aligned(1)));

template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* __restrict__ base, int64_t off, int valid, float (&v)[kCols]) {
    if (!VEC && valid == kCols) {
        const words4_any* p = reinterpret_cast<const words4_any*>((const char*)base + off * (DT == kF32 ? 4 : 2));
        RawCols8<DT> r;
#pragma unroll
        for (int i = 0; i < (DT == kF32 ? 2 : 1); i++) {
            const words4_any w = p[i];
            r.w[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        r.get(v);
    } else {
        load_cols<DT, VEC>(base, off, valid, v);
    }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(void* __restrict__ base, int64_t off, int valid, const float (&v)[kCols]) {
    if (!VEC && valid == kCols) {
        words4_any* p = reinterpret_cast<words4_any*>((char*)base + off * (DT == kF32 ? 4 : 2));
        if constexpr (DT == kF32) {
#pragma unroll
            for (int i = 0; i < 2; i++)
                p[i] = words4_any{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                  __float_as_uint(v[4 * i + 3])};
        } else {
            p[0] = words4_any{pk16<DT>(v[0], v[1]), pk16<DT>(v[2], v[3]), pk16<DT>(v[4], v[5]), pk16<DT>(v[6], v[7])};
        }
    } else {
        store_cols<DT, VEC>(base, off, valid, v);
    }
}

// grid: (512-column segments, rows / waves per block); a wave takes rows blockIdx.y * 4 + wave, then on in strides.
template <int DT, int ACT, bool VEC>
__global__ void __launch_bounds__(64 * kWavesPerBlock) quant_kernel(const QuantArgs a) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t c = (int64_t)blockIdx.x * kWaveCols + lane * kCols;
    const int valid = (int)(a.n - c < 0 ? 0 : (a.n - c < kCols ? a.n - c : kCols));
    for (int64_t r = (int64_t)blockIdx.y * kWavesPerBlock + wave; r < a.rows; r += (int64_t)gridDim.y * kWavesPerBlock) {
        float v[kCols] = {};
        if (valid > 0) {
            load8<DT, VEC>(a.in, r * a.in_stride + c, valid, v);
            if constexpr (ACT != 0) {
                float u[kCols];
                load8<DT, VEC>(a.in, r * a.in_stride + a.n + c, valid, u);
#pragma unroll
                for (int i = 0; i < kCols; i++) v[i] = i < valid ? gated<ACT>(v[i], u[i]) : 0.0f;
            }
        }
        uint32_t top = max_bits8(v);                     // every lane takes part in its group's maximum
        top = dpp_max<0xB1>(top);
        top = dpp_max<0x4E>(top);
        const uint32_t byte = scale_byte(top, a.ceil != 0);
        const uint32_t codes = encode8(v, byte);
        if (valid > 0) {
            uint8_t* q = a.q + r * a.q_stride + c / 2;
            if constexpr (VEC) {
                *reinterpret_cast<uint32_t*>(q) = codes;
            } else if (valid == kCols) {
                *reinterpret_cast<word_any*>(q) = codes;
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (2 * i < valid) q[i] = (uint8_t)(codes >> (8 * i));
            }
            if ((lane & 3) == 0) a.s[r * a.s_stride + c / kGroup] = (uint8_t)byte;
        }
    }
}

struct DequantArgs {
    const uint8_t* q;
    int64_t q_stride;
    const uint8_t* s;
    int64_t s_stride, rows, n;
    void* out;
    int64_t out_stride;
};

template <int DT, bool VEC>
__global__ void __launch_bounds__(64 * kWavesPerBlock) dequant_kernel(const DequantArgs a) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    if constexpr (VEC && DT == kF32) {           // whole lines a store: four columns a lane, two of such pieces
        for (int64_t r = (int64_t)blockIdx.y * kWavesPerBlock + wave; r < a.rows; r += (int64_t)gridDim.y * kWavesPerBlock) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t c = (int64_t)blockIdx.x * kWaveCols + h * (kWaveCols / 2) + lane * 4;
                if (c >= a.n) continue;
                const uint32_t w = *reinterpret_cast<const uint16_t*>(a.q + r * a.q_stride + c / 2);
                const float s = scale_value(a.s[r * a.s_stride + c / kGroup]);
                const v2f x0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), x1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
                __builtin_nontemporal_store(v4f{x0[0], x0[1], x1[0], x1[1]}, reinterpret_cast<v4f*>((float*)a.out + r * a.out_stride + c));
            }
        }
        return;
    }
    const int64_t c = (int64_t)blockIdx.x * kWaveCols + lane * kCols;
    if (c >= a.n) return;
    const int valid = (int)(a.n - c < kCols ? a.n - c : kCols);
    for (int64_t r = (int64_t)blockIdx.y * kWavesPerBlock + wave; r < a.rows; r += (int64_t)gridDim.y * kWavesPerBlock) {
        const uint8_t* q = a.q + r * a.q_stride + c / 2;
        uint32_t w = 0;
        if constexpr (VEC) {
            w = *reinterpret_cast<const uint32_t*>(q);
        } else if (valid == kCols) {
            w = *reinterpret_cast<const word_any*>(q);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (2 * i < valid) w |= (uint32_t)q[i] << (8 * i);
        }
        const float s = scale_value(a.s[r * a.s_stride + c / kGroup]);
        float v[kCols];
        const v2f x0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), x1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
        const v2f x2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), x3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
        v[0] = x0[0]; v[1] = x0[1]; v[2] = x1[0]; v[3] = x1[1];
        v[4] = x2[0]; v[5] = x2[1]; v[6] = x3[0]; v[7] = x3[1];
        store8<DT, VEC>(a.out, r * a.out_stride + c, valid, v);
    }
}

dim3 rows_grid(int64_t rows, int64_t n) {
    const int64_t blocks = ceil_div(rows, kWavesPerBlock);
    return dim3((unsigned)ceil_div(n, kWaveCols), (unsigned)std::min<int64_t>(blocks, 65535));
}

template <int DT, int ACT>
void launch_quant(hipStream_t st, bool vec, const QuantArgs& a) {
    const dim3 grid = rows_grid(a.rows, a.n), block(64 * kWavesPerBlock);
    if (vec) hipLaunchKernelGGL((quant_kernel<DT, ACT, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((quant_kernel<DT, ACT, false>), grid, block, 0, st, a);
}

template <int DT>
void launch_quant_act(hipStream_t st, int act, bool vec, const QuantArgs& a) {
    switch (act) {
        case 0: return launch_quant<DT, 0>(st, vec, a);
        case 1: return launch_quant<DT, 1>(st, vec, a);
        case 2: return launch_quant<DT, 2>(st, vec, a);
        case 3: return launch_quant<DT, 3>(st, vec, a);
        case 4: return launch_quant<DT, 4>(st, vec, a);
        default: return launch_quant<DT, 5>(st, vec, a);
    }
}

template <int DT>
void launch_dequant(hipStream_t st, bool vec, const DequantArgs& a) {
    const dim3 grid = rows_grid(a.rows, a.n), block(64 * kWavesPerBlock);
    if (vec) hipLaunchKernelGGL((dequant_kernel<DT, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((dequant_kernel<DT, false>), grid, block, 0, st, a);
}

bool natural(const void* p, int dt) { return reinterpret_cast<uintptr_t>(p) % (dt == MOE_F32 ? 4 : 2) == 0; }

bool vec_codes(const uint8_t* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 4 == 0 && stride % 4 == 0; }

}  // namespace
}  // namespace mx4
}  // namespace moe

using namespace moe;

extern "C" int moe_mx4_quant(const void* in, int dt, int64_t in_stride, int64_t rows, int64_t n, int act, int rule,
                             uint8_t* out_q, int64_t q_stride, uint8_t* out_s, int64_t s_stride, void* stream) {
    if (!dtype_ok(dt)) return MOE_ERR_DTYPE;
    if (act < MOE_ACT_IDENTITY || act > MOE_ACT_MUL || (rule != MOE_MX_FLOOR && rule != MOE_MX_CEIL)) return MOE_ERR_SHAPE;
    if (rows < 0 || n < 0 || n % 2 || n > mx4::kMaxCols) return MOE_ERR_SHAPE;
    if (rows == 0 || n == 0) return MOE_OK;
    if (!in || !out_q || !out_s) return MOE_ERR_NULL;
    const int64_t width = act == MOE_ACT_IDENTITY ? n : 2 * n;
    if (in_stride < width || q_stride < n / 2 || s_stride < ceil_div(n, mx4::kGroup)) return MOE_ERR_SHAPE;
    if (!mx4::natural(in, dt)) return MOE_ERR_ALIGN;
    const bool vec = n % 8 == 0 && aligned16(in) && in_stride % 8 == 0 && mx4::vec_codes(out_q, q_stride);
    const mx4::QuantArgs a{in, in_stride, rows, n, out_q, q_stride, out_s, s_stride, rule == MOE_MX_CEIL};
    if (dt == MOE_F32) mx4::launch_quant_act<kF32>(as_stream(stream), act, vec, a);
    else if (dt == MOE_BF16) mx4::launch_quant_act<kBF16>(as_stream(stream), act, vec, a);
    else mx4::launch_quant_act<kF16>(as_stream(stream), act, vec, a);
    return launch_status();
}

extern "C" int moe_mx4_dequant(const uint8_t* q, int64_t q_stride, const uint8_t* s, int64_t s_stride, int64_t rows,
                               int64_t n, void* out, int out_dt, int64_t out_stride, void* stream) {
    if (!dtype_ok(out_dt)) return MOE_ERR_DTYPE;
    if (rows < 0 || n < 0 || n % 2 || n > mx4::kMaxCols) return MOE_ERR_SHAPE;
    if (rows == 0 || n == 0) return MOE_OK;
    if (!q || !s || !out) return MOE_ERR_NULL;
    if (q_stride < n / 2 || s_stride < ceil_div(n, mx4::kGroup) || out_stride < n) return MOE_ERR_SHAPE;
    if (!mx4::natural(out, out_dt)) return MOE_ERR_ALIGN;
    const bool vec = n % 8 == 0 && aligned16(out) && out_stride % 8 == 0 && mx4::vec_codes(q, q_stride);
    const mx4::DequantArgs a{q, q_stride, s, s_stride, rows, n, out, out_stride};
    if (out_dt == MOE_F32) mx4::launch_dequant<kF32>(as_stream(stream), vec, a);
    else if (out_dt == MOE_BF16) mx4::launch_dequant<kBF16>(as_stream(stream), vec, a);
    else mx4::launch_dequant<kF16>(as_stream(stream), vec, a);
    return launch_status();
}
