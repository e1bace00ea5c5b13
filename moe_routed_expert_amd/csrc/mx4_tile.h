// Tile engine of the MXFP4 x MXFP4 grouped products (mx4_gemm.hip): C[p, q] = sum_k P[p, k] Q[q, k] on
// v_mfma_scale_f32_16x16x128 with E2M1 operands, an E8M0 scale per 32 k on either side and fp32 accumulators.  The scales
// are applied inside the MFMA, so the accumulators run through the whole reduction; its sums of 128 scaled products and
// the accumulator were within 2^-23 of the sum of magnitudes, whatever the scales (checked on the device).
//
// A workgroup owns a BP x BQ tile and walks k in steps of 256 elements: 128 bytes of codes and 8 scale bytes a row.  Both
// go from global memory straight into a stage of an LDS ring (S - 1 steps in flight): codes by 16-byte pieces as in
// b16_tile.h, whose slot swizzle and waits are used here, scales by words.  A step is two MFMAs per pair of 16-row
// sub-tiles.  Lane l of an MFMA holds row l % 16 and 32 k of its own, and any four blocks of 32 may meet in one MFMA as
// long as both operands take the same ones: quarter q = l / 16 takes blocks 2q (first MFMA) and 2q + 1 (second), so its
// two scales are one 16-bit word of the row's eight and the MFMA picks the byte (op_sel) - no shift, no unpacking.
// Pieces past the end of k come from a page of zeros, and so do scale words wholly past it; the scale bytes of a word
// that straddles the end are masked to 0, since a scale byte of 255 there would make a NaN of the zeros.
#pragma once

#include "b16_tile.h"
#include "mx4.h"

namespace moe {
namespace mx4 {

using b16::arrive;
using b16::block_barrier;
using b16::fresh;
using b16::last_at_most;
using b16::lds_offset;
using b16::parts_per_group;
using b16::pieces;
using b16::wait_loads;

constexpr int kStepK = 256;                   // k per ring stage
constexpr int kRowBytes = kStepK / 2;
constexpr int kRowScales = kStepK / kGroup;

// BP x BQ tile, WP x WQ waves, S ring stages, WGS workgroups resident on a CU.
template <int BP_, int BQ_, int WP_, int WQ_, int S_, int WGS_>
struct Cfg {
    static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, S = S_;
    static constexpr int NW = WP * WQ, THREADS = 64 * NW;
    static constexpr int MP = BP / 16 / WP, MQ = BQ / 16 / WQ;
    static constexpr int WAVES_PER_EU = NW * WGS_ / 4 > 0 ? NW * WGS_ / 4 : 1;
    static constexpr int CODES = (BP + BQ) * kRowBytes;
    static constexpr int STAGE = CODES + (BP + BQ) * kRowScales;
    static constexpr int P_LOADS = BP / 8 / NW, Q_LOADS = BQ / 8 / NW;       // 16-byte DMAs of a wave and step
    static constexpr int S_GROUPS = (BP + BQ) / 32;                          // 4-byte DMAs of a step, 32 rows each
    static constexpr int S_LOADS = (S_GROUPS + NW - 1) / NW;                 // of a wave (some twice, the same words)
    static constexpr int LOADS = P_LOADS + Q_LOADS + S_LOADS;
    static_assert(BP % 32 == 0 && BQ % 32 == 0 && (BP / 8) % NW == 0 && (BQ / 8) % NW == 0, "waves cover the rows evenly");
};

// 64 lanes x 4 bytes from each lane's src to the LDS bytes [dst, dst + 256) in lane order (see b16::dma16).
__device__ __forceinline__ void dma4(const void* src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(dst) : "memory", "m0");
}

// The 8-row groups of an operand that a wave stages.  A row that does not exist (nullptr) is a row of zeros.
template <int LOADS, int NW>
struct CodeRows {
    const char* p[LOADS];
    int k0;                                                                 // first byte of this lane's pieces

    // row(r): the codes of tile row r, or nullptr.
    template <class Row>
    __device__ __forceinline__ void set(const Row& row, int wave, int lane) {
#pragma unroll
        for (int j = 0; j < LOADS; j++) {
            const int r = (j * NW + wave) * 8 + lane / 8;
            const int c = (lane % 8) ^ ((r >> 1) & 7);                      // the same for every j
            const char* at = row(r);
            p[j] = at ? at + c * 16 : nullptr;
            k0 = c * 16;
        }
    }
    // Load j of step kt of rows of `bytes` codes (0: zeros), into the operand's part of the stage at LDS byte dst.
    __device__ __forceinline__ void issue(int j, uint32_t dst, int kt, int64_t bytes, int wave) const {
        const int64_t at = (int64_t)kt * kRowBytes;
        const bool in = k0 < bytes - at && p[j] != nullptr;
        b16::dma16(in ? p[j] + at : (const char*)&b16::kZeroPiece, dst + (j * NW + wave) * 1024);
    }
};

// This lane's fragment addresses in a stage: sub-tile m of 16 rows from row 16 * sub0; MFMA ks takes piece 2q + ks.
struct CodeFrag {
    uint32_t a;
    __device__ __forceinline__ void set(int sub0, int lane) {
        const int r = lane & 15, q = lane >> 4;
        a = (uint32_t)(sub0 * 2048 + r * 128 + (((2 * q) ^ (r >> 1)) << 4));
    }
    __device__ __forceinline__ v4i read(uint32_t part, int m, int ks) const {
        return *(const MOE_LDS v4i*)(uintptr_t)(part + (a ^ (ks << 4)) + m * 2048);
    }
};

// The scales of blocks 2q and 2q + 1 of sub-tile m's row, in the low 16 bits.
struct ScaleFrag {
    uint32_t a;
    __device__ __forceinline__ void set(int sub0, int lane) { a = (uint32_t)(sub0 * 128 + (lane & 15) * 8 + (lane >> 4) * 2); }
    __device__ __forceinline__ uint32_t read(uint32_t part, int m) const {
        return *(const MOE_LDS uint16_t*)(uintptr_t)(part + a + m * 128);
    }
};

// Which of the lane's two scales lie before the end of k, `left` blocks on from the stage's first.
__device__ __forceinline__ uint32_t scale_mask(int left, int lane) {
    const int b = 2 * (lane >> 4);
    return (left > b ? 0xFFu : 0u) | (left > b + 1 ? 0xFF00u : 0u);
}

template <int KS>
__device__ __forceinline__ v4f mfma(const v4i& a, uint32_t sa, const v4i& b, uint32_t sb, const v4f& c) {
    const v8i a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, KS, (int)sa, KS, (int)sb);
}

// The parts of a stage.
template <class C>
struct StageParts {
    uint32_t p, q, sp, sq;
    __device__ __forceinline__ explicit StageParts(uint32_t at)
        : p(at), q(at + C::BP * kRowBytes), sp(at + C::CODES), sq(at + C::CODES + C::BP * kRowScales) {}
};

// One step of a wave's MP x MQ sub-tiles.  Q is the MFMA's row operand, so lane l holds of sub-tile (m, n) the element
// p = 16m + l % 16, q = 16n + 4 (l / 16) + 0..3.
template <class C>
__device__ __forceinline__ void step_plain(v4f (&acc)[C::MP][C::MQ], const CodeFrag& fp, const CodeFrag& fq, const ScaleFrag& sp,
                                           const ScaleFrag& sq, uint32_t at, uint32_t mask) {
    const StageParts<C> st(at);
    uint32_t qs[C::MQ], ps[C::MP];
#pragma unroll
    for (int n = 0; n < C::MQ; n++) qs[n] = sq.read(st.sq, n) & mask;
#pragma unroll
    for (int m = 0; m < C::MP; m++) ps[m] = sp.read(st.sp, m) & mask;
#pragma unroll
    for (int ks = 0; ks < 2; ks++) {
        v4i q[C::MQ];
#pragma unroll
        for (int n = 0; n < C::MQ; n++) q[n] = fq.read(st.q, n, ks);
#pragma unroll
        for (int m = 0; m < C::MP; m++) {
            const v4i p = fp.read(st.p, m, ks);
#pragma unroll
            for (int n = 0; n < C::MQ; n++)
                acc[m][n] = ks == 0 ? mfma<0>(q[n], qs[n], p, ps[m], acc[m][n]) : mfma<1>(q[n], qs[n], p, ps[m], acc[m][n]);
        }
    }
}

}  // namespace mx4
}  // namespace moe
