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
    static constexpr int PER = (LOADS + 2 * MP - 3) / (2 * MP - 2) > 1 ? 2 : 1;   // loads of a group of the pipelined step
    static_assert(NW % 2 == 0 && BP % 32 == 0 && BQ % 32 == 0 && (BP / 8) % NW == 0 && (BQ / 8) % NW == 0, "waves cover the rows evenly");
};

// Piece c (16 bytes, one block of 32) of tile row r lies in slot slot_of(c) ^ ((r >> 1) & 7) of the row's eight: the lanes
// that one LDS cycle serves (eight rows of one quarter of the wave, eight other rows of the next) fall into different banks.
__device__ __forceinline__ int slot_of(int c) { return (c >> 1) | ((c & 1) << 2); }
__device__ __forceinline__ int piece_in(int slot) { return ((slot & 3) << 1) | (slot >> 2); }

// The loads into LDS, 64 lanes of 16 or 4 bytes in lane order, written in asm as b16::dma16 is: the compiler would wait for
// all of them before any LDS read.
//   dma16 / dma4  from an address of each lane's own: operands of any extent.
//   buf16 / buf4  from a buffer (base and extent in scalar registers) at a 32-bit offset of each lane's own plus a scalar one:
//                 no vector instruction per load, and an offset of kNowhere or more is out of range, which reads as zeros.
__device__ __forceinline__ void dma4(const void* src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(dst) : "memory", "m0");
}
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ v4i buffer_of(const char* base, int64_t extent) {
    const uint64_t b = (uint64_t)base;
    return v4i{(int)(uint32_t)b, (int)(uint32_t)(b >> 32), (int)extent, 0x00020000};
}
__device__ __forceinline__ void buf16(uint32_t off, const v4i& buf, uint32_t at, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds" ::"v"(off), "s"(buf), "s"(dst), "s"(at) : "memory", "m0");
}
__device__ __forceinline__ void buf4(uint32_t off, const v4i& buf, uint32_t at, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %3 offen lds" ::"v"(off), "s"(buf), "s"(dst), "s"(at) : "memory", "m0");
}

// DMA j of a wave's code loads takes tile rows 8 (j NW + wave) .. + 7, a row per 8 lanes; the byte of the row's 128 that the
// lane's slot holds is the same for every j, since NW is even.
template <int NW>
__device__ __forceinline__ int code_row(int j, int wave, int lane) { return (j * NW + wave) * 8 + lane / 8; }
__device__ __forceinline__ int code_byte(int wave, int lane) { return 16 * piece_in((lane % 8) ^ ((wave * 4 + lane / 16) & 7)); }

// This lane's fragment addresses in a stage: sub-tile m of 16 rows from row 16 * sub0; MFMA ks takes piece 2q + ks.
struct CodeFrag {
    uint32_t a;
    __device__ __forceinline__ void set(int sub0, int lane) {
        const int r = lane & 15, q = lane >> 4;
        a = (uint32_t)(sub0 * 2048 + r * 128 + ((q ^ (r >> 1)) << 4));
    }
    __device__ __forceinline__ v4i read(uint32_t part, int m, int ks) const {
        return *(const MOE_LDS v4i*)(uintptr_t)(part + (a ^ (ks << 6)) + m * 2048);
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
template <class C, bool MASKED>
__device__ __forceinline__ void step_plain(v4f (&acc)[C::MP][C::MQ], const CodeFrag& fp, const CodeFrag& fq, const ScaleFrag& sp,
                                           const ScaleFrag& sq, uint32_t at, uint32_t mask) {
    const StageParts<C> st(at);
    uint32_t qs[C::MQ], ps[C::MP];
#pragma unroll
    for (int n = 0; n < C::MQ; n++) qs[n] = sq.read(st.sq, n) & (MASKED ? mask : 0xFFFFu);
#pragma unroll
    for (int m = 0; m < C::MP; m++) ps[m] = sp.read(st.sp, m) & (MASKED ? mask : 0xFFFFu);
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

// The same step as a software pipeline (b16::step_pipelined), for tiles whose MFMAs are the bound: 2 MP groups of MQ MFMAs,
// each group's P fragment and scales read while the group before it is multiplied; the workgroup meets before the last
// group, which covers the first reads of the next stage; the loads of the stage that takes the last one's place are spread
// over the first groups, PER each.  No branch lies within a step (the producer moves on between steps) and the accumulators are
// named at its end: the compiler would sink the MFMAs past a branch, and the loads before it would go out all at once.
template <class C>
struct Frags {
    v4i p[2], q[2][C::MQ];
    uint32_t ps[C::MP], qs[C::MQ], qn[C::MQ];          // scales; qn: the next stage's
    __device__ __forceinline__ void first(const CodeFrag& fp, const CodeFrag& fq, const ScaleFrag& sp, const ScaleFrag& sq, uint32_t at) {
        const StageParts<C> st(at);
#pragma unroll
        for (int n = 0; n < C::MQ; n++) q[0][n] = fq.read(st.q, n, 0);
        p[0] = fp.read(st.p, 0, 0);
#pragma unroll
        for (int n = 0; n < C::MQ; n++) qn[n] = sq.read(st.sq, n);
        ps[0] = sp.read(st.sp, 0);
    }
};

template <class C, bool MASKED, class Part>
__device__ __forceinline__ void step_pipelined(v4f (&acc)[C::MP][C::MQ], Frags<C>& f, const CodeFrag& fp, const CodeFrag& fq,
                                               const ScaleFrag& sp, const ScaleFrag& sq, uint32_t at, uint32_t next, uint32_t mask,
                                               const Part& part) {
    constexpr int MP = C::MP, MQ = C::MQ, G = 2 * MP, PARTS = C::LOADS, PER = C::PER;
    static_assert((G - 2) * PER >= PARTS, "all loads of a step go out before the workgroup meets");
    constexpr int Q1 = MP > MQ ? MP - 1 - MQ : 0;         // from this group on, one fragment of Q's second half each
    static_assert(MP >= 4 && MP >= MQ, "Q's second half is read before its first group");
    const StageParts<C> st(at);
#pragma unroll
    for (int i = 0; i < G; i++) {
        const int m = i % MP, ks = i / MP;
        if (i == G - 1) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            arrive<C::S, PARTS>();
        }
#pragma unroll
        for (int u = 0; u < PER; u++) {
            const int j = i * PER + u;
            if (j < PARTS) part(j);
        }
        if (ks == 0) {
            if (m == 0) {
#pragma unroll
                for (int n = 0; n < MQ; n++) f.qs[n] = MASKED ? f.qn[n] & mask : f.qn[n];
            }
            if constexpr (MASKED) f.ps[m] &= mask;
        }
        if (i < G - 1) {
            if (i >= Q1 && i - Q1 < MQ) f.q[1][i - Q1] = fq.read(st.q, i - Q1, 1);
            f.p[(i + 1) % 2] = fp.read(st.p, (i + 1) % MP, (i + 1) / MP);
            if (i + 1 < MP) f.ps[i + 1] = sp.read(st.sp, i + 1);
        } else {
            f.first(fp, fq, sp, sq, next);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < MQ; n++)
            acc[m][n] = ks == 0 ? mfma<0>(f.q[0][n], f.qs[n], f.p[i % 2], f.ps[m], acc[m][n])
                                : mfma<1>(f.q[1][n], f.qs[n], f.p[i % 2], f.ps[m], acc[m][n]);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < MP; m++)
#pragma unroll
        for (int n = 0; n < MQ; n++) asm volatile("" : "+v"(acc[m][n]));
}

}  // namespace mx4
}  // namespace moe
