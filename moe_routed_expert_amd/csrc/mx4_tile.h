// Tile engine of the MXFP4 x MXFP4 grouped products (mx4_gemm.hip): C[p, q] = sum_k P[p, k] Q[q, k] on
// v_mfma_scale_f32_16x16x128 with E2M1 operands, an E8M0 scale per 32 k on either side and fp32 accumulators.  The scales
// are applied inside the MFMA, so the accumulators run through the whole reduction; its sums of 128 scaled products and
// the accumulator were within 2^-23 of the sum of magnitudes, whatever the scales (checked on the device).
//
// A workgroup owns a BP x BQ tile and walks k in steps of 256 elements, 128 bytes of codes a row, which go from global memory
// straight into a stage of an LDS ring by 16-byte pieces.  A step is two MFMAs per pair of 16-row sub-tiles.  Lane l of an
// MFMA holds row l % 16 and 32 k of its own, and any four blocks of 32 may meet in one MFMA as long as both operands take the
// same ones: quarter q = l / 16 takes blocks 2q (first MFMA) and 2q + 1 (second), so its two scales are one 16-bit word of the
// row's eight bytes and the MFMA picks the byte (op_sel) - no shift, no unpacking.
// Scales are loaded for a chunk of four steps at a time, 32 bytes a row: a load costs the CU's address path a cycle per line
// it touches, however little of it (with the scales of one step at a time a layer of 256 experts took 444 us instead of 405).
// From LDS a chunk goes to registers, a pair of 16-bit words each.
// Pieces past the end of k read as zeros, and so do scale words wholly past it; the scale bytes of a word that straddles the
// end are masked to 0, since a scale byte of 255 there would make a NaN of the zeros.
//
// What bounds it (8 x 2048 rows to 4096 columns of 8192, 1.1 TFLOP): the MFMAs are busy in 42 % of the cycles at 295 us
// (3.7 PFLOP/s) once the clock has come up; with operands of zeros 268, so 10 % is power.  Timed without the loads 243 (zeros):
// of it 165 the steps, 30 the change of tiles, 22 each the epilogues and the chunks of scales.  Tried and not kept: four waves
// of 128 x 128, which halve the reads of LDS but leave one wave a SIMD (398 us against 337), loads spread over all of a
// step, reads three groups ahead (the same), lines asked for ahead of their loads (8 us more).
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

using b16::kMaxExperts;
using b16::kMaxWidth;
using b16::kPanel;
using b16::kXcds;

constexpr int kStagger = 5;                   // an expert's tiles walk k in rotation from step kStagger * e (b16_gemm.hip)

constexpr int kStepK = 256;                   // k per ring stage
constexpr int kRowBytes = kStepK / 2;
constexpr int kRowScales = kStepK / kGroup;
constexpr int kChunk = 4;                     // steps whose scales are loaded at once
constexpr int kAhead = 2;                     // groups ahead of its MFMAs that a P fragment is read (step_pipelined)

// BP x BQ tile, WP x WQ waves, S ring stages, WGS workgroups resident on a CU.
template <int BP_, int BQ_, int WP_, int WQ_, int S_, int WGS_>
struct Cfg {
    static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, S = S_;
    static constexpr int NW = WP * WQ, THREADS = 64 * NW;
    static constexpr int MP = BP / 16 / WP, MQ = BQ / 16 / WQ;
    static constexpr int WAVES_PER_EU = NW * WGS_ / 4 > 0 ? NW * WGS_ / 4 : 1;
    static constexpr int CODES = (BP + BQ) * kRowBytes;
    static constexpr int CHUNK = (BP + BQ) * kChunk * kRowScales;            // bytes of a chunk of scales
    static constexpr int LDS = S * CODES + CHUNK;
    static constexpr int P_LOADS = BP / 8 / NW, Q_LOADS = BQ / 8 / NW;       // 16-byte DMAs of a wave and step, eight rows each; a chunk takes as many of 4 bytes
    static constexpr int LOADS = P_LOADS + Q_LOADS;
    // One step's code for all of a chunk: with a chunk's four written out, which takes the scales where they are, the largest
    // tile needs more than its 256 registers (385 us instead of 291 for 8 x 2048 rows to 4096 columns of 8192); the others gain
    // (128 x 256: 250 -> 236 us for 256 x 96 rows to 2 x 1024 of 4096).
    static constexpr bool ROLLED = MP > 4;
    static_assert(NW % 2 == 0 && BP % 32 == 0 && BQ % 32 == 0 && (BP / 8) % NW == 0 && (BQ / 8) % NW == 0,
                  "waves cover the rows evenly");
};

// Piece c (16 bytes, one block of 32) of tile row r lies in slot slot_of(c) ^ ((r >> 1) & 7) of the row's eight.  The slots
// of four lanes next to each other then hold one 64-byte half of the row's line (spread over both halves, the loads take the
// CU's address path twice as long), and the lanes that one LDS cycle serves (eight rows of one quarter of the wave, eight
// others of the next, pieces two apart) fall into different banks.
__device__ __forceinline__ int slot_of(int c) { return (c & 4) | ((c & 1) << 1) | ((c >> 1) & 1); }   // its own inverse

// The loads into LDS, 64 lanes of 16 or 4 bytes in lane order, written in asm as b16::dma16 is: the compiler would wait for
// all of them before any LDS read.
//   dma16 / dma4  from an address of each lane's own: operands of any extent.
//   buf16 / buf4  from a buffer (base and extent in scalar registers) at a 32-bit offset of each lane's own plus a scalar one:
//                 no vector instruction per load, and an offset of kNowhere or more is out of range, which reads as zeros.  Both
//                 offsets count in the range check, also where the scalar one alone is past the extent (checked on the device).
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
__device__ __forceinline__ int code_byte(int wave, int lane) { return 16 * slot_of((lane % 8) ^ ((wave * 4 + lane / 16) & 7)); }

// This lane's fragment addresses in a stage: sub-tile m of 16 rows from row 16 * sub0; MFMA ks takes piece 2q + ks.
struct CodeFrag {
    uint32_t a;
    __device__ __forceinline__ void set(int sub0, int lane) {
        const int r = lane & 15, q = lane >> 4;
        a = (uint32_t)(sub0 * 2048 + r * 128 + ((slot_of(2 * q) ^ (r >> 1)) << 4));
    }
    __device__ __forceinline__ v4i read(uint32_t part, int m, int ks) const {
        return *(const MOE_LDS v4i*)(uintptr_t)(part + (a ^ (ks << 5)) + m * 2048);
    }
};

// Byte of a chunk at which this lane's words of 16-row sub-tile sub0 lie: four steps' words of its row and half.
__device__ __forceinline__ uint32_t scale_lane(int sub0, int lane) {
    return (uint32_t)((sub0 * 16 + (lane & 15)) * (kChunk * kRowScales) + (lane >> 5) * (kChunk * 4));
}

// The scales of M sub-tiles' rows of a chunk, two steps a word: the lane's pairs, of blocks 2q and 2q + 1.  MFMA ks of step u
// takes byte 2 (u & 1) + ks of its word, or (ROLLED: one step's code serves all) ks of `now`.
template <int M, bool ROLLED>
struct Scales {
    uint32_t pair[2][M], now[ROLLED ? M : 1];
    __device__ __forceinline__ void take(int u) {
        const int shift = (u & 1) * 16;
        const uint32_t late = u & 2 ? ~0u : 0u;        // (by bits: a choice between the arrays would put them into memory)
#pragma unroll
        for (int m = 0; m < (ROLLED ? M : 0); m++) now[m] = ((pair[1][m] & late) | (pair[0][m] & ~late)) >> shift;
    }
    template <int U>
    __device__ __forceinline__ uint32_t word(int m) const { return ROLLED ? now[ROLLED ? m : 0] : pair[U / 2][m]; }
    __device__ __forceinline__ void read(uint32_t at, int lane) {
        const uint32_t sel = (lane >> 4) & 1 ? 0x07060302u : 0x05040100u;      // the quarter's half of either word
#pragma unroll
        for (int m = 0; m < M; m++) {
            const v4i w = *(const MOE_LDS v4i*)(uintptr_t)(at + m * 16 * kChunk * kRowScales);
            pair[0][m] = __builtin_amdgcn_perm((uint32_t)w[1], (uint32_t)w[0], sel);
            pair[1][m] = __builtin_amdgcn_perm((uint32_t)w[3], (uint32_t)w[2], sel);
        }
    }
    __device__ __forceinline__ void mask(uint32_t low, uint32_t high) {
#pragma unroll
        for (int m = 0; m < M; m++) {
            pair[0][m] &= low;
            pair[1][m] &= high;
        }
    }
};

// Which of the lane's two scales of two steps lie before the end of k, `left` blocks on from the first one's start.
__device__ __forceinline__ uint32_t scale_mask(int left, int lane) {
    const int b = 2 * (lane >> 4);
    return (left > b ? 0xFFu : 0u) | (left > b + 1 ? 0xFF00u : 0u) | (left > kRowScales + b ? 0xFF0000u : 0u) |
           (left > kRowScales + b + 1 ? 0xFF000000u : 0u);
}

template <int KS>
__device__ __forceinline__ v4f mfma(const v4i& a, uint32_t sa, const v4i& b, uint32_t sb, const v4f& c) {
    const v8i a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, KS, (int)sa, KS, (int)sb);
}

// One step of a wave's MP x MQ sub-tiles.  Q is the MFMA's row operand, so lane l holds of sub-tile (m, n) the element
// p = 16m + l % 16, q = 16n + 4 (l / 16) + 0..3.
template <class C, int U>
__device__ __forceinline__ void step_plain(v4f (&acc)[C::MP][C::MQ], const CodeFrag& fp, const CodeFrag& fq, const Scales<C::MP, C::ROLLED>& sp,
                                           const Scales<C::MQ, C::ROLLED>& sq, uint32_t at) {
    const uint32_t at_q = at + C::BP * kRowBytes;
#pragma unroll
    for (int ks = 0; ks < 2; ks++) {
        v4i q[C::MQ];
#pragma unroll
        for (int n = 0; n < C::MQ; n++) q[n] = fq.read(at_q, n, ks);
#pragma unroll
        for (int m = 0; m < C::MP; m++) {
            const v4i p = fp.read(at, m, ks);
#pragma unroll
            for (int n = 0; n < C::MQ; n++)
                acc[m][n] = ks == 0 ? mfma<2 * (U & 1)>(q[n], sq.template word<U>(n), p, sp.template word<U>(m), acc[m][n])
                                    : mfma<2 * (U & 1) + 1>(q[n], sq.template word<U>(n), p, sp.template word<U>(m), acc[m][n]);
        }
    }
}

// The same step as a software pipeline (b16::step_pipelined), for tiles whose MFMAs are the bound: 2 MP groups of MQ MFMAs,
// each group's P fragment read kAhead groups before.  Ahead of the last kAhead groups all of the stage is in registers and the
// workgroup meets: the next stage has landed for every wave and this one is free, so these groups read the first fragments of
// the next one and ask for the stage that takes this one's place (a step earlier than spread over the step to come: 250 ->
// 235 us for 256 x 96 rows, with the chunks written out).  No branch lies within a step (the producer moves on between steps)
// and the accumulators are named at its end: the compiler would sink the MFMAs past a branch, and the loads before it would go
// out all at once.
template <class C>
struct Frags {
    v4i p[4], q[2][C::MQ];
    __device__ __forceinline__ void first(const CodeFrag& fp, const CodeFrag& fq, uint32_t at) {
#pragma unroll
        for (int n = 0; n < C::MQ; n++) q[0][n] = fq.read(at + C::BP * kRowBytes, n, 0);
#pragma unroll
        for (int i = 0; i < kAhead; i++) p[i] = fp.read(at, i, 0);
    }
};

template <class C, int U, class Part>
__device__ __forceinline__ void step_pipelined(v4f (&acc)[C::MP][C::MQ], Frags<C>& f, const CodeFrag& fp, const CodeFrag& fq,
                                               const Scales<C::MP, C::ROLLED>& sp, const Scales<C::MQ, C::ROLLED>& sq, uint32_t at, uint32_t next,
                                               const Part& part) {
    constexpr int MP = C::MP, MQ = C::MQ, G = 2 * MP, PARTS = C::LOADS, MEET = G - kAhead;
    constexpr int PER = (PARTS + kAhead - 1) / kAhead;
    constexpr int Q1 = MP > MQ ? MP - 1 - MQ : 0;         // from this group on, one fragment of Q's second half each
    constexpr int Q0 = (MQ + kAhead - 1) / kAhead;        // from the meeting on, fragments of the next stage's Q each
    static_assert(MP >= 4 && MP >= MQ && kAhead < MP, "Q's second half is read before its first group");
    const uint32_t at_q = at + C::BP * kRowBytes, next_q = next + C::BP * kRowBytes;
#pragma unroll
    for (int i = 0; i < G; i++) {
        const int m = i % MP, ks = i / MP;
        if (i == MEET) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            arrive<C::S, PARTS>();
        }
#pragma unroll
        for (int u = 0; u < PER; u++) {
            const int j = (i - MEET) * PER + u;
            if (j >= 0 && j < PARTS) part(j);
        }
        if (i >= Q1 && i - Q1 < MQ) f.q[1][i - Q1] = fq.read(at_q, i - Q1, 1);
        if (i < MEET) {
            f.p[(i + kAhead) % 4] = fp.read(at, (i + kAhead) % MP, (i + kAhead) / MP);
        } else {
#pragma unroll
            for (int u = 0; u < Q0; u++) {
                const int n = (i - MEET) * Q0 + u;
                if (n < MQ) f.q[0][n] = fq.read(next_q, n, 0);
            }
            f.p[(i + kAhead) % 4] = fp.read(next, i - MEET, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < MQ; n++)
            acc[m][n] = ks == 0 ? mfma<2 * (U & 1)>(f.q[0][n], sq.template word<U>(n), f.p[i % 4], sp.template word<U>(m), acc[m][n])
                                : mfma<2 * (U & 1) + 1>(f.q[1][n], sq.template word<U>(n), f.p[i % 4], sp.template word<U>(m), acc[m][n]);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < MP; m++)
#pragma unroll
        for (int n = 0; n < MQ; n++) asm volatile("" : "+v"(acc[m][n]));
}

struct GemmArgs {
    const char* a;
    int64_t a_stride;                         // bytes, as all strides of codes and scales
    const char* a_s;
    int64_t a_s_stride;
    int64_t a_n;                              // rows of a, for the map's bounds
    const int32_t* a_rows;
    const char* w;
    int64_t w_stride_e, w_stride_n;
    const char* w_s;
    int64_t w_s_stride_e, w_s_stride_n;
    int n_experts;
    int64_t N, K;                             // fused: N = I, the act columns
    const int32_t* offsets;
    int m_rows;
    int n_tiles;
    void* out;                                // fused: codes
    int out_dt;
    int64_t out_stride;                       // elements (fused: bytes)
    uint8_t* s;                               // fused: scale bytes
    int64_t s_stride;
    int act, ceil;
};

__device__ __forceinline__ uint32_t max_lanes16_32(uint32_t v) {
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = a[0] > a[1] ? a[0] : a[1];
    const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return b[0] > b[1] ? b[0] : b[1];
}

// The fused epilogue of a wave's sub-tiles, two of gate and two of up: rows row0 + 16m + lane % 16 (below `rows`), act columns
// col0 .. col0 + 31.
template <int ACT, int MP, int MQ>
__device__ __forceinline__ void store_act(const GemmArgs& g, const v4f (&acc)[MP][MQ], int64_t row0, int rows, int64_t col0, int lane) {
    const int r = lane & 15, q = lane >> 4;
#pragma unroll
    for (int m = 0; m < MP; m++) {
        if (m * 16 >= rows) break;                                          // wave-uniform
        float h[8];
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) h[4 * n + i] = gated<ACT>(acc[m][n][i], acc[m][n + 2][i]);
        const uint32_t byte = scale_byte(max_lanes16_32(max_bits8(h)), g.ceil != 0);
        const uint32_t codes = encode8(h, byte);
        if (m * 16 + r < rows) {
            const int64_t row = row0 + m * 16 + r;
            uint8_t* out = (uint8_t*)g.out + row * g.out_stride + col0 / 2 + 2 * q;
            *reinterpret_cast<uint16_t*>(out) = (uint16_t)codes;
            *reinterpret_cast<uint16_t*>(out + 8) = (uint16_t)(codes >> 16);
            if (q == 0) g.s[row * g.s_stride + col0 / kGroup] = (uint8_t)byte;
        }
    }
}

template <int MP, int MQ>
__device__ __forceinline__ void store_act_of(const GemmArgs& g, const v4f (&acc)[MP][MQ], int64_t row0, int rows, int64_t col0, int lane) {
    switch (g.act) {
        case 1: return store_act<1>(g, acc, row0, rows, col0, lane);
        case 2: return store_act<2>(g, acc, row0, rows, col0, lane);
        case 3: return store_act<3>(g, acc, row0, rows, col0, lane);
        case 4: return store_act<4>(g, acc, row0, rows, col0, lane);
        default: return store_act<5>(g, acc, row0, rows, col0, lane);
    }
}

// A tile: rows row0 .. row0 + rows - 1 of an expert, output columns from n0.
struct Tile {
    int expert, row0, rows, n0;
};

// The tiles of a launch, COLS output columns each: numbered in panels of kPanel M tiles, M fastest, and dealt so that the
// workgroups of an XCD stand next to each other (b16_gemm.hip).  Built by the whole workgroup from the device's offsets, with
// 2 NW + 2 words of scratch LDS.
template <class C, int COLS>
struct Walk {
    const GemmArgs& g;
    const int* first_tile;                    // LDS: M tiles before expert e
    int m_tiles, tiles, G, start;

    __device__ __forceinline__ int clamped(int e) const { return min(max(g.offsets[e], 0), g.m_rows); }

    __device__ __forceinline__ Walk(const GemmArgs& args, int* table, uint32_t* scratch, int tid, int lane, int wave)
        : g(args), first_tile(table) {
        constexpr int EPT = kMaxExperts / C::THREADS;  // consecutive experts of a thread
        const int E = g.n_experts;
        uint32_t count[EPT], mine = 0, down = 0;
#pragma unroll
        for (int i = 0; i < EPT; i++) {
            const int e = tid * EPT + i;
            count[i] = 0;
            if (e < E) {
                const int lo = clamped(e), to = clamped(e + 1);
                count[i] = (uint32_t)pieces(max(to, lo) - lo, C::BP);
                down += to < lo;
            }
            mine += count[i];
        }
        uint32_t w = mine, d = down;
        b16::block_exclusive_scan2<C::NW>(w, d, scratch, lane, wave);
#pragma unroll
        for (int i = 0; i < EPT; i++) {
            const int e = tid * EPT + i;
            if (e < E) table[e] = (int)w;
            w += count[i];
        }
        if (tid == C::THREADS - 1) {
            scratch[2 * C::NW] = w;
            scratch[2 * C::NW + 1] = d + down;
        }
        __syncthreads();
        m_tiles = __builtin_amdgcn_readfirstlane((int)scratch[2 * C::NW]);
        // Experts that overlap may have more tiles than the host counted on, and share rows: nothing is computed.
        tiles = __builtin_amdgcn_readfirstlane((int)scratch[2 * C::NW + 1]) != 0 ? 0 : m_tiles * g.n_tiles;
        block_barrier();                       // the scratch words are free
        G = gridDim.x;
        start = (int)(blockIdx.x % kXcds) * (G / kXcds) + (int)(blockIdx.x / kXcds);
    }

    __device__ __forceinline__ Tile locate(int t, int lane) const {
        const int per = kPanel * g.n_tiles;
        const int panel = t / per, r = t - panel * per;
        const int height = min(kPanel, m_tiles - panel * kPanel);
        const int nt = r / height, mt = panel * kPanel + r - nt * height;
        const int e = last_at_most([&](int i) { return first_tile[i]; }, g.n_experts, mt, lane);
        Tile ti;
        ti.expert = e;
        uint32_t lo, hi;                       // (a vector load would wait for every load in flight)
        scalar_read2(g.offsets + e, g.offsets + e + 1, lo, hi);
        const int from = min(max((int)lo, 0), g.m_rows), end = min(max((int)hi, 0), g.m_rows);
        ti.row0 = from + (mt - __builtin_amdgcn_readfirstlane(first_tile[e])) * C::BP;
        ti.rows = min(end - ti.row0, C::BP);
        ti.n0 = nt * COLS;
        return ti;
    }
    // A's row of row r of a tile: rows past the tile's repeat the last one (their results are dropped); -1: a row of zeros,
    // whose map entry is no row of A.
    __device__ __forceinline__ int64_t a_row(const Tile& ti, int r) const {
        const int64_t at = ti.row0 + min(r, ti.rows - 1);
        if (!g.a_rows) return at;
        const int64_t m = g.a_rows[at];
        return m >= 0 && m < g.a_n ? m : -1;
    }
    // The bank's row of row r of a tile.  Fused: 32 gate rows, then the 32 up rows of the same columns, and so on.  Columns past
    // the last repeat it.
    template <bool FUSED>
    __device__ __forceinline__ int64_t w_row(const Tile& ti, int r) const {
        if (!FUSED) return min(ti.n0 + r, (int)g.N - 1);
        const int c = min(ti.n0 + (r >> 6) * 32 + (r & 31), (int)g.N - 1);
        return c + (r & 32 ? g.N : 0);
    }
};

// The tiles of W from `first` on in halves of C::BP rows, the second of which may have none.
template <class C, class W>
struct Halves {
    const W& whole;
    int first, start, tiles, G;

    __device__ __forceinline__ Tile locate(int t, int lane) const {
        Tile ti = whole.locate(first + t / 2, lane);
        const int past = (t & 1) * C::BP;
        ti.row0 += past;
        ti.rows = min(ti.rows - past, C::BP);
        return ti;
    }
    __device__ __forceinline__ int64_t a_row(const Tile& ti, int r) const { return whole.a_row(ti, r); }
    template <bool FUSED>
    __device__ __forceinline__ int64_t w_row(const Tile& ti, int r) const { return whole.template w_row<FUSED>(ti, r); }
};

}  // namespace mx4
}  // namespace moe
