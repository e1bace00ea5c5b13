// Tile engine of the 16-bit grouped products (b16_gemm.hip, b16_wgrad.hip): C[p, q] = sum_k P[p, k] Q[q, k]
// on v_mfma_f32_16x16x32 with bf16 or fp16 operands and fp32 accumulators.
//
// A workgroup owns a BP x BQ tile of C and walks k in steps of 64.  Each step's operands go from global memory
// straight into one stage of an LDS ring (global_load_lds_dwordx4: no registers, S - 1 steps in flight), and
// the waves read MFMA fragments from there.  An operand lies in memory in one of two ways:
//   KMajor  k is contiguous (P[p][k]): a stage holds T rows of 64 k, 128 bytes a row, and a fragment (8
//           consecutive k of one row per lane) is one ds_read_b128;
//   TMajor  the tile's own index is contiguous (P[k][p]): a stage holds 64 k rows of T elements, and a
//           fragment is two ds_read_b64_tr_b16, each of which hands a group of 16 lanes 4 k of 16 columns
//           transposed (lane i gets column i), so no operand is ever transposed in memory or in registers.
// The DMA writes 64 consecutive 16-byte slots per wave instruction, so the bank swizzle is applied to the
// address each lane reads: slot `pos` of a row holds 16-byte piece pos ^ f(row), with f chosen below so that
// the lanes an LDS cycle serves fall into different banks.
// A step's pieces past the end of k (the last step of a K that is no multiple of 64, or an expert's last rows
// in the weight gradient) come from a 16-byte page of zeros, on both operands: a zero on one side alone would
// not silence an infinity or NaN that follows in memory on the other.
#pragma once

#include "device.h"
#include "host.h"

namespace moe {
namespace b16 {

constexpr int kStep = 64;                     // k per ring stage

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
#define MOE_LDS __attribute__((address_space(3)))

constexpr int kXcds = 8;
constexpr int kMaxExperts = 1024;                   // experts of the tables in LDS
constexpr int kPanel = 4;                           // tiles of a panel (the walks below)
constexpr int64_t kMaxWidth = 1 << 20;              // widths: tile coordinates are held as int

// BP x BQ tile, WP x WQ waves, S ring stages, WGS workgroups resident on a CU.
template <int BP_, int BQ_, int WP_, int WQ_, int S_, int WGS_>
struct Cfg {
    static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, S = S_;
    static constexpr int NW = WP * WQ, THREADS = 64 * NW;
    static constexpr int MP = BP / 16 / WP, MQ = BQ / 16 / WQ;
    static constexpr int WAVES_PER_EU = NW * WGS_ / 4;
};

// ceil(rows / size): up to 2^31 - 1 rows, whose rounded-up sum passes an int.
__host__ __device__ __forceinline__ int pieces(int rows, int size) { return (int)(((unsigned)rows + (unsigned)size - 1) / (unsigned)size); }

static __device__ const uint4 kZeroPiece = {0u, 0u, 0u, 0u};

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(const MOE_LDS char*)p;
}

// 64 lanes x 16 bytes from each lane's src to the LDS bytes [dst, dst + 1024) in lane order.  The instruction
// writes no register, so nothing the compiler allocates can be overwritten by it; its completion is waited for
// with wait_loads before the barrier that publishes the stage.  m0 holds the LDS address, and the compiler is told so:
// it keeps nothing of its own there; the s_nop is the wait state between an m0 write and an LDS-direct load.
__device__ __forceinline__ void dma16(const void* src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst) : "memory", "m0");
}

// Waits until at most N of this wave's vector memory operations are in flight (they retire in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A workgroup barrier that leaves vector memory operations in flight; LDS accesses before it are complete.
__device__ __forceinline__ void block_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A copy of v that the compiler takes for a new value: what is computed from it (a tile's addresses) is not
// hoisted out of the tile loop, where it would hold registers through the k loop.
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

template <bool F16>
__device__ __forceinline__ v4f mfma16x16x32(v8s a, v8s b, v4f c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Exclusive scans of a and b (one word of each per thread) over a block of NW waves; sums: 2 NW words of LDS.
template <int NW>
__device__ __forceinline__ void block_exclusive_scan2(uint32_t& a, uint32_t& b, uint32_t* sums, int lane, int wave) {
    uint32_t x = a, y = b;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const uint32_t u = __shfl_up(x, d, kWave), v = __shfl_up(y, d, kWave);
        if (lane >= d) {
            x += u;
            y += v;
        }
    }
    if (lane == kWave - 1) {
        sums[wave] = x;
        sums[NW + wave] = y;
    }
    __syncthreads();
    a = x - a;
    b = y - b;
#pragma unroll
    for (int w = 0; w < NW; w++) {
        a += w < wave ? sums[w] : 0;
        b += w < wave ? sums[NW + w] : 0;
    }
}

// The largest i < n with value(i) <= k, for a non-decreasing table of at most 1024 entries with value(0) <= k: two
// reads of the table by the whole wave, where a binary search would take ten in a row.
template <class F>
__device__ __forceinline__ int last_at_most(const F& value, int n, int k, int lane) {
    const int i = lane * 16;
    const uint64_t blocks = __ballot(i < n && value(i < n ? i : 0) <= k);
    const int b = __popcll(blocks) - 1;
    const int j = b * 16 + (lane & 15);
    const uint64_t in = __ballot(j < n && value(j < n ? j : 0) <= k) & 0xFFFFu;
    return __builtin_amdgcn_readfirstlane(b * 16 + __popcll(in) - 1);
}

// T rows of an operand whose k is contiguous, staged by NW waves.  Row r's 16-byte piece c sits at slot
// c ^ ((r >> 1) & 7): 16 consecutive rows of one piece cover 256 bytes, all 64 banks.
template <int T, int NW>
struct KMajor {
    static constexpr int BYTES = T * kStep * 2;
    static constexpr int GROUPS = T / 8;                                    // 8-row groups, one DMA each
    static constexpr int LOADS = GROUPS / NW;                               // per wave and step
    static_assert(GROUPS % NW == 0, "waves cover the rows evenly");
    const char* p[LOADS];
    int k0;                                                                 // first k of this lane's pieces

    __device__ __forceinline__ static int group(int j, int wave) { return j * NW + wave; }

    // Rows base + r * stride (bytes); rows from `valid` on repeat the last one (their results are dropped).
    __device__ __forceinline__ void set(const void* base, int64_t stride, int valid, int wave, int lane) {
#pragma unroll
        for (int j = 0; j < LOADS; j++) {
            const int r = group(j, wave) * 8 + lane / 8;
            const int c = (lane % 8) ^ ((r >> 1) & 7);                      // the same for every j
            p[j] = (const char*)base + (int64_t)(r < valid ? r : valid - 1) * stride + c * 16;
            k0 = c * 8;
        }
    }
    // Load j of step kt of a reduction over klen, into the stage at LDS byte dst.
    __device__ __forceinline__ void issue(int j, uint32_t dst, int kt, int64_t klen, int wave, int lane) const {
        const bool in = k0 < klen - (int64_t)kt * kStep;
        const char* src = p[j] + (int64_t)kt * (kStep * 2);
        dma16(in ? src : (const char*)&kZeroPiece, dst + group(j, wave) * 1024);
    }

    // This lane's fragment addresses in a stage: sub-tile m of 16 rows from row 16 * sub0, k half ks.
    struct Frag {
        uint32_t a0, a1;
        __device__ __forceinline__ void set(int sub0, int lane) {
            const int r = lane & 15;
            a0 = (uint32_t)(sub0 * 2048 + r * 128 + (((lane >> 4) ^ (r >> 1)) << 4));
            a1 = a0 ^ 64;
        }
        __device__ __forceinline__ v8s read(uint32_t stage, int m, int ks) const {
            return *(const MOE_LDS v8s*)(uintptr_t)(stage + (ks ? a1 : a0) + m * 2048);
        }
    };
};

// 64 k rows of T elements of an operand whose own index is contiguous.  Row k's 32-byte column pair c sits at
// c ^ g(k), g(k) = (k & 3) | ((k >> 3) & 1) << 2: the eight rows that two groups of 16 lanes read for one
// sub-tile (8q .. 8q+3 and 8(q+1) .. 8(q+1)+3) fall into the eight 32-byte parts of 256 bytes.  (T = 64: a row is
// 128 bytes, so k's lowest bit chooses the half already and g(k) = ((k >> 1) & 1) | ((k >> 3) & 1) << 1.)
template <int T, int NW>
struct TMajor {
    static constexpr int BYTES = T * kStep * 2;
    static constexpr int PIECES = T / 8;                                    // 16-byte pieces of a row
    static constexpr int ROWS = 64 / PIECES;                                // rows of one DMA
    static constexpr int LOADS = kStep / (ROWS * NW);
    static_assert((T % 128 == 0 || T == 64) && LOADS * ROWS * NW == kStep, "whole swizzle groups");
    const char* p[LOADS];
    int64_t stride;

    __device__ __forceinline__ static int row(int j, int wave, int lane) { return (j * NW + wave) * ROWS + lane / PIECES; }
    __device__ __forceinline__ static int swizzle(int k) {
        return T == 64 ? ((k >> 1) & 1) | (((k >> 3) & 1) << 1) : (k & 3) | (((k >> 3) & 1) << 2);
    }

    // k rows base + k * stride (bytes); column pieces from `valid` elements on repeat the last one.
    __device__ __forceinline__ void set(const void* base, int64_t stride_bytes, int valid, int wave, int lane) {
        stride = stride_bytes;
#pragma unroll
        for (int j = 0; j < LOADS; j++) {
            const int k = row(j, wave, lane);
            const int c = (lane % PIECES) ^ (swizzle(k) << 1);
            const int last = valid / 8 - 1;
            p[j] = (const char*)base + k * stride + (c < last ? c : last) * 16;
        }
    }
    __device__ __forceinline__ void issue(int j, uint32_t dst, int kt, int64_t klen, int wave, int lane) const {
        const bool in = row(j, wave, lane) < klen - (int64_t)kt * kStep;
        const char* src = p[j] + (int64_t)kt * kStep * stride;
        dma16(in ? src : (const char*)&kZeroPiece, dst + (j * NW + wave) * 1024);
    }

    struct Frag {
        uint32_t a;
        __device__ __forceinline__ void set(int sub0, int lane) {
            const int q = lane >> 4, r = (lane >> 2) & 3;
            a = (uint32_t)((8 * q + r) * (T * 2) + (sub0 >> 3) * 256 + (((sub0 & 7) ^ swizzle(8 * q + r)) << 5) + (lane & 3) * 8);
        }
        __device__ __forceinline__ v8s read(uint32_t stage, int m, int ks) const {
            const uint32_t at = stage + (a ^ ((m & 7) << 5)) + (m >> 3) * 256 + ks * (32 * T * 2);
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS v4s*)(uintptr_t)at);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS v4s*)(uintptr_t)(at + 4 * T * 2));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
};

// One k step of a wave's MP x MQ sub-tiles of 16 x 16.  Q is the MFMA's row operand, so lane l holds of
// sub-tile (m, n) the element p = 16m + l % 16, q = 16n + 4 (l / 16) + 0..3: four consecutive q.
template <int MP, int MQ, bool F16, class FP, class FQ>
__device__ __forceinline__ void step_mfma(v4f (&acc)[MP][MQ], const FP& fp, const FQ& fq, uint32_t p_stage,
                                          uint32_t q_stage) {
#pragma unroll
    for (int ks = 0; ks < 2; ks++) {
        v8s q[MQ];
#pragma unroll
        for (int n = 0; n < MQ; n++) q[n] = fq.read(q_stage, n, ks);
#pragma unroll
        for (int m = 0; m < MP; m++) {
            const v8s p = fp.read(p_stage, m, ks);
#pragma unroll
            for (int n = 0; n < MQ; n++) acc[m][n] = mfma16x16x32<F16>(q[n], p, acc[m][n]);
        }
    }
}

// The wait and the barrier that make the next stage readable: all but the S - 2 stages after it (LPS loads each)
// have to be in.  (Stores retire in the same order, so a tile's first wait covers its predecessor's stores as well.
// Counting them out of it, with the stage's last parts requested before the stores, gained nothing once the stores
// bypass the caches' order, and its registers cost more.)
template <int S, int LPS>
__device__ __forceinline__ void arrive() {
    wait_loads<(S - 2) * LPS>();
    block_barrier();
}

// The same step as a software pipeline, for tiles whose MFMAs are the bound: 2 MP groups of MQ MFMAs, each group's P
// fragment read while the group before it is multiplied (three groups ahead measured the same).  Before its last
// group the last fragments of this stage are in registers and the workgroup meets: the next stage has landed for
// every wave, and this one is free.  That group then covers the first reads of the next stage, so no MFMA waits for
// LDS at a stage's start, and the PARTS loads of the stage that takes this one's place (`part(j)`) are spread over
// it and the groups of the next step: requested at once they fill the CU's address queue and the waves stall on it
// (dense products ran 5 % slower).  ROWS >= MP: the sub-tile rows of acc; a step may take the first MP only.
template <int MQ>
struct Frags {
    v8s p[2];
    v8s q[2][MQ];
    template <class FP, class FQ>
    __device__ __forceinline__ void first(const FP& fp, const FQ& fq, uint32_t p_stage, uint32_t q_stage) {
#pragma unroll
        for (int n = 0; n < MQ; n++) q[0][n] = fq.read(q_stage, n, 0);
        p[0] = fp.read(p_stage, 0, 0);
    }
};

// Parts a group, and so the parts that the group after the meeting requests.
template <int MP, int PARTS>
constexpr int parts_per_group = (PARTS + 2 * MP - 1) / (2 * MP);

// `late(i)` runs in the groups before the meeting (group i): what has to be in the next stage by then.
template <int MP, bool F16, int S, int PARTS, int ROWS, int MQ, class FP, class FQ, class Part, class Late>
__device__ __forceinline__ void step_pipelined(v4f (&acc)[ROWS][MQ], Frags<MQ>& f, const FP& fp, const FQ& fq,
                                               uint32_t p_stage, uint32_t q_stage, uint32_t p_next, uint32_t q_next,
                                               const Part& part, const Late& late) {
    constexpr int G = 2 * MP, PER = parts_per_group<MP, PARTS>;
    constexpr int Q1 = MP > MQ ? MP - 1 - MQ : 0;         // from this group on, one fragment of Q's second half each
    static_assert(MP >= 4 && MP >= MQ, "Q's second half is read before its first group");
#pragma unroll
    for (int i = 0; i < G; i++) {
        if (i == G - 1) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            arrive<S, PARTS>();
        }
#pragma unroll
        for (int u = 0; u < PER; u++) {
            const int j = ((i + 1) % G) * PER + u;
            if (j < PARTS) part(j);
        }
        late(i);
        if (i < G - 1) {
            if (i >= Q1 && i - Q1 < MQ) f.q[1][i - Q1] = fq.read(q_stage, i - Q1, 1);
            f.p[(i + 1) % 2] = fp.read(p_stage, (i + 1) % MP, (i + 1) / MP);
        } else {
            f.first(fp, fq, p_next, q_next);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < MQ; n++) acc[i % MP][n] = mfma16x16x32<F16>(f.q[i / MP][n], f.p[i % 2], acc[i % MP][n]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Lanes r and r + 8 of each 16 exchange halves: a holds 16 bytes of row r at one place, b 16 bytes of the same row 64
// bytes further on.  After it a holds row r % 8 and b row 8 + r % 8, lanes below 8 the first place and the others the
// second, so each of two stores writes 128 bytes (a whole cache line) of eight rows instead of half lines of sixteen.
__device__ __forceinline__ void line_exchange(v4i& a, v4i& b, bool low) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int give = low ? b[i] : a[i];
        const int got = __builtin_amdgcn_update_dpp(give, give, 0x128, 0xF, 0xF, false);     // row_ror:8
        a[i] = low ? a[i] : got;
        b[i] = low ? got : b[i];
    }
}

// A wave's sub-tiles to out[p][q] (row stride in elements; `out` at the wave's element (0, 0)), rows below
// `rows`, columns below `cols` (a multiple of 8); ADD: onto what is there, in fp32 before the rounding.  A 2-byte
// type's sub-tiles n and n + 1 are first joined: a permlane32 and a permlane16 swap of the packed words hand lane
// 16q + r the eight columns 8q .. 8q+7 of row r.  Two such pieces (or two fp32 sub-tiles) then leave as whole lines
// (line_exchange), past the caches' usual order: kept as ordinary dirty lines they pushed the operands out of L2
// and were written back only when the next tile's loads needed their place.  The moves run in every lane, outside
// the bounds.
template <int DT, bool ADD, int MP, int MQ>
__device__ __forceinline__ void store_wave(void* out, int64_t stride, int rows, int cols, const v4f (&acc)[MP][MQ],
                                           int lane) {
    constexpr int ESZ = DT == kF32 ? 4 : 2;
    constexpr int JOIN = DT == kF32 ? 1 : 2;             // sub-tiles of a 16-byte piece per lane
    const bool vec = stride % (16 / ESZ) == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    const int r0 = lane & 15, q4 = 4 * (lane >> 4);
    const bool low = r0 < 8;
    char* row = (char*)out + r0 * (stride * ESZ);
    const int64_t step = 16 * stride * ESZ;
#pragma unroll
    for (int m = 0; m < MP; m++) {
        if (m * 16 >= rows) break;                                           // wave-uniform
        asm volatile("" ::: "memory");         // row by row: the accumulators leave few registers for addresses
        const bool in = m * 16 + r0 < rows;
        if constexpr (MQ % (2 * JOIN) == 0 && !ADD) {
            if (vec) {
                char* line = row - (low ? 0 : 8 * stride * ESZ);             // row r % 8 of the sixteen
                const bool in_a = m * 16 + (r0 & 7) < rows, in_b = m * 16 + 8 + (r0 & 7) < rows;
#pragma unroll
                for (int n = 0; n < MQ; n += 2 * JOIN) {
                    v4i piece[2];
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const v4f x = acc[m][n + h * JOIN];
                        if constexpr (DT == kF32) {
                            piece[h] = __builtin_bit_cast(v4i, x);
                        } else {
                            const v4f y = acc[m][n + h * JOIN + 1];
                            const auto s0 = __builtin_amdgcn_permlane32_swap(pk16<DT>(x[0], x[1]), pk16<DT>(y[0], y[1]), false, false);
                            const auto s1 = __builtin_amdgcn_permlane32_swap(pk16<DT>(x[2], x[3]), pk16<DT>(y[2], y[3]), false, false);
                            const auto t0 = __builtin_amdgcn_permlane16_swap(s0[0], s0[1], false, false);
                            const auto t1 = __builtin_amdgcn_permlane16_swap(s1[0], s1[1], false, false);
                            piece[h] = v4i{(int)t0[0], (int)t1[0], (int)t0[1], (int)t1[1]};
                        }
                    }
                    line_exchange(piece[0], piece[1], low);
                    const int c = n * 16 + (low ? 0 : 16 * JOIN) + q4 * JOIN;
                    if (in_a && c < cols) __builtin_nontemporal_store(piece[0], reinterpret_cast<v4i*>(line + c * ESZ));
                    if (in_b && c < cols)
                        __builtin_nontemporal_store(piece[1], reinterpret_cast<v4i*>(line + 8 * stride * ESZ + c * ESZ));
                }
                row += step;
                continue;
            }
        }
#pragma unroll
        for (int n = 0; n < MQ; n++) {
            const int c = n * 16 + q4;
            if (in && c < cols) {
                v4f v = acc[m][n];
                if constexpr (ADD) {
#pragma unroll
                    for (int i = 0; i < 4; i++) v[i] += load_as_f32<DT>(row, c + i);
                }
                if (vec) {
                    if constexpr (DT == kF32) *reinterpret_cast<v4f*>(row + c * 4) = v;
                    else *reinterpret_cast<uint2*>(row + c * 2) = make_uint2(pk16<DT>(v[0], v[1]), pk16<DT>(v[2], v[3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++) store_from_f32<DT>(row, c + i, v[i]);
                }
            }
        }
        row += step;
    }
}

// The same for a run-time type; `at` is the wave's first element of out, in elements.
template <int MP, int MQ>
__device__ __forceinline__ void store_wave_dt(void* out, int out_dt, bool add, int64_t at, int64_t stride, int rows, int cols,
                                              const v4f (&acc)[MP][MQ], int lane) {
    char* p = (char*)out + at * (out_dt == MOE_F32 ? 4 : 2);
    if (out_dt == MOE_F32) add ? store_wave<kF32, true>(p, stride, rows, cols, acc, lane) : store_wave<kF32, false>(p, stride, rows, cols, acc, lane);
    else if (out_dt == MOE_BF16) add ? store_wave<kBF16, true>(p, stride, rows, cols, acc, lane) : store_wave<kBF16, false>(p, stride, rows, cols, acc, lane);
    else add ? store_wave<kF16, true>(p, stride, rows, cols, acc, lane) : store_wave<kF16, false>(p, stride, rows, cols, acc, lane);
}

}  // namespace b16
}  // namespace moe
