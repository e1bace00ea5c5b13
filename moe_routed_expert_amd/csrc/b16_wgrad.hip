// Weight gradient of the grouped products: dW[e][n][k] = sum over the rows r of expert e of dY[r][n] A[r][k].
// Both operands lie with the reduction as their slow dimension, so both are read through the transposing LDS
// loads of b16_tile.h and nothing is transposed in memory.  A may be the 8-bit checkpoint of a forward pass:
// its e4m3 codes and 1 x 128 scales are read (half the bytes), and each 16-bit operand value
// round(code * scale) is formed once per workgroup on its way into LDS.  With power-of-two scales
// (moe_act_checkpoint; from 2^-124 on) that product is exact in bf16 and no rounding is added.  (In fp16
// its top value is held in range.)
//
// Persistent workgroups walk the tiles of every expert, expert by expert, so experts of unequal length are
// shared by all of them; an expert without rows gets zeros.  Where the gradient has few tiles and many rows
// (small matrices, long sequences), the experts' rows are cut into chunks of one length, so long experts count as
// several: their fp32 partial gradients go to a workspace and are summed in a fixed order, without atomics, so
// results do not depend on timing.  Tile and cut are chosen by estimated time (wgrad_plan): the partials are written
// and read once more, so a cut pays only where the device would be far from full.
//
// Two transposing reads a fragment and both operands' loads bound it where experts have many rows (8 experts, 16384
// rows, 8192 x 4096 in fp32: 1000 us, 1.10 PFLOP/s), the gradient's stores where they have few (256 experts, 24576 rows
// from 8 bits, 2048 x 4096 in bf16: 1235 us for 4.3 GB, which a kernel of such stores alone writes in 772 us).
// A gradient that is added on is read element by element and stored by half lines: on one set of inputs the first takes
// 1000 us written and 1170 added on, the second 1040 and 3060.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "b16_tile.h"

namespace moe {
namespace b16 {


struct WgradArgs {
    const char* dy;
    int64_t dy_stride;                // bytes
    const char* a;
    int64_t a_stride;                 // bytes
    const float* a_s;                 // e4m3: scales
    int64_t a_s_stride;
    const int32_t* offsets;
    int m_rows;
    int n_experts;
    int64_t N, K;
    int n_tiles, k_tiles;
    int chunk_rows, max_chunks;       // rows of a chunk (0: an expert's rows are one), and chunks that the workspace holds
    char* out;                        // dW, or the fp32 partials [chunk][N][K]
    int out_dt;
    int64_t stride_e, stride_n;       // elements
    int accumulate;
};

// 64 rows of T e4m3 columns with a scale per row and 128 columns, staged through registers into the layout of
// TMajor: a thread's piece is 16 columns of one row (one scale), two 16-byte pieces of the stage.
template <int T, int NW, bool F16>
struct TSaved {
    static constexpr int BYTES = T * kStep * 2;
    static constexpr int PIECES = T / 16;
    static constexpr int PER = T * kStep / 16 / (64 * NW);                  // pieces of a thread
    static constexpr int LOADS = 0;                                         // none that wait_loads counts
    static_assert(PER >= 1, "every thread has a piece");
    const char* p[PER];
    const float* s[PER];
    int64_t stride, s_stride;
    uint4 code[PER];
    float scale[PER];

    __device__ __forceinline__ static int row(int j, int tid) { return (j * 64 * NW + tid) / PIECES; }

    __device__ __forceinline__ void set(const char* base, int64_t stride_bytes, const float* scales, int64_t scale_stride,
                                        int valid, int col0, int tid) {
        stride = stride_bytes;
        s_stride = scale_stride;
#pragma unroll
        for (int j = 0; j < PER; j++) {
            const int c = (j * 64 * NW + tid) % PIECES, last = valid / 16 - 1;
            const int cc = c < last ? c : last;
            p[j] = base + row(j, tid) * stride + cc * 16;
            s[j] = scales + row(j, tid) * s_stride + (col0 + cc * 16) / 128;
        }
    }
    // Requests step kt; rows past klen read as code 0, scale 0.
    __device__ __forceinline__ void load(int kt, int64_t klen, int tid) {
#pragma unroll
        for (int j = 0; j < PER; j++) {
            const bool in = row(j, tid) < klen - (int64_t)kt * kStep;
            const char* src = p[j] + (int64_t)kt * kStep * stride;
            const float* ss = s[j] + (int64_t)kt * kStep * s_stride;
            code[j] = *reinterpret_cast<const uint4*>(in ? src : (const char*)&kZeroPiece);
            scale[j] = *(in ? ss : (const float*)&kZeroPiece);
        }
    }
    // fp16's values from 63488 on are saved as 65536, which fp16 does not hold: a product past its range is held at 65504,
    // so that finite rows stay finite.  minimum and maximum keep a NaN.  (As a branch on the few scales that reach there it
    // broke up the step's schedule: 8 experts, 16384 rows, 8192 x 4096 took 1322 us, with these two instructions a pair
    // 1162, without them 1172.)
    __device__ __forceinline__ static uint32_t in_range(uint32_t pair) {
        if constexpr (!F16) return pair;
        typedef _Float16 v2h __attribute__((ext_vector_type(2)));
        const v2h top = {(_Float16)65504.0f, (_Float16)65504.0f};
        const v2h h = __builtin_elementwise_minimum(__builtin_bit_cast(v2h, pair), top);
        return __builtin_bit_cast(uint32_t, (v2h)__builtin_elementwise_maximum(h, -top));
    }
    // Piece j into the stage at dst.
    __device__ __forceinline__ void commit(int j, uint32_t dst, int tid) const {
        const int k = row(j, tid), c = (j * 64 * NW + tid) % PIECES;
        const uint32_t at = dst + k * (T * 2) + ((c ^ TMajor<T, NW>::swizzle(k)) << 5);
        const uint32_t w[4] = {code[j].x, code[j].y, code[j].z, code[j].w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
            const v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            o[2 * i] = in_range(pk16<F16 ? kF16 : kBF16>(lo[0] * scale[j], lo[1] * scale[j]));
            o[2 * i + 1] = in_range(pk16<F16 ? kF16 : kBF16>(hi[0] * scale[j], hi[1] * scale[j]));
        }
        *(MOE_LDS v4i*)(uintptr_t)at = v4i{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
        *(MOE_LDS v4i*)(uintptr_t)(at + 16) = v4i{(int)o[4], (int)o[5], (int)o[6], (int)o[7]};
    }
};

template <class C, bool SAVED, bool F16>
__global__ void __launch_bounds__(C::THREADS, C::WAVES_PER_EU) b16_wgrad_kernel(const WgradArgs g) {
    using P = TMajor<C::BP, C::NW>;
    using QD = TMajor<C::BQ, C::NW>;
    using Q = std::conditional_t<SAVED, TSaved<C::BQ, C::NW, F16>, QD>;
    constexpr int S = C::S, STAGE = P::BYTES + Q::BYTES, LPS = P::LOADS + Q::LOADS;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[S * STAGE];
    __shared__ int first_row[kMaxExperts + 1], first_chunk[kMaxExperts + 1];   // offsets, clamped to [0, m_rows]
    __shared__ uint32_t wave_sum[2 * C::NW];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int per = g.n_tiles * g.k_tiles;
    for (int e = tid; e <= g.n_experts; e += C::THREADS) first_row[e] = min(max(g.offsets[e], 0), g.m_rows);
    __syncthreads();
    // Offsets that decrease name rows twice: nothing is written, as in the products.  (Every wave looks at all of them.)
    bool decreases = false;
    for (int e = lane; e < g.n_experts; e += kWave) decreases |= first_row[e + 1] < first_row[e];
    if (__any(decreases)) return;
    int chunks = g.n_experts;
    if (g.chunk_rows > 0) {
        constexpr int EPT = kMaxExperts / C::THREADS;
        int n[EPT];
        uint32_t sum = 0;
#pragma unroll
        for (int i = 0; i < EPT; i++) {
            const int e = tid * EPT + i;
            n[i] = e < g.n_experts ? pieces(max(first_row[e + 1] - first_row[e], 0), g.chunk_rows) : 0;
            sum += n[i];
        }
        uint32_t before = sum, none = 0;
        block_exclusive_scan2<C::NW>(before, none, wave_sum, lane, wave);
#pragma unroll
        for (int i = 0; i < EPT; i++) {
            const int e = tid * EPT + i;
            if (e < g.n_experts) first_chunk[e] = (int)before;
            before += n[i];
            if (e == g.n_experts - 1) first_chunk[e + 1] = (int)before;
        }
        __syncthreads();
        chunks = min(__builtin_amdgcn_readfirstlane(first_chunk[g.n_experts]), g.max_chunks);
    }
    const int tiles = per * chunks;
    const int G = gridDim.x;
    const int start = (int)(blockIdx.x % kXcds) * (G / kXcds) + (int)(blockIdx.x / kXcds);

    struct Tile {
        int chunk, row0, rows, n0, k0;
    };
    auto locate = [&](int t) {
        Tile ti;
        ti.chunk = t / per;
        t -= ti.chunk * per;
        const int panel = t / (kPanel * g.k_tiles);
        t -= panel * kPanel * g.k_tiles;
        const int height = min(kPanel, g.n_tiles - panel * kPanel);
        const int kt = t / height;
        ti.k0 = kt * C::BQ;
        ti.n0 = (panel * kPanel + t - kt * height) * C::BP;
        int expert = ti.chunk, from = 0;
        if (g.chunk_rows > 0) {                        // the last expert whose first chunk is <= this one
            const int lo = last_at_most([&](int e) { return first_chunk[e]; }, g.n_experts, ti.chunk, lane);
            expert = lo;
            from = (ti.chunk - __builtin_amdgcn_readfirstlane(first_chunk[lo])) * g.chunk_rows;
        }
        const int lo = __builtin_amdgcn_readfirstlane(first_row[expert]) + from;
        ti.row0 = lo;
        ti.rows = max(__builtin_amdgcn_readfirstlane(first_row[expert + 1]) - lo, 0);
        if (g.chunk_rows > 0) ti.rows = min(ti.rows, g.chunk_rows);
        return ti;
    };
    // an expert without rows still takes one step, of zeros, so that its tiles are stored
    auto steps_of = [&](const Tile& ti) { return max(1, pieces(ti.rows, kStep)); };

    // Producer, as in b16_gemm_kernel: past the last tile it goes on with zeros (prod_rows = 0).
    const uint32_t lds = lds_offset(ring);
    P p;
    Q q;
    int prod_t = start, prod_kt = 0, prod_steps = 1, prod_rows = 0, prod_stage = 0;
    uint32_t saved_dst = 0;                            // SAVED: where the step that is in registers goes
    auto aim = [&]() {
        prod_rows = 0;
        if (prod_t >= tiles) return;
        const Tile ti = locate(prod_t);
        prod_steps = steps_of(ti);
        prod_rows = ti.rows;
        const int l = fresh(lane);
        p.set(g.dy + ti.row0 * g.dy_stride + (int64_t)ti.n0 * 2, g.dy_stride, (int)min(g.N - ti.n0, (int64_t)C::BP), wave, l);
        const int valid = (int)min(g.K - ti.k0, (int64_t)C::BQ);
        if constexpr (SAVED)
            q.set(g.a + ti.row0 * g.a_stride + ti.k0, g.a_stride, g.a_s + ti.row0 * g.a_s_stride, g.a_s_stride, valid, ti.k0, wave * kWave + l);
        else
            q.set(g.a + ti.row0 * g.a_stride + (int64_t)ti.k0 * 2, g.a_stride, valid, wave, l);
    };
    auto part = [&](int j) {
        const uint32_t dst = lds + prod_stage * STAGE;
        if constexpr (SAVED) {
            if (j == 0) {
                q.load(prod_kt, prod_rows, tid);
                saved_dst = dst + P::BYTES;
            }
        }
        if (j < P::LOADS) p.issue(j, dst, prod_kt, prod_rows, wave, lane);
        else if constexpr (!SAVED) q.issue(j - P::LOADS, dst + P::BYTES, prod_kt, prod_rows, wave, lane);
        if (j == LPS - 1) {
            prod_stage = prod_stage + 1 == S ? 0 : prod_stage + 1;
            if (++prod_kt == prod_steps) {
                prod_kt = 0;
                prod_t += G;
                aim();
            }
        }
    };
    // SAVED: the pieces that part 0 asked for go to LDS shortly before the stage is published
    auto late = [&](int i) {
        if constexpr (SAVED) {
#pragma unroll
            for (int j = 0; j < Q::PER; j++)
                if (i == 2 * C::MP - 2 - 2 * (Q::PER - 1 - j)) q.commit(j, saved_dst, tid);
        }
    };
    auto produce = [&]() {
#pragma unroll
        for (int j = 0; j < LPS; j++) part(j);
    };
    if (start >= tiles) return;
    aim();
#pragma unroll 1
    for (int i = 0; i < S - 1; i++) {
        produce();
        if constexpr (SAVED)
            for (int j = 0; j < Q::PER; j++) q.commit(j, saved_dst, tid);
    }

    typename P::Frag fp;
    typename QD::Frag fq;
    const int wp = wave / C::WQ, wq = wave % C::WQ;
    fp.set(wp * C::MP, lane);
    fq.set(wq * C::MQ, lane);

    int stage = 0;
    Frags<C::MQ> f;
    arrive<S, LPS>();
    f.first(fp, fq, lds, lds + P::BYTES);
#pragma unroll
    for (int j = 0; j < parts_per_group<C::MP, LPS>; j++) part(j);
#pragma unroll 1
    for (int t = start; t < tiles; t += G) {
        const Tile ti = locate(t);
        const int steps = steps_of(ti);
        v4f acc[C::MP][C::MQ];
#pragma unroll
        for (int m = 0; m < C::MP; m++)
#pragma unroll
            for (int n = 0; n < C::MQ; n++) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int kt = 0; kt < steps; kt++) {
            const uint32_t at = lds + stage * STAGE;
            stage = stage + 1 == S ? 0 : stage + 1;
            const uint32_t next = lds + stage * STAGE;
            step_pipelined<C::MP, F16, S, LPS>(acc, f, fp, fq, at, at + P::BYTES, next, next + P::BYTES, part, late);
        }
        const int rows = (int)min(g.N - ti.n0, (int64_t)C::BP) - wp * C::MP * 16;
        const int64_t c0 = ti.k0 + wq * C::MQ * 16;
        const int cols = (int)min(g.K - c0, (int64_t)(C::MQ * 16));
        if (rows > 0 && cols > 0) {
            const int64_t o = ti.chunk * g.stride_e + (int64_t)(ti.n0 + wp * C::MP * 16) * g.stride_n + c0;
            store_wave_dt(g.out, g.out_dt, g.accumulate != 0, o, g.stride_n, rows, cols, acc, fresh(lane));
        }
    }
    wait_loads<0>();                                   // no load may write LDS after the workgroup has left it
}

// The chunks' partial gradients, [chunk][n][k] in fp32, summed for each expert (onto what is there, when accumulating)
// and rounded once.  Four consecutive k a thread, an expert per blockIdx.y; its chunks are counted again from the
// offsets.  Eight chunks are asked for at once: one by one each cost a trip to memory (a
// gradient of 64 x 128 over 391 chunks took 179 us, and 24 now).  A gradient of few elements is shared further: its SPLIT waves take an equal run of chunks each, and wave 0
// adds their sums in order.  The order depends on the counts alone.
constexpr int kJoinSplit = 16;

template <int DT, int SPLIT>
__global__ void __launch_bounds__(SPLIT == 1 ? 256 : 64 * SPLIT)
wgrad_join_kernel(const float* __restrict__ part, const int32_t* __restrict__ offsets, int m_rows, int chunk_rows,
                  int max_chunks, int64_t N, int64_t K, void* __restrict__ out, int64_t stride_e, int64_t stride_n,
                  int accumulate) {
    constexpr int THREADS = SPLIT == 1 ? 256 : 64 * SPLIT, OWN = THREADS / SPLIT;      // elements (of four) a workgroup
    __shared__ int wave_sum[THREADS / kWave], wave_decreases[THREADS / kWave];
    __shared__ v4f others[SPLIT == 1 ? 1 : SPLIT][SPLIT == 1 ? 1 : OWN];
    const int e = blockIdx.y, tid = threadIdx.x;
    auto chunks_of = [&](int x, bool& decreases) {
        const int lo = min(max(offsets[x], 0), m_rows), hi = min(max(offsets[x + 1], 0), m_rows);
        decreases |= hi < lo;
        return pieces(max(hi - lo, 0), chunk_rows);
    };
    int before = 0;
    bool decreases = false;                            // then there are no parts, and nothing is written
    for (int x = tid; x < (int)gridDim.y; x += THREADS) {
        const int n = chunks_of(x, decreases);
        before += x < e ? n : 0;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) before += __shfl_xor(before, d, kWave);
    const bool any = __any(decreases);
    if (tid % kWave == 0) {
        wave_sum[tid / kWave] = before;
        wave_decreases[tid / kWave] = any;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / kWave; i++)
        if (wave_decreases[i]) return;
    int first = 0;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; i++) first += wave_sum[i];
    int last = min(first + chunks_of(e, decreases), max_chunks);
    const int lane = tid % OWN, share = SPLIT == 1 ? 0 : tid / OWN;
    if constexpr (SPLIT > 1) {
        const int run = (max(last - first, 0) + SPLIT - 1) / SPLIT;
        first += share * run;
        last = min(last, first + run);
    }
    const int64_t i = ((int64_t)blockIdx.x * OWN + lane) * 4;
    const bool in = i < N * K;
    v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
    const float* p = part + (in ? i : 0);
    for (int c = first; c < last; c += 8) {
        v4f v[8];
#pragma unroll
        for (int u = 0; u < 8; u++) v[u] = *reinterpret_cast<const v4f*>(p + min(c + u, last - 1) * (N * K));
#pragma unroll
        for (int u = 0; u < 8; u++)
            if (c + u < last) sum += v[u];
    }
    if constexpr (SPLIT > 1) {
        others[share][lane] = sum;
        __syncthreads();
        if (share > 0) return;
#pragma unroll
        for (int s = 1; s < SPLIT; s++) sum += others[s][lane];
    }
    if (!in) return;
    const int64_t n = i / K, k = i - n * K, o = e * stride_e + n * stride_n + k;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float v = sum[j];
        if (accumulate) v += load_as_f32<DT>(out, o + j);
        store_from_f32<DT>(out, o + j, v);
    }
}

template <int DT>
void launch_join(hipStream_t st, const float* part, const WgradArgs& g, void* dw, int64_t stride_e, int64_t stride_n, int accumulate) {
    const int64_t quads = g.N * g.K / 4;
    if (quads * g.n_experts >= 65536)                 // a workgroup of 256 for every CU
        hipLaunchKernelGGL((wgrad_join_kernel<DT, 1>), dim3((unsigned)ceil_div(quads, 256), (unsigned)g.n_experts), dim3(256), 0, st, part,
                           g.offsets, g.m_rows, g.chunk_rows, g.max_chunks, g.N, g.K, dw, stride_e, stride_n, accumulate);
    else
        hipLaunchKernelGGL((wgrad_join_kernel<DT, kJoinSplit>), dim3((unsigned)ceil_div(quads, 64), (unsigned)g.n_experts), dim3(64 * kJoinSplit), 0, st,
                           part, g.offsets, g.m_rows, g.chunk_rows, g.max_chunks, g.N, g.K, dw, stride_e, stride_n, accumulate);
}

template <class C, bool SAVED, bool F16>
int wgrad_resident() {
    static std::atomic<int> cached[64];   // concurrent first calls may both fill it, with the same value
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
    int c = cached[dev].load(std::memory_order_relaxed);
    if (c == 0) {
        int per_cu = 0, cus = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, b16_wgrad_kernel<C, SAVED, F16>, C::THREADS, 0) != hipSuccess ||
            hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            return 0;
        c = per_cu * cus;
        if (c > 0) cached[dev].store(c, std::memory_order_relaxed);
    }
    return c;
}

template <class C, bool SAVED, bool F16>
int wgrad_launch_cfg(hipStream_t st, WgradArgs g) {
    const int64_t nt = ceil_div(g.N, C::BP), kt = ceil_div(g.K, C::BQ);
    const int64_t tiles = nt * kt * (g.chunk_rows > 0 ? g.max_chunks : g.n_experts);
    if (nt * kt > 0x7FFFFFFF / 64 || tiles > 0x7FFFFFFF - (1 << 20)) return MOE_ERR_SHAPE;
    g.n_tiles = (int)nt;
    g.k_tiles = (int)kt;
    int wgs = wgrad_resident<C, SAVED, F16>() / kXcds * kXcds;
    if (wgs < kXcds) return MOE_ERR_HIP;
    wgs = (int)std::min<int64_t>(wgs, ceil_div(tiles, kXcds) * kXcds);
    hipLaunchKernelGGL((b16_wgrad_kernel<C, SAVED, F16>), dim3((unsigned)wgs), dim3(C::THREADS), 0, st, g);
    return launch_status();
}

using Tile256 = Cfg<256, 256, 2, 4, 2, 1>;
using Tile256x128 = Cfg<256, 128, 4, 2, 3, 1>;
using Tile128 = Cfg<128, 128, 2, 2, 2, 2>;

template <class C>
int wgrad_launch(hipStream_t st, bool saved, bool f16, const WgradArgs& g) {
    if (saved) return f16 ? wgrad_launch_cfg<C, true, true>(st, g) : wgrad_launch_cfg<C, true, false>(st, g);
    return f16 ? wgrad_launch_cfg<C, false, true>(st, g) : wgrad_launch_cfg<C, false, false>(st, g);
}

bool wgrad_shape_ok(int64_t m_rows, int64_t E, int64_t N, int64_t K) {
    return m_rows >= 0 && m_rows <= 0x7FFFFFFF && E >= 1 && E <= kMaxExperts && N >= 8 && N <= kMaxWidth && N % 8 == 0 &&
           K >= 8 && K <= kMaxWidth && K % 8 == 0;
}

// The tile, and the rows of a chunk (0: the experts' rows stay whole).
struct WgradPlan {
    int tile, chunk_rows;
};

// Measured per tile: the workgroups that the device's 256 CUs hold, and the time of a step in us when they are few and
// when they are all there.
struct WgradCost {
    int bp, bq, slots;
    double alone, full;
};
constexpr WgradCost kWgradCosts[] = {{128, 128, 512, 0.80, 1.07}, {256, 128, 256, 0.83, 1.00}, {256, 256, 256, 1.33, 1.86}};

// The plan of least estimated time, in us: rounds of workgroups times (a chunk's steps, and 4.3 for its start and
// stores), or the bytes at 5 TB/s if that is more, and for cut rows the join: 6.8 and its bytes at 4.9 TB/s.  Whole
// ranges are taken as 1.12 of the average expert's, 1.35 where one round has to wait for the longest (the counts are
// on the device); a cut adds half a chunk an expert.  Chunks are tried that fill the device once or twice, and the
// length at which steps and join would balance.  A tenth of the work is added so that tiles bound by the same bytes are
// told apart.  Over 42 problems from 2 to 100000 rows and 1 to 224 experts the plan took 2.1 % more time than the best of
// all tiles and chunk lengths in the mean and 12 % at most.
WgradPlan wgrad_plan(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K) {
    const double R = (double)m_rows, E = (double)n_experts, NK = (double)N * (double)K;
    WgradPlan best{0, 0};
    double least = 0.0;
    for (int i = 0; i < 3; i++) {
        const WgradCost& c = kWgradCosts[i];
        const double nt = (double)(ceil_div(N, c.bp) * ceil_div(K, c.bq));
        auto time = [&](double chunks, double rows, bool cut) {
            const double tiles = chunks * nt, rounds = std::ceil(tiles / c.slots - 1e-9);
            const double step = c.alone + (c.full - c.alone) * std::min(1.0, std::max(0.0, i == 0 ? tiles / 256.0 - 1.0 : tiles / 256.0));
            const double uneven = cut || n_experts == 1 ? 1.0 : rounds > 1.0 ? 1.12 : 1.35;
            const double steps = std::max(1.0, std::ceil(rows / kStep)) * uneven;
            const double work = rounds * (steps * step + 4.3);
            const double bytes = R * (double)(N + K) * 2.0 + chunks * NK * (cut ? 4.0 : 2.0);
            return std::max(work, bytes / 5e6 + 3.0) + 0.1 * work + (cut ? 6.8 + (chunks + E) * 4.0 * NK / 4.9e6 : 0.0);
        };
        const double whole = time(E, R / E, false);
        if (i == 0 || whole < least) {
            least = whole;
            best = {i, 0};
        }
        const double balance = std::sqrt(R * kStep / c.alone * 4.0 * NK / 4.9e6);
        for (int j = 0; j < 3; j++) {
            const double room = j * c.slots / nt - (n_experts == 1 ? 0.0 : E);      // chunks of j rounds
            if (j > 0 && std::floor(room) < 1.0) continue;
            const double want = j == 0 ? balance : R / std::floor(room);
            const double rows = std::max(256.0, std::ceil(want / kStep) * kStep);
            if (rows * E > R || rows >= R) continue;                                   // would not cut an average expert
            const double t = time(n_experts == 1 ? std::ceil(R / rows) : R / rows + 0.5 * E, rows, true);
            if (t < least) {
                least = t;
                best = {i, (int)rows};
            }
        }
    }
    return best;
}

int64_t wgrad_max_chunks(int64_t m_rows, int64_t E, int64_t chunk_rows) { return m_rows / chunk_rows + E; }

}  // namespace b16
}  // namespace moe

using namespace moe;

extern "C" size_t moe_b16_grouped_wgrad_workspace_size(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K) {
    if (!b16::wgrad_shape_ok(m_rows, n_experts, N, K)) return 0;
    const int rows = b16::wgrad_plan(m_rows, n_experts, N, K).chunk_rows;
    return rows > 0 ? (size_t)b16::wgrad_max_chunks(m_rows, n_experts, rows) * N * K * 4 : 0;
}

extern "C" int moe_b16_grouped_wgrad_plan(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K, int32_t plan[3]) {
    if (!plan) return MOE_ERR_NULL;
    if (!b16::wgrad_shape_ok(m_rows, n_experts, N, K)) return MOE_ERR_SHAPE;
    const b16::WgradPlan p = b16::wgrad_plan(m_rows, n_experts, N, K);
    plan[0] = b16::kWgradCosts[p.tile].bp;
    plan[1] = b16::kWgradCosts[p.tile].bq;
    plan[2] = p.chunk_rows;
    return MOE_OK;
}

extern "C" int moe_b16_grouped_wgrad(const void* dy, int64_t dy_stride, int dt, const void* a, int64_t a_stride,
                                     int a_dt, const float* a_s, int64_t a_s_stride, const int32_t* expert_offsets,
                                     int64_t n_experts, int64_t N, int64_t K, int64_t m_rows, void* dw, int dw_dt,
                                     int64_t dw_stride_e, int64_t dw_stride_n, int accumulate, void* workspace,
                                     size_t ws_bytes, void* stream) {
    if ((dt != MOE_BF16 && dt != MOE_F16) || !dtype_ok(dw_dt)) return MOE_ERR_DTYPE;
    const bool saved = a_dt == MOE_E4M3;
    if (!saved && a_dt != dt) return MOE_ERR_DTYPE;
    if (!b16::wgrad_shape_ok(m_rows, n_experts, N, K) || (saved && K % 16)) return MOE_ERR_SHAPE;
    if (accumulate != 0 && accumulate != 1) return MOE_ERR_SHAPE;
    if (!dw || !expert_offsets) return MOE_ERR_NULL;
    if (dw_stride_n < K || (n_experts > 1 && dw_stride_e / dw_stride_n < N)) return MOE_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(dw) % (dw_dt == MOE_F32 ? 4 : 2)) return MOE_ERR_ALIGN;
    if (m_rows > 0) {
        if (!dy || !a || (saved && !a_s)) return MOE_ERR_NULL;
        if (dy_stride < N || a_stride < K || (saved && a_s_stride < ceil_div(K, 128))) return MOE_ERR_SHAPE;
        if (!aligned16(dy) || !aligned16(a) || dy_stride % 8 || a_stride % (saved ? 16 : 8)) return MOE_ERR_ALIGN;
    }
    b16::WgradArgs g{};
    g.dy = (const char*)dy; g.dy_stride = dy_stride * 2;
    g.a = (const char*)a; g.a_stride = saved ? a_stride : a_stride * 2;
    g.a_s = a_s; g.a_s_stride = a_s_stride;
    g.offsets = expert_offsets; g.m_rows = (int)m_rows; g.n_experts = (int)n_experts; g.N = N; g.K = K;
    const b16::WgradPlan plan = b16::wgrad_plan(m_rows, n_experts, N, K);
    g.chunk_rows = plan.chunk_rows;
    g.out = (char*)dw; g.out_dt = dw_dt; g.stride_e = dw_stride_e; g.stride_n = dw_stride_n;
    g.accumulate = accumulate;
    auto st = as_stream(stream);
    if (g.chunk_rows > 0) {
        g.max_chunks = (int)b16::wgrad_max_chunks(m_rows, n_experts, g.chunk_rows);
        if (!workspace) return MOE_ERR_NULL;
        if (ws_bytes < (size_t)g.max_chunks * N * K * 4) return MOE_ERR_WORKSPACE;
        if (!aligned16(workspace)) return MOE_ERR_ALIGN;
        g.out = (char*)workspace; g.out_dt = MOE_F32; g.stride_e = N * K; g.stride_n = K; g.accumulate = 0;
    }
    const bool f16 = dt == MOE_F16;
    const int rc = plan.tile == 0   ? b16::wgrad_launch<b16::Tile128>(st, saved, f16, g)
                   : plan.tile == 1 ? b16::wgrad_launch<b16::Tile256x128>(st, saved, f16, g)
                                    : b16::wgrad_launch<b16::Tile256>(st, saved, f16, g);
    if (rc != MOE_OK || g.chunk_rows == 0) return rc;
    const float* part = (const float*)workspace;
    if (dw_dt == MOE_F32) b16::launch_join<kF32>(st, part, g, dw, dw_stride_e, dw_stride_n, accumulate);
    else if (dw_dt == MOE_BF16) b16::launch_join<kBF16>(st, part, g, dw, dw_stride_e, dw_stride_n, accumulate);
    else b16::launch_join<kF16>(st, part, g, dw, dw_stride_e, dw_stride_n, accumulate);
    return launch_status();
}
