// Grouped products with MXFP4 on both sides, and the gate/up product with the gated activation and its MXFP4 requant in
// the epilogue.  Rows are sorted by expert; out[r, n] = sum_k A[r, k] W[e(r)][n, k].  Slot mode is the decode form: every
// row streams its own expert.
//
// MI355X design of the grouped mode (the tile engine is mx4_tile.h): persistent workgroups walk the tiles in panels, as
// b16_gemm.hip does, and the load pipeline runs on across tiles.  A rows may be named by a map, so the tokens' codes are
// read in place and no gathered copy is written.
// The fused form's tile holds 32 gate columns and the matching 32 up columns in every wave (MQ = 4 sub-tiles: two of
// gate, two of up), so a lane forms act(gate) * up from its own accumulators, the four lanes of a row hold a whole scale
// group of 32, and its maximum is two lane moves.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "mx4_tile.h"

namespace moe {
namespace mx4 {
namespace {

// A workgroup's tiles of `walk`: start, start + G, ... below `tiles`.
// BUF: the operands are read as buffers (every extent below kNowhere bytes, K a multiple of 128: scale words are whole); else
// by 64-bit addresses, with the last words' scales masked.
template <class C, bool FUSED, bool BUF, class W>
__device__ __forceinline__ void run_tiles(const GemmArgs& g, const W& walk, uint8_t* ring, int lane, int wave) {
    constexpr int S = C::S, LPS = C::LOADS;
    constexpr int COLS = FUSED ? C::BQ / 2 : C::BQ;    // output columns of a tile
    static_assert(C::MQ == 4, "a wave holds 32 gate and 32 up columns, or 64 columns");
    const uint32_t lds = lds_offset(ring), chunk_at = lds + S * C::CODES;
    const int steps = (int)((g.K + kStepK - 1) / kStepK), blocks = (int)(g.K / kGroup), words = (blocks + 3) / 4;
    const int chunks = (steps + kChunk - 1) / kChunk;
    auto first_chunk = [&](int expert) { return expert * kStagger % chunks; };

    // The tile last looked up: the producers and the consumer come to a tile one after the other.
    Tile near{};
    int near_t = -1;
    auto tile_of = [&](int t) __attribute__((always_inline)) {
        if (t != near_t) {
            near = walk.locate(t, lane);
            near_t = t;
        }
        return near;
    };

    // Producer of codes: the step that is requested next.  Past the last tile it goes on with zeros into stages that nobody
    // reads, so the loads in flight can be counted the same way to the end.
    int prod_t = walk.start, prod_left = 0, prod_kt = 0, prod_stage = 0;
    const int row_byte = code_byte(wave, lane);
    // !BUF: each lane's source of every load, and the bytes of a row (0 past the last tile)
    const char *p_src[BUF ? 1 : C::P_LOADS], *q_src[BUF ? 1 : C::Q_LOADS], *s_src[BUF ? 1 : C::LOADS];
    int64_t prod_bytes = 0;
    // BUF: each lane's offsets; what the step's lanes past the end of k (the last step's second half, or all of them past the
    // last tile) take instead is or-ed in.  The rows of W that a lane takes differ from one load to the next by as much in every
    // lane: one offset of the lane's own and a scalar one per load.  (Rows past the last are past the end of the bank, or
    // the fused form's gate rows past the last some rows of up; their columns are dropped.)
    uint32_t p_off[BUF ? C::P_LOADS : 1], q_off = 0, code_out = 0;
    uint32_t sp_off[BUF ? C::P_LOADS : 1], sq_off = 0;
    auto w_past = [&](int j) __attribute__((always_inline)) {                  // rows from a lane's first to that of load j
        const int r = j * C::NW * 8;
        return FUSED ? (r >> 6) * 32 + (r & 31) + (r & 32 ? (int)g.N : 0) : r;
    };
    auto w_first = [&](const Tile& ti, int l) __attribute__((always_inline)) {
        const int r = code_row<C::NW>(0, wave, l);
        return ti.n0 + (FUSED ? (r & 31) + (r & 32 ? (int)g.N : 0) : r);
    };
    const bool half_step = BUF && g.K % kStepK != 0;
    v4i a_buf, as_buf, w_buf, ws_buf;
    if constexpr (BUF) {
        a_buf = buffer_of(g.a, (g.a_n - 1) * g.a_stride + g.K / 2);
        as_buf = buffer_of(g.a_s, (g.a_n - 1) * g.a_s_stride + blocks);
    }
    const int64_t bank = FUSED ? 2 * g.N : g.N;
    auto outside = [&]() __attribute__((always_inline)) {
        code_out = prod_t >= walk.tiles || (half_step && prod_kt == steps - 1 && row_byte >= kRowBytes / 2) ? kNowhere : 0u;
    };
    auto aim = [&]() __attribute__((always_inline)) {
        prod_bytes = prod_t < walk.tiles ? g.K / 2 : 0;
        if (prod_t < walk.tiles) {
            const Tile ti = tile_of(prod_t);
            const int l = fresh(lane);
            prod_left = steps;
            prod_kt = first_chunk(ti.expert) * kChunk;
            const char* w = g.w + ti.expert * g.w_stride_e;
            if constexpr (BUF) w_buf = buffer_of(w, (bank - 1) * g.w_stride_n + g.K / 2);
#pragma unroll
            for (int j = 0; j < C::P_LOADS; j++) {
                const int64_t m = walk.a_row(ti, code_row<C::NW>(j, wave, l));
                if constexpr (BUF) p_off[j] = m < 0 ? kNowhere : (uint32_t)(m * g.a_stride) + row_byte;
                else p_src[j] = m < 0 ? nullptr : g.a + m * g.a_stride + row_byte;
            }
            if constexpr (BUF) {
                q_off = (uint32_t)w_first(ti, l) * (uint32_t)g.w_stride_n + row_byte;
            } else {
#pragma unroll
                for (int j = 0; j < C::Q_LOADS; j++)
                    q_src[j] = w + walk.template w_row<FUSED>(ti, code_row<C::NW>(j, wave, l)) * g.w_stride_n + row_byte;
            }
        }
        if constexpr (BUF) outside();
    };
    // Load j of the step that is requested next.
    auto part = [&](int j) __attribute__((always_inline)) {
        const uint32_t dst = lds + prod_stage * C::CODES + wave * 1024 + j * C::NW * 1024;
        if constexpr (BUF) {
            if (j < C::P_LOADS) buf16(p_off[j] | code_out, a_buf, prod_kt * kRowBytes, dst);
            else buf16(q_off | code_out, w_buf, (uint32_t)w_past(j - C::P_LOADS) * (uint32_t)g.w_stride_n + prod_kt * kRowBytes, dst);
        } else {
            const int64_t at = (int64_t)prod_kt * kRowBytes;
            const char* src = j < C::P_LOADS ? p_src[j] : q_src[j - C::P_LOADS];
            b16::dma16(row_byte < prod_bytes - at && src ? src + at : (const char*)&b16::kZeroPiece, dst);
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {                      // past the step whose loads have gone out
        prod_stage = prod_stage + 1 == S ? 0 : prod_stage + 1;
        prod_kt = prod_kt + 1 == steps ? 0 : prod_kt + 1;
        if (--prod_left <= 0) {
            prod_t += walk.G;
            aim();
        } else if (half_step) {
            outside();
        }
    };
    auto produce = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < LPS; j++) part(j);
        advance();
    };

    // Producer of scales: the chunk that is requested next (a tile's chunks in the order of its steps).  DMA j of a wave takes
    // eight rows, eight words of each; lane 8i + 4h + t: the word of step t's blocks 4h .. 4h+3, so that a lane of the
    // consumer finds its four words next to each other.
    int sc_t = walk.start, sc_left = 0, sc_c = 0;
    const int sc_word = 2 * (lane & 3) + ((lane >> 2) & 1);
    auto aim_scales = [&]() __attribute__((always_inline)) {
        sc_left = chunks;
        if (sc_t >= walk.tiles) return;
        const Tile ti = tile_of(sc_t);
        const int l = fresh(lane);
        sc_c = first_chunk(ti.expert);
        const char* w_s = g.w_s + ti.expert * g.w_s_stride_e;
        if constexpr (BUF) ws_buf = buffer_of(w_s, (bank - 1) * g.w_s_stride_n + blocks);
        if constexpr (BUF) sq_off = (uint32_t)w_first(ti, l) * (uint32_t)g.w_s_stride_n + sc_word * 4;
#pragma unroll
        for (int j = 0; j < C::LOADS; j++) {
            if (j < C::P_LOADS) {
                const int64_t m = walk.a_row(ti, code_row<C::NW>(j, wave, l));
                if constexpr (BUF) sp_off[j] = m < 0 ? kNowhere : (uint32_t)(m * g.a_s_stride) + sc_word * 4;
                else s_src[j] = m < 0 ? nullptr : g.a_s + m * g.a_s_stride + sc_word * 4;
            } else if constexpr (!BUF) {
                s_src[j] = w_s + walk.template w_row<FUSED>(ti, code_row<C::NW>(j - C::P_LOADS, wave, l)) * g.w_s_stride_n + sc_word * 4;
            }
        }
    };
    auto request_scales = [&]() __attribute__((always_inline)) {
        if (sc_left == 0) {
            sc_t += walk.G;
            aim_scales();
        }
        const bool in = sc_t < walk.tiles && sc_word < words - 2 * kChunk * sc_c;
        const uint32_t at = (uint32_t)sc_c * (kChunk * kRowScales);
#pragma unroll
        for (int j = 0; j < C::LOADS; j++) {
            const uint32_t dst = chunk_at + (j * C::NW + wave) * 256;                  // (BP / 8 = P_LOADS * NW: W's rows follow)
            if constexpr (BUF) {
                if (j < C::P_LOADS) buf4(in ? sp_off[j] : kNowhere, as_buf, at, dst);
                else buf4(in ? sq_off : kNowhere, ws_buf, (uint32_t)w_past(j - C::P_LOADS) * (uint32_t)g.w_s_stride_n + at, dst);
            } else {
                dma4(in && s_src[j] ? s_src[j] + at : (const char*)&b16::kZeroPiece, dst);
            }
        }
        sc_c = sc_c + 1 == chunks ? 0 : sc_c + 1;
        sc_left--;
    };

    aim_scales();
    request_scales();
    aim();
    constexpr bool PIPED = C::MP >= 4;                 // a wave's MFMAs are worth the software pipeline
#pragma unroll 1
    for (int i = 0; i < (PIPED ? S : S - 1); i++) produce();

    CodeFrag fp, fq;
    const int wp = wave / C::WQ, wq = wave % C::WQ;
    fp.set(wp * C::MP, lane);
    fq.set(wq * C::MQ, lane);
    Scales<C::MP, C::ROLLED> sp;
    Scales<C::MQ, C::ROLLED> sq;
    const uint32_t sp_at = chunk_at + scale_lane(wp * C::MP, lane), sq_at = chunk_at + C::BP * kChunk * kRowScales + scale_lane(wq * C::MQ, lane);

    int stage = 0;
    Frags<C> f;
    wait_loads<0>();                                   // the first chunk, and (all of) the first stages
    block_barrier();
    if constexpr (PIPED) f.first(fp, fq, lds);
    int before = kChunk;                               // steps of the chunk before
#pragma unroll 1
    for (int t = walk.start; t < walk.tiles; t += walk.G) {
        const Tile ti = tile_of(t);
        const int rows = ti.rows - wp * C::MP * 16;    // of this wave
        v4f acc[C::MP][C::MQ];
#pragma unroll
        for (int m = 0; m < C::MP; m++)
#pragma unroll
            for (int n = 0; n < C::MQ; n++) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        int c = first_chunk(ti.expert);
#pragma unroll 1
        for (int i = 0; i < chunks; i++) {
            // The chunk's scales to registers.  It was requested in the second step of the chunk before, ahead of that step's
            // codes: behind a whole chunk the waits for the steps since cover it.  (!PIPED: the workgroup meets at the
            // start of a step, so the meeting that publishes it is here.)
            if (before == 1) {
                block_barrier();                       // everyone has read the one before
                request_scales();
            }
            if (before < kChunk) {
                wait_loads<0>();
                block_barrier();
            } else if constexpr (!PIPED) {
                arrive<S, LPS>();
            }
            sp.read(sp_at, lane);
            sq.read(sq_at, lane);
            if constexpr (!BUF) {
                const int left = blocks - c * kChunk * kRowScales;
                const uint32_t low = scale_mask(left, lane), high = scale_mask(left - 2 * kRowScales, lane);
                sp.mask(low, high);
                sq.mask(low, high);
            }
            const int n_steps = min(kChunk, steps - c * kChunk);
            auto step = [&](auto number, int u) __attribute__((always_inline)) {
                constexpr int U = decltype(number)::value;
                const uint32_t at = lds + stage * C::CODES;
                stage = stage + 1 == S ? 0 : stage + 1;
                if constexpr (PIPED) {
                    if (u == 1) request_scales();
                    step_pipelined<C, U>(acc, f, fp, fq, sp, sq, at, lds + stage * C::CODES, part);
                    advance();
                } else {
                    if (u > 0) arrive<S, LPS>();
                    if (u == 1) request_scales();
                    produce();                         // into the stage that the step before this one read
                    step_plain<C, U>(acc, fp, fq, sp, sq, at);
                }
            };
            if constexpr (C::ROLLED) {
#pragma unroll 1
                for (int u = 0; u < n_steps; u++) {
                    sp.take(u);
                    sq.take(u);
                    step(std::integral_constant<int, 0>{}, u);
                }
            } else {
                step(std::integral_constant<int, 0>{}, 0);
                if (n_steps > 1) step(std::integral_constant<int, 1>{}, 1);
                if (n_steps > 2) step(std::integral_constant<int, 2>{}, 2);
                if (n_steps > 3) step(std::integral_constant<int, 3>{}, 3);
            }
            before = n_steps;
            c = c + 1 == chunks ? 0 : c + 1;
        }
        const int64_t c0 = ti.n0 + wq * (COLS / C::WQ);
        const int cols = (int)min(g.N - c0, (int64_t)(COLS / C::WQ));
        const int64_t r0 = ti.row0 + wp * C::MP * 16;
        if (rows > 0 && cols > 0) {
            if constexpr (FUSED) store_act_of(g, acc, r0, rows, c0, fresh(lane));
            else b16::store_wave_dt(g.out, g.out_dt, false, r0 * g.out_stride + c0, g.out_stride, rows, cols, acc, fresh(lane));
        }
    }
    wait_loads<0>();                                   // no load may write LDS after the workgroup has left it
}

// The tiles of C, a round of one on every workgroup after the other.  HALF: a last round that would leave half of the card
// idle or more is done by tiles of half the rows (C itself: it is not), each the only one of its workgroup.  16384 rows of
// eight uneven experts, 1088 tiles for 256 workgroups, take 329 us to 4096 columns of 8192, 358 with whole tiles, and 295
// where the rows make 1024 tiles.
template <class C, class HALF, bool FUSED, bool BUF>
__global__ void __launch_bounds__(C::THREADS, C::WAVES_PER_EU) mx4_gemm_kernel(const GemmArgs g) {
    constexpr bool SPLIT = !std::is_same<C, HALF>::value;
    static_assert(!SPLIT || (HALF::BP * 2 == C::BP && HALF::BQ == C::BQ && HALF::NW == C::NW), "a half has C's columns and waves");
    __shared__ __attribute__((aligned(1024))) uint8_t ring[C::LDS > HALF::LDS ? C::LDS : HALF::LDS];
    __shared__ int first_tile[kMaxExperts];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    Walk<C, FUSED ? C::BQ / 2 : C::BQ> walk(g, first_tile, reinterpret_cast<uint32_t*>(ring), tid, lane, wave);
    const int rest = walk.tiles % walk.G;
    const bool split = SPLIT && rest * 2 <= walk.G;
    if (split) walk.tiles -= rest;
    if (walk.start < walk.tiles) run_tiles<C, FUSED, BUF>(g, walk, ring, lane, wave);
    if constexpr (SPLIT) {
        if (!split || walk.start >= rest * 2) return;
        block_barrier();                               // everyone has done with the ring
        const Halves<HALF, decltype(walk)> halves{walk, walk.tiles, walk.start, rest * 2, walk.G};
        if (halves.locate(walk.start, lane).rows > 0) run_tiles<HALF, FUSED, BUF>(g, halves, ring, lane, wave);
    }
}

template <class C, class HALF, bool FUSED, bool BUF>
int resident_blocks() {
    static std::atomic<int> cached[64];   // concurrent first calls may both fill it, with the same value
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
    int c = cached[dev].load(std::memory_order_relaxed);
    if (c == 0) {
        int per_cu = 0, cus = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, (mx4_gemm_kernel<C, HALF, FUSED, BUF>), C::THREADS, 0) != hipSuccess ||
            hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            return 0;
        c = per_cu * cus;
        if (c > 0) cached[dev].store(c, std::memory_order_relaxed);
    }
    return c;
}

using Tile256 = Cfg<256, 256, 2, 4, 2, 1>;
using Tile128 = Cfg<128, 256, 2, 4, 3, 1>;
using Tile64 = Cfg<64, 256, 2, 4, 3, 1>;
using Tile64x64 = Cfg<64, 64, 4, 1, 3, 2>;
using Tile32x64 = Cfg<32, 64, 2, 1, 4, 2>;

template <class C, class HALF, bool FUSED, bool BUF>
int launch_form(hipStream_t st, GemmArgs g) {
    const int64_t n_tiles = ceil_div(g.N, FUSED ? C::BQ / 2 : C::BQ);
    const int64_t most = (g.m_rows / C::BP + std::min<int64_t>(g.n_experts, g.m_rows)) * n_tiles;
    if (most > 0x7FFFFFFF - (1 << 20)) return MOE_ERR_SHAPE;
    int wgs = resident_blocks<C, HALF, FUSED, BUF>() / kXcds * kXcds;
    if (wgs < kXcds) return MOE_ERR_HIP;
    wgs = (int)std::min<int64_t>(wgs, ceil_div(most, kXcds) * kXcds);
    g.n_tiles = (int)n_tiles;
    hipLaunchKernelGGL((mx4_gemm_kernel<C, HALF, FUSED, BUF>), dim3((unsigned)wgs), dim3(C::THREADS), 0, st, g);
    return launch_status();
}

template <class C, class HALF, bool FUSED>
int launch_cfg(hipStream_t st, const GemmArgs& g) {
    const int64_t bank = (FUSED ? 2 : 1) * g.N, scales = g.K / kGroup;
    // (a tile may name up to BQ rows of W past the bank's last, whose offsets still have to stay below kNowhere)
    const bool buf = g.K % 128 == 0 && std::max({(g.a_n - 1) * g.a_stride + g.K / 2, (g.a_n - 1) * g.a_s_stride + scales,
                                                 (bank + C::BQ) * g.w_stride_n, (bank + C::BQ) * g.w_s_stride_n}) < (int64_t)kNowhere;
    return buf ? launch_form<C, HALF, FUSED, true>(st, g) : launch_form<C, HALF, FUSED, false>(st, g);
}

// Which tile.  A round of tiles, one on every slot of the card, takes a step's time for each 256 of k and a time for its ends;
// both in microseconds, fitted to 516 products timed with all five (1 to 256 experts of 1 to 4096 rows, even and dealt at
// random; N x K from 512 x 2048 to 4096 x 8192).  The rule loses 1.2 % to the best tile on average and 29 % at most.  Two
// sides, to 4096 columns of 8192: 128 x 512 rows take 1408 us by 128 x 256 and 1302 by 256 x 256, 32 x 512 dealt at random
// 390 and 395; 8 x 32 rows 31 by 64 x 64 and 43 by 128 x 256.
// The slots of the 32 x 64 tile are fitted too: two of its workgroups fit a CU's LDS, 512 on the card, and 1024 is the number that
// told its times best.
struct TileCost {
    int bp, bq, slots;
    double step, ends;
};
constexpr TileCost kCosts[] = {{32, 64, 1024, 0.40, 6.8}, {64, 64, 512, 0.40, 2.5}, {64, 256, 256, 0.76, 1.6},
                               {128, 256, 256, 0.96, 3.8}, {256, 256, 256, 1.74, 6.7}};
constexpr int kFirstSplit = 3;                    // from this one on a last round of half the slots or fewer takes the tile before

int pick_tile(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K) {
    const double E = (double)n_experts, R = (double)m_rows, steps = (double)ceil_div(K, kStepK);
    const double used = n_experts == 1 ? 1.0 : std::min(R, E * (1.0 - std::pow(1.0 - 1.0 / E, R)));   // experts with rows
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < 5; i++) {
        const TileCost& c = kCosts[i];
        const double x = R / used / c.bp;
        const double per = n_experts == 1 ? std::ceil(x) : std::max(1.0, x + 0.32 * std::min(1.0, x));    // M tiles of one
        const double rounds = used * per * (double)ceil_div(N, c.bq) / c.slots, whole = std::floor(rounds + 1e-9), part = rounds - whole;
        auto cost = [&](int j) { return steps * kCosts[j].step + kCosts[j].ends; };
        auto at_most = [&](double f) { return i >= kFirstSplit && f <= 0.5 ? cost(i - 1) : cost(i); };    // a round of f of the slots
        const double even = whole * cost(i) + (part > 1e-9 ? at_most(part) : 0.0);
        const double t = 0.42 * even + 0.58 * std::max(rounds * cost(i), at_most(rounds));                  // (loads differ)
        if (i == 0 || t < least) {
            least = t;
            best = i;
        }
    }
    return best;
}

// N: rows of an expert's bank (fused: 2I).
template <bool FUSED>
int grouped_launch(hipStream_t st, const GemmArgs& g) {
    switch (pick_tile(g.m_rows, g.n_experts, FUSED ? 2 * g.N : g.N, g.K)) {
        case 0: return launch_cfg<Tile32x64, Tile32x64, FUSED>(st, g);
        case 1: return launch_cfg<Tile64x64, Tile64x64, FUSED>(st, g);
        case 2: return launch_cfg<Tile64, Tile64, FUSED>(st, g);
        case 3: return launch_cfg<Tile128, Tile64, FUSED>(st, g);
        default: return launch_cfg<Tile256, Tile128, FUSED>(st, g);
    }
}

// ------------------------------------------------------------------ slot mode
// A group of KS waves holds 16 columns of one row, each wave a part of k; W is the MFMA's row operand and the row of A
// stands in all 16 columns of the other.  The sums of the waves meet in LDS in order.  U windows of 256 of k are in flight.
template <int KS, int U, bool FUSED>
__global__ void __launch_bounds__(64 * KS * (FUSED ? 4 : 1))
mx4_slot_kernel(const GemmArgs g, const int32_t* __restrict__ slots, int64_t a_row_div, int col_groups) {
    constexpr int SUBS = FUSED ? 4 : 1;                // 16-column sub-tiles of a workgroup (fused: two of gate, two of up)
    __shared__ float part[SUBS][KS][16];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int sub = wave / KS, ks = wave % KS;
    const int l16 = lane & 15, quad = lane >> 4;
    const int64_t r = blockIdx.x / (unsigned)col_groups;
    const int64_t n0 = (int64_t)(blockIdx.x % (unsigned)col_groups) * (FUSED ? 32 : 16);
    const int slot = slots[r];
    const int64_t ar = g.a_rows ? (int64_t)g.a_rows[r] : r / a_row_div;
    const bool live = slot >= 0 && slot < g.n_experts;
    if (live) {
        const bool row_there = ar >= 0 && ar < g.a_n;  // else a row of zeros, which a NaN of the bank makes NaN all the same
        const int64_t col = FUSED ? n0 + (sub & 1) * 16 : n0;
        const int64_t row = min(col + l16, g.N - 1) + (FUSED && sub >= 2 ? g.N : 0);
        const char* w = g.w + slot * g.w_stride_e + row * g.w_stride_n;
        const char* ws = g.w_s + slot * g.w_s_stride_e + row * g.w_s_stride_n;
        const char* a = g.a + (row_there ? ar : 0) * g.a_stride;
        const char* as = g.a_s + (row_there ? ar : 0) * g.a_s_stride;
        const int windows = (int)((g.K + kStepK - 1) / kStepK), blocks = (int)(g.K / kGroup);
        const int per = (windows + KS - 1) / KS;
        const int end = min((ks + 1) * per, windows);
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int t0 = ks * per; t0 < end; t0 += U) {
            v4i w0[U], w1[U], x0[U], x1[U];
            uint32_t sw[U], sx[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                // this lane's blocks 8t + 2 quad and the next, whose scales are one aligned pair of bytes; past the end the last
                // block is read and counted as zero
                const int b = t0 + u < end ? 8 * (t0 + u) + 2 * quad : blocks, b0 = min(b, blocks - 1), b1 = min(b + 1, blocks - 1);
                w0[u] = *reinterpret_cast<const v4i*>(w + b0 * 16);
                w1[u] = *reinterpret_cast<const v4i*>(w + b1 * 16);
                sw[u] = *reinterpret_cast<const uint16_t*>(ws + (b0 & ~1));
                x0[u] = *reinterpret_cast<const v4i*>(a + b0 * 16);
                x1[u] = *reinterpret_cast<const v4i*>(a + b1 * 16);
                sx[u] = *reinterpret_cast<const uint16_t*>(as + (b0 & ~1));
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int b = t0 + u < end ? 8 * (t0 + u) + 2 * quad : blocks;
                const v4i zero = {0, 0, 0, 0};
                if (!row_there) { x0[u] = zero; x1[u] = zero; sx[u] = 0; }
                if (b >= blocks) { w0[u] = zero; x0[u] = zero; sw[u] = 0; sx[u] = 0; }
                if (b + 1 >= blocks) { w1[u] = zero; x1[u] = zero; sw[u] &= 255u; sx[u] &= 255u; }
                acc = mfma<0>(w0[u], sw[u], x0[u], sx[u], acc);
                acc = mfma<1>(w1[u], sw[u], x1[u], sx[u], acc);
            }
        }
        if (l16 == 0) {
#pragma unroll
            for (int i = 0; i < 4; i++) part[sub][ks][4 * quad + i] = acc[i];
        }
    }
    __syncthreads();
    if (wave != 0) return;
    auto total = [&](int s, int c) {
        float v = live ? part[s][0][c] : 0.0f;
#pragma unroll
        for (int k = 1; k < KS; k++) v += live ? part[s][k][c] : 0.0f;
        return v;
    };
    if constexpr (FUSED) {
        // a column a lane for the gate, eight a lane for the codes
        const int c = lane & 31;
        const float gt = total(c / 16, c % 16), up = total(2 + c / 16, c % 16);
        float v = 0.0f;
        switch (g.act) {
            case 1: v = gated<1>(gt, up); break;
            case 2: v = gated<2>(gt, up); break;
            case 3: v = gated<3>(gt, up); break;
            case 4: v = gated<4>(gt, up); break;
            default: v = gated<5>(gt, up); break;
        }
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; i++) h[i] = __shfl(v, 8 * (lane & 3) + i, kWave);
        uint32_t top = max_bits8(h);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1, kWave));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2, kWave));
        const uint32_t byte = live ? scale_byte(top, g.ceil != 0) : 0u;
        const uint32_t codes = live ? encode8(h, byte) : 0u;
        if (lane < 4) {
            uint8_t* out = (uint8_t*)g.out + r * g.out_stride + n0 / 2 + 4 * lane;
            *reinterpret_cast<uint16_t*>(out) = (uint16_t)codes;
            *reinterpret_cast<uint16_t*>(out + 2) = (uint16_t)(codes >> 16);
            if (lane == 0) g.s[r * g.s_stride + n0 / kGroup] = (uint8_t)byte;
        }
    } else if (lane < 16 && n0 + lane < g.N) {
        const float v = total(0, lane);
        const int64_t o = r * g.out_stride + n0 + lane;
        if (g.out_dt == MOE_F32) store_from_f32<kF32>(g.out, o, v);
        else if (g.out_dt == MOE_BF16) store_from_f32<kBF16>(g.out, o, v);
        else store_from_f32<kF16>(g.out, o, v);
    }
}

template <int KS, int U, bool FUSED>
int slot_launch_ks(hipStream_t st, const GemmArgs& g, const int32_t* slots, int64_t a_row_div) {
    constexpr int THREADS = 64 * KS * (FUSED ? 4 : 1);
    const int64_t groups = ceil_div(g.N, FUSED ? 32 : 16);
    if (groups * g.m_rows >= (int64_t)1 << (FUSED ? 22 : 24)) return MOE_ERR_SHAPE;   // a grid's threads fit 32 bits, whatever KS
    hipLaunchKernelGGL((mx4_slot_kernel<KS, U, FUSED>), dim3((unsigned)(groups * g.m_rows)), dim3(THREADS), 0, st, g, slots, a_row_div,
                       (int)groups);
    return launch_status();
}

// The parts of k go by K alone, so that the fused form's sums are those of the plain one.  A wave asks for as many windows at
// once as it has, two at most: one at a time, with the scales in single bytes, 64 rows of 4096 x 4096 took 137 us, two 105
// (5.4 TB/s); four 105, and fused 133, for they leave half the waves a unit.  Where each of the four waves has one window,
// asking for two of which one is not there costs 53 us instead of 29 (64 rows of 4096 x 1024).  Small calls are
// latency: eight rows of 1536 x 2048 take 5.3 us (2.5 TB/s).
template <bool FUSED>
int slot_launch(hipStream_t st, const GemmArgs& g, const int32_t* slots, int64_t a_row_div) {
    if (g.K <= 2 * kStepK) return slot_launch_ks<1, 2, FUSED>(st, g, slots, a_row_div);
    return g.K > 4 * kStepK ? slot_launch_ks<4, 2, FUSED>(st, g, slots, a_row_div) : slot_launch_ks<4, 1, FUSED>(st, g, slots, a_row_div);
}

// Checks that both products share; MOE_OK when the call may go on.  bank_rows: N, or 2I.
int check_operands(const GemmArgs& g, int64_t n_experts, int64_t m_rows, int64_t bank_rows, int mode, const int32_t* slot_ids,
                   int64_t a_row_div) {
    if (n_experts > 0) {
        if (!g.a || !g.a_s || !g.w || !g.w_s) return MOE_ERR_NULL;
        const int64_t codes = g.K / 2, scales = ceil_div(g.K, 128) * 4;
        if (g.a_n < 1 || g.a_stride < codes || g.w_stride_n < codes || g.a_s_stride < scales || g.w_s_stride_n < scales) return MOE_ERR_SHAPE;
        if (n_experts > 1 && (g.w_stride_e / g.w_stride_n < bank_rows || g.w_s_stride_e / g.w_s_stride_n < bank_rows)) return MOE_ERR_SHAPE;
        if (!aligned16(g.a) || !aligned16(g.w) || g.a_stride % 16 || g.w_stride_n % 16 || g.w_stride_e % 16) return MOE_ERR_ALIGN;
        if (reinterpret_cast<uintptr_t>(g.a_s) % 4 || reinterpret_cast<uintptr_t>(g.w_s) % 4 || g.a_s_stride % 4 || g.w_s_stride_n % 4 ||
            g.w_s_stride_e % 4)
            return MOE_ERR_ALIGN;
    }
    if (mode == MOE_MODE_SLOT) {
        if (!slot_ids) return MOE_ERR_NULL;
        if (a_row_div < 1) return MOE_ERR_SHAPE;
        return n_experts > 0 && !g.a_rows && ceil_div(m_rows, a_row_div) > g.a_n ? MOE_ERR_SHAPE : MOE_OK;
    }
    if (n_experts < 1 || n_experts > kMaxExperts) return MOE_ERR_SHAPE;
    if (!g.offsets) return MOE_ERR_NULL;
    return !g.a_rows && m_rows > g.a_n ? MOE_ERR_SHAPE : MOE_OK;
}

bool widths_ok(int64_t N, int64_t K, int64_t of) {
    return N >= of && N <= kMaxWidth && N % of == 0 && K >= kGroup && K <= kMaxWidth && K % kGroup == 0;
}

}  // namespace
}  // namespace mx4
}  // namespace moe

using namespace moe;

extern "C" int moe_mx4_grouped_tile(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K, int32_t tile[2]) {
    if (!tile) return MOE_ERR_NULL;
    if (m_rows < 1 || m_rows > 0x7FFFFFFF || n_experts < 1 || n_experts > mx4::kMaxExperts || !mx4::widths_ok(N, K, 8)) return MOE_ERR_SHAPE;
    const mx4::TileCost& c = mx4::kCosts[mx4::pick_tile(m_rows, n_experts, N, K)];
    tile[0] = c.bp;
    tile[1] = c.bq;
    return MOE_OK;
}

extern "C" int moe_mx4_grouped_gemm(const uint8_t* a_q, int64_t a_stride, const uint8_t* a_s, int64_t a_s_stride, int64_t a_n,
                                    const int32_t* a_rows, const uint8_t* w_q, int64_t w_stride_e, int64_t w_stride_n,
                                    const uint8_t* w_s, int64_t w_s_stride_e, int64_t w_s_stride_n, int64_t n_experts, int64_t N,
                                    int64_t K, int mode, const int32_t* expert_offsets, const int32_t* slot_ids, int64_t m_rows,
                                    int64_t a_row_div, void* out, int out_dt, int64_t out_stride, void* stream) {
    if (mode != MOE_MODE_GROUPED && mode != MOE_MODE_SLOT) return MOE_ERR_SHAPE;
    if (!dtype_ok(out_dt)) return MOE_ERR_DTYPE;
    if (m_rows < 0 || m_rows > 0x7FFFFFFF || n_experts < 0 || n_experts > 0x7FFFFFFF || !mx4::widths_ok(N, K, 8)) return MOE_ERR_SHAPE;
    if (m_rows == 0) return MOE_OK;
    if (!out) return MOE_ERR_NULL;
    if (out_stride < N) return MOE_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(out) % (out_dt == MOE_F32 ? 4 : 2)) return MOE_ERR_ALIGN;
    mx4::GemmArgs g{};
    g.a = (const char*)a_q; g.a_stride = a_stride; g.a_s = (const char*)a_s; g.a_s_stride = a_s_stride; g.a_n = a_n; g.a_rows = a_rows;
    g.w = (const char*)w_q; g.w_stride_e = w_stride_e; g.w_stride_n = w_stride_n;
    g.w_s = (const char*)w_s; g.w_s_stride_e = w_s_stride_e; g.w_s_stride_n = w_s_stride_n;
    g.n_experts = (int)n_experts; g.N = N; g.K = K; g.offsets = expert_offsets; g.m_rows = (int)m_rows;
    g.out = out; g.out_dt = out_dt; g.out_stride = out_stride;
    const int st = mx4::check_operands(g, n_experts, m_rows, N, mode, slot_ids, a_row_div);
    if (st != MOE_OK) return st;
    if (mode == MOE_MODE_SLOT) return mx4::slot_launch<false>(as_stream(stream), g, slot_ids, a_row_div);
    return mx4::grouped_launch<false>(as_stream(stream), g);
}

extern "C" int moe_mx4_grouped_gemm_act_quant(const uint8_t* a_q, int64_t a_stride, const uint8_t* a_s, int64_t a_s_stride,
                                              int64_t a_n, const int32_t* a_rows, const uint8_t* w_q, int64_t w_stride_e,
                                              int64_t w_stride_n, const uint8_t* w_s, int64_t w_s_stride_e, int64_t w_s_stride_n,
                                              int64_t n_experts, int64_t I, int64_t K, int mode, const int32_t* expert_offsets,
                                              const int32_t* slot_ids, int64_t m_rows, int64_t a_row_div, int act, int rule,
                                              uint8_t* out_q, int64_t q_stride, uint8_t* out_s, int64_t s_stride, void* stream) {
    if (mode != MOE_MODE_GROUPED && mode != MOE_MODE_SLOT) return MOE_ERR_SHAPE;
    if (act < MOE_ACT_SILU_MUL || act > MOE_ACT_MUL || (rule != MOE_MX_FLOOR && rule != MOE_MX_CEIL)) return MOE_ERR_SHAPE;
    if (m_rows < 0 || m_rows > 0x7FFFFFFF || n_experts < 0 || n_experts > 0x7FFFFFFF || !mx4::widths_ok(I, K, mx4::kGroup)) return MOE_ERR_SHAPE;
    if (m_rows == 0) return MOE_OK;
    if (!out_q || !out_s) return MOE_ERR_NULL;
    if (q_stride < I / 2 || s_stride < I / mx4::kGroup) return MOE_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(out_q) % 2 || q_stride % 2) return MOE_ERR_ALIGN;
    mx4::GemmArgs g{};
    g.a = (const char*)a_q; g.a_stride = a_stride; g.a_s = (const char*)a_s; g.a_s_stride = a_s_stride; g.a_n = a_n; g.a_rows = a_rows;
    g.w = (const char*)w_q; g.w_stride_e = w_stride_e; g.w_stride_n = w_stride_n;
    g.w_s = (const char*)w_s; g.w_s_stride_e = w_s_stride_e; g.w_s_stride_n = w_s_stride_n;
    g.n_experts = (int)n_experts; g.N = I; g.K = K; g.offsets = expert_offsets; g.m_rows = (int)m_rows;
    g.out = out_q; g.out_stride = q_stride; g.s = out_s; g.s_stride = s_stride; g.act = act; g.ceil = rule == MOE_MX_CEIL;
    const int st = mx4::check_operands(g, n_experts, m_rows, 2 * I, mode, slot_ids, a_row_div);
    if (st != MOE_OK) return st;
    if (mode == MOE_MODE_SLOT) return mx4::slot_launch<true>(as_stream(stream), g, slot_ids, a_row_div);
    return mx4::grouped_launch<true>(as_stream(stream), g);
}
