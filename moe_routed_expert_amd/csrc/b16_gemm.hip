// Grouped products with 16-bit operands: the expert GEMMs of banks that are not block-quantized, and their
// data gradient.  Rows are sorted by expert; out[r, n] = sum_k A[r, k] W[e(r)](n, k) with W held [N][K] (the
// forward) or [K][N] (the data gradient, which reduces over the rows of the bank as the forward holds it).
// Slot mode is the decode form: every row streams its own expert.
//
// MI355X design of the grouped mode (the tile engine is b16_tile.h).
//  * Tiles from 32 x 64 to 256 x 256, by estimated time (pick_tile).  Persistent workgroups, one per CU (two of the
//    64 x 64 tile): a tile's LDS ring takes most of the CU's 160 KB.  Each reads the device offsets once into an LDS
//    table of every expert's first M tile and walks its tiles; the load pipeline runs on across tiles, so a tile's
//    first steps are in flight while the tile before it is multiplied and stored.
//  * Tiles are numbered in panels of kPanel M tiles, M fastest, and tile t of round s goes to workgroup t % G
//    with the workgroups of one XCD next to each other: the tiles that an XCD works on at one time form a
//    patch whose A rows and weight columns meet in its L2.
//  * Bound by the bank's bytes where experts have few rows: 256 experts of 2048 x 4096 and 24576 rows take 754 us
//    (6.1 TB/s over banks, rows and output).  Bound by the MFMAs' feed where they have many: 8 experts of 2048 rows,
//    4096 x 8192 take 860 us (1.28 PFLOP/s; the matrix units are busy two thirds of the cycles, and zeros as data
//    take 771 us).  Bound by latency where there is little: 333 rows over 16 experts, 1000 x 520 take 10.3 us a call and 9.5
//    in a graph of such calls, of which 6.4 are there at K = 8 already.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "b16_tile.h"

namespace moe {
namespace b16 {


// The tiles of expert e walk k in rotation from step kStagger * e.  With every tile at the same k, the 128-byte
// pieces that are read at one time lie a whole number of bank rows apart and crowd some of the HBM channels: a read
// of 4 GiB in this pattern ran at 5.55 TB/s from a common k and at 6.35 TB/s from staggered ones.  Tiles of one
// expert keep step, since they share its weights and rows in L2.
constexpr int kStagger = 5;

struct GemmArgs {
    const char* a;
    int64_t a_stride;                 // bytes
    const char* w;
    int64_t w_stride_e, w_stride_r;   // bytes: expert, row of the bank
    int n_experts;
    int64_t N, K;
    const int32_t* offsets;
    int m_rows;
    int n_tiles;                      // N tiles
    int by_size;                      // whole tiles of all experts first, then the last ones by size
    int main_wgs;                     // by_size: workgroups of the launch that a tail launch follows, or 0
    int main_n_tiles;                 // and its N tiles
    void* out;
    int out_dt;
    int64_t out_stride;               // elements
};

// TAIL: the launch behind a by_size one of tiles twice as high.  It takes all last tiles of at most C::BP rows where with
// them the main launch would need more rounds than without, one or several, and is empty otherwise; both find out from
// the offsets.  A last round of few 256 x 256 tiles, with one step in flight each, waits for memory; 128 x 128
// tiles with three in flight share it among more workgroups: 8 experts of ragged rows, 16384 x 8192 to 4096 1026 -> 964
// us, one of 4200 rows, 8192 x 8192 544 -> 462, 16 of 2048 rows, 2048 x 2048 250 -> 252.  (Tail tiles of 128 x 256:
// 982 us, 481, 245.)  An empty tail costs about 1 % of 250 us.  Whole rounds of short tiles gain a little too: experts of
// 1100 rows, NT, in the tail and (where that holds no more than one round) in the main launch, 16 of 4096 x 4096 557 and
// 575 us, 32 of 2048 x 4096 565 and 585, 64 of them 1119 - 1199 and 1171 - 1177, 256 of 4096 x 2048 4718 and 4852; least
// where most of them would have fitted a round that is there already: 64 ragged experts (8.5 rounds and 1.1) 1179 and 1161.
template <class C, bool QT, bool F16, bool TAIL>
__global__ void __launch_bounds__(C::THREADS, C::WAVES_PER_EU) b16_gemm_kernel(const GemmArgs g) {
    using P = KMajor<C::BP, C::NW>;
    using Q = std::conditional_t<QT, TMajor<C::BQ, C::NW>, KMajor<C::BQ, C::NW>>;
    constexpr int S = C::S, STAGE = P::BYTES + Q::BYTES, LPS = P::LOADS + Q::LOADS;
    constexpr int TB = TAIL ? 2 * C::BP : C::BP;       // rows of the table's tiles
    __shared__ __attribute__((aligned(1024))) uint8_t ring[S * STAGE];
    // Before expert e: its rows, and the M tiles of three kinds ([n_experts] is the total): whole ones (BP rows),
    // and last ones of more and of at most BP / 2 rows.  (Not by_size: all of them are of the first kind.)
    __shared__ int first_row[kMaxExperts + 1], first_whole[kMaxExperts + 1];
    __shared__ uint16_t first_long[kMaxExperts + 1], first_short[kMaxExperts + 1];
    __shared__ int decreases;                          // offsets that are below the one before
    __shared__ uint32_t wave_sum[2 * C::NW];

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int E = g.n_experts;

    // the tile table: EPT consecutive experts per thread, a scan of the counts over the block (the two kinds of last
    // tiles and the decreases in one word, 11, 11 and 10 bits: an expert adds to one of them, so only 1024 decreases
    // could pass theirs, and then no expert has rows)
    {
        constexpr int EPT = kMaxExperts / C::THREADS;
        int whole[EPT];
        uint32_t last[EPT], sum_w = 0, sum_l = 0;
#pragma unroll
        for (int i = 0; i < EPT; i++) {
            const int e = tid * EPT + i;
            whole[i] = 0;
            last[i] = 0;
            if (e < E) {
                const int lo = min(max(g.offsets[e], 0), g.m_rows), to = min(max(g.offsets[e + 1], 0), g.m_rows), hi = max(to, lo);
                const int rest = g.by_size ? (hi - lo) % TB : 0;
                first_row[e] = lo;
                if (e == E - 1) first_row[E] = hi;
                whole[i] = pieces(hi - lo - rest, TB);
                last[i] = to < lo ? 1u << 22 : rest > TB / 2 ? 1u : rest > 0 ? 1u << 11 : 0u;
            }
            sum_w += whole[i];
            sum_l += last[i];
        }
        uint32_t w = sum_w, l = sum_l;
        block_exclusive_scan2<C::NW>(w, l, wave_sum, lane, wave);
#pragma unroll
        for (int i = 0; i < EPT; i++) {
            const int e = tid * EPT + i;
            if (e < E) {
                first_whole[e] = (int)w;
                first_long[e] = (uint16_t)(l & 0x7FFu);
                first_short[e] = (uint16_t)(l >> 11 & 0x7FFu);
            }
            w += whole[i];
            l += last[i];
            if (e == E - 1) {
                first_whole[E] = (int)w;
                first_long[E] = (uint16_t)(l & 0x7FFu);
                first_short[E] = (uint16_t)(l >> 11 & 0x7FFu);
                decreases = (int)(l >> 22);
            }
        }
        __syncthreads();
    }
    // Experts that overlap may have more tiles than the host counted on, and share rows: nothing is computed.
    if (__builtin_amdgcn_readfirstlane(decreases) != 0) return;
    const int whole_tiles = __builtin_amdgcn_readfirstlane(first_whole[E]);
    const int long_tiles = __builtin_amdgcn_readfirstlane(first_long[E]);
    const int short_tiles = __builtin_amdgcn_readfirstlane(first_short[E]);
    const int main_tiles = (whole_tiles + long_tiles) * g.main_n_tiles;
    const bool tail = g.main_wgs > 0 && ceil_div(main_tiles + short_tiles * g.main_n_tiles, g.main_wgs) > ceil_div(main_tiles, g.main_wgs);
    const int m_first = TAIL ? whole_tiles + long_tiles : 0;
    const int m_tiles = TAIL ? (tail ? short_tiles : 0) : whole_tiles + long_tiles + (tail ? 0 : short_tiles);
    const int tiles = m_tiles * g.n_tiles;
    const int G = gridDim.x;
    const int start = (int)(blockIdx.x % kXcds) * (G / kXcds) + (int)(blockIdx.x / kXcds);

    // Tile of this workgroup in round s.  The tiles that do not fill a last round go to the workgroups from the other
    // end: whole tiles come first, so those had the shorter tiles of the round before.
    auto tile_at = [&](int s) { return s * G + ((s + 1) * G > tiles ? G - 1 - start : start); };

    struct Tile {
        int expert, row0, rows, n0;
    };
    auto locate = [&](int t) {
        const int per = kPanel * g.n_tiles;
        const int panel = t / per, r = t - panel * per;
        const int height = min(kPanel, m_tiles - panel * kPanel);
        const int nt = r / height, mt = m_first + panel * kPanel + r - nt * height;
        // the last expert whose first tile of the kind is <= its number: the tile's expert
        const bool whole = mt < whole_tiles, is_long = mt < whole_tiles + long_tiles;
        const int k = whole ? mt : mt - whole_tiles - (is_long ? 0 : long_tiles);
        auto first = [&](int e) { return whole ? first_whole[e] : is_long ? (int)first_long[e] : (int)first_short[e]; };
        const int lo = last_at_most(first, E, k, lane);
        Tile ti;
        ti.expert = lo;
        const int from = __builtin_amdgcn_readfirstlane(first_row[lo]), end = __builtin_amdgcn_readfirstlane(first_row[lo + 1]);
        ti.row0 = whole ? from + (k - __builtin_amdgcn_readfirstlane(first(lo))) * TB : end - (end - from) % TB;
        ti.rows = min(end - ti.row0, C::BP);
        ti.n0 = nt * C::BQ;
        return ti;
    };

    const uint32_t lds = lds_offset(ring);
    const int steps = (int)((g.K + kStep - 1) / kStep);

    // Producer: the ring stage, tile and step that are requested next.  Past the last tile it goes on with zeros
    // (prod_k = 0) into stages that nobody reads, so the loads in flight can be counted the same way to the end.
    P p;
    Q q;
    int prod_t = tile_at(0), prod_round = 0, prod_left = 0, prod_kt = 0, prod_stage = 0;   // steps left of the tile, and the next one's k
    int64_t prod_k = 0;
    auto aim = [&]() {
        prod_k = prod_t < tiles ? g.K : 0;
        if (prod_t >= tiles) return;
        const Tile ti = locate(prod_t);
        const int l = fresh(lane);
        prod_left = steps;
        prod_kt = ti.expert * kStagger % steps;
        p.set(g.a + ti.row0 * g.a_stride, g.a_stride, ti.rows, wave, l);
        const char* w = g.w + ti.expert * g.w_stride_e;
        const int valid = (int)min(g.N - ti.n0, (int64_t)C::BQ);
        if constexpr (QT) q.set(w + (int64_t)ti.n0 * 2, g.w_stride_r, valid, wave, l);
        else q.set(w + ti.n0 * g.w_stride_r, g.w_stride_r, valid, wave, l);
    };
    auto part = [&](int j) {
        const uint32_t dst = lds + prod_stage * STAGE;
        if (j < P::LOADS) p.issue(j, dst, prod_kt, prod_k, wave, lane);
        else q.issue(j - P::LOADS, dst + P::BYTES, prod_kt, prod_k, wave, lane);
        if (j == LPS - 1) {
            prod_stage = prod_stage + 1 == S ? 0 : prod_stage + 1;
            prod_kt = prod_kt + 1 == steps ? 0 : prod_kt + 1;
            if (--prod_left <= 0) {
                prod_t = tile_at(++prod_round);
                aim();
            }
        }
    };
    auto produce = [&]() {
#pragma unroll
        for (int j = 0; j < LPS; j++) part(j);
    };
    if (tile_at(0) >= tiles) return;
    aim();
    constexpr bool PIPED = C::MP >= 4;                 // a wave's MFMAs are worth the software pipeline
#pragma unroll 1
    for (int i = 0; i < S - 1; i++) produce();

    typename P::Frag fp;
    typename Q::Frag fq;
    const int wp = wave / C::WQ, wq = wave % C::WQ;
    fp.set(wp * C::MP, lane);
    fq.set(wq * C::MQ, lane);

    int stage = 0;
    Frags<C::MQ> f;
    if constexpr (PIPED) {
        arrive<S, LPS>();
        f.first(fp, fq, lds, lds + P::BYTES);
#pragma unroll
        for (int j = 0; j < parts_per_group<C::MP, LPS>; j++) part(j);
    }
#pragma unroll 1
    for (int round = 0, t; (t = tile_at(round)) < tiles; round++) {
        const Tile ti = locate(t);
        const int rows = min(ti.rows, C::BP) - wp * C::MP * 16;       // of this wave
        const int subs = (rows + 15) / 16;
        v4f acc[C::MP][C::MQ];
#pragma unroll
        for (int m = 0; m < C::MP; m++)
#pragma unroll
            for (int n = 0; n < C::MQ; n++) acc[m][n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (PIPED) {
            // A wave with at most half its rows in use leaves the other half's MFMAs out (a tile's two wave rows share
            // their SIMDs, so a last tile of few rows takes about half the time).  Two loops in a row, of which one
            // runs: as branches of one loop they would keep two sets of accumulators.
            const bool half = C::MP == 8 && subs <= 4;
            uint32_t at = lds + stage * STAGE;
            auto next_stage = [&]() {
                stage = stage + 1 == S ? 0 : stage + 1;
                return lds + stage * STAGE;
            };
#pragma unroll 1
            for (int kt = half ? steps : 0; kt < steps; kt++) {
                const uint32_t next = next_stage();
                step_pipelined<C::MP, F16, S, LPS>(acc, f, fp, fq, at, at + P::BYTES, next, next + P::BYTES, part, [](int) {});
                at = next;
            }
            if constexpr (C::MP == 8) {
                static_assert(parts_per_group<C::MP, LPS> == parts_per_group<4, LPS>, "one phase of the parts");
#pragma unroll 1
                for (int kt = half ? 0 : steps; kt < steps; kt++) {
                    const uint32_t next = next_stage();
                    step_pipelined<4, F16, S, LPS>(acc, f, fp, fq, at, at + P::BYTES, next, next + P::BYTES, part, [](int) {});
                    at = next;
                }
            }
        } else {
#pragma unroll 1
            for (int kt = 0; kt < steps; kt++) {
                const uint32_t at = lds + stage * STAGE;
                stage = stage + 1 == S ? 0 : stage + 1;
                arrive<S, LPS>();
                produce();                             // into the stage that the step before this one read
                step_mfma<C::MP, C::MQ, F16>(acc, fp, fq, at, at + P::BYTES);
            }
        }
        const int64_t c0 = ti.n0 + wq * C::MQ * 16;
        const int cols = (int)min(g.N - c0, (int64_t)(C::MQ * 16));
        if (rows > 0 && cols > 0)
            store_wave_dt(g.out, g.out_dt, false, (ti.row0 + wp * C::MP * 16) * g.out_stride + c0, g.out_stride, rows, cols, acc, fresh(lane));
    }
    wait_loads<0>();                                   // no load may write LDS after the workgroup has left it
}

template <class C, bool QT, bool F16, bool TAIL>
int resident_blocks() {
    static std::atomic<int> cached[64];   // concurrent first calls may both fill it, with the same value
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
    int c = cached[dev].load(std::memory_order_relaxed);
    if (c == 0) {
        int per_cu = 0, cus = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, b16_gemm_kernel<C, QT, F16, TAIL>, C::THREADS, 0) != hipSuccess ||
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
using Tile64x64 = Cfg<64, 64, 2, 2, 4, 2>;
using Tile32x64 = Cfg<32, 64, 1, 4, 8, 1>;
using TileTail = Cfg<128, 128, 2, 4, 4, 1>;
static_assert(2 * TileTail::BP == Tile256::BP, "the tail takes the last tiles of at most half the rows");

template <class C, bool QT, bool F16>
int launch_cfg(hipStream_t st, GemmArgs g) {
    constexpr bool TAILED = std::is_same_v<C, Tile256>;
    const int64_t n_tiles = ceil_div(g.N, C::BQ);
    const int64_t most = (g.m_rows / C::BP + std::min<int64_t>(g.n_experts, g.m_rows)) * n_tiles;
    if (most > 0x7FFFFFFF - (1 << 20)) return MOE_ERR_SHAPE;
    int wgs = resident_blocks<C, QT, F16, false>() / kXcds * kXcds;
    if (wgs < kXcds) return MOE_ERR_HIP;
    wgs = (int)std::min<int64_t>(wgs, ceil_div(most, kXcds) * kXcds);
    g.n_tiles = (int)n_tiles;
    // only for experts of several whole tiles: an expert's last tile then reads its weights once more
    g.by_size = g.m_rows / g.n_experts >= 4 * C::BP;
    g.main_n_tiles = (int)n_tiles;
    g.main_wgs = TAILED && g.by_size ? wgs : 0;
    hipLaunchKernelGGL((b16_gemm_kernel<C, QT, F16, false>), dim3((unsigned)wgs), dim3(C::THREADS), 0, st, g);
    if constexpr (TAILED) {                            // E <= m_rows / 1024, so its tiles are at most half of `most`
        if (g.main_wgs > 0) {
            using T = TileTail;
            g.n_tiles = (int)ceil_div(g.N, T::BQ);
            int tail = resident_blocks<T, QT, F16, true>() / kXcds * kXcds;
            if (tail < kXcds) return MOE_ERR_HIP;
            tail = (int)std::min<int64_t>(tail, ceil_div((int64_t)g.n_experts * g.n_tiles, kXcds) * kXcds);
            hipLaunchKernelGGL((b16_gemm_kernel<T, QT, F16, true>), dim3((unsigned)tail), dim3(T::THREADS), 0, st, g);
        }
    }
    return launch_status();
}

template <class C>
int launch_form(hipStream_t st, bool trans, bool f16, const GemmArgs& g) {
    if (trans) return f16 ? launch_cfg<C, true, true>(st, g) : launch_cfg<C, true, false>(st, g);
    return f16 ? launch_cfg<C, false, true>(st, g) : launch_cfg<C, false, false>(st, g);
}


// The tile is the one with the least estimated time, in us: rounds of workgroups times (k steps times a step's time
// plus 4 for a tile's start and stores), but no less than the bytes at 5.7 TB/s.  A step's time and the workgroups
// that the device's 256 CUs hold are measured per tile; the tiles are estimated from rows per expert alone, since
// the counts are on the device.  Over 36 problems from 1 to 24576 rows and 1 to 256 experts the choice took 1.6 % more
// time than the best tile in the mean and 14 % at most; a rule by rows per expert alone (64, 128, 256 rows a tile up to
// 64, 256 and more) 25 % more in the mean and 2.9 times at most.
struct TileCost {
    int bp, bq, slots;
    double step;
};
constexpr TileCost kCosts[] = {{32, 64, 256, 0.28}, {64, 64, 512, 0.50}, {64, 256, 256, 0.68}, {128, 256, 256, 0.88}, {256, 256, 256, 1.45}};

int pick_tile(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K) {
    const double E = (double)n_experts, R = (double)m_rows, steps = (double)ceil_div(K, kStep);
    const double used = n_experts == 1 ? 1.0 : std::min(R, E * (1.0 - std::pow(1.0 - 1.0 / E, R)));   // experts with rows
    const double r = R / used;
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < 5; i++) {
        const TileCost& c = kCosts[i];
        const double per = n_experts == 1 ? std::ceil(r / c.bp) : (r <= 0.5 * c.bp ? 1.0 : r / c.bp + 0.5);   // M tiles of one
        const double tiles = used * per * (double)ceil_div(N, c.bq) * (n_experts == 1 ? 1.0 : 1.05);
        const double work = std::ceil(tiles / c.slots - 1e-9) * (steps * c.step + 4.0);
        const double bytes = used * (double)N * (double)K * 2.0 * std::ceil(per / kPanel) + R * (double)(K + N) * 2.0;
        const double t = std::max(work, bytes / 5.7e6) + 0.1 * work;
        if (i == 0 || t < least) {
            least = t;
            best = i;
        }
    }
    return best;
}

int grouped_launch(hipStream_t st, bool trans, bool f16, const GemmArgs& g) {
    switch (pick_tile(g.m_rows, g.n_experts, g.N, g.K)) {
        case 0: return launch_form<Tile32x64>(st, trans, f16, g);
        case 1: return launch_form<Tile64x64>(st, trans, f16, g);
        case 2: return launch_form<Tile64>(st, trans, f16, g);
        case 3: return launch_form<Tile128>(st, trans, f16, g);
        default: return launch_form<Tile256>(st, trans, f16, g);
    }
}

// ------------------------------------------------------------------ slot mode
// One wave holds COLS columns of one row: its lanes take 8 consecutive k each (512 a chunk), products and sums in fp32,
// and the lanes' sums meet in six shuffles.  Bound by streaming the row's expert, so a wave asks for UNROLL chunks of
// all its columns (8 KB of weights) at once before it multiplies: 8 routes of 1536 x 2048, one of them inactive, take
// 8.6 us a call (4.9 TB/s); 64 routes 67 us (5.9 TB/s), one row of 8192 x 8192 26 us.  Four columns a wave and a loop
// over single chunks took 77 and 48 us for these two.
constexpr int kSlotWaves = 4;

template <bool F16>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint16_t lo = (uint16_t)(w[i] & 0xFFFFu), hi = (uint16_t)(w[i] >> 16);
        x[2 * i] = F16 ? f16_to_f32(lo) : bf16_to_f32(lo);
        x[2 * i + 1] = F16 ? f16_to_f32(hi) : bf16_to_f32(hi);
    }
}

template <bool F16, int COLS, int UNROLL>
__global__ void __launch_bounds__(64 * kSlotWaves)
b16_slot_kernel(const GemmArgs g, const int32_t* __restrict__ slots, int64_t a_row_div, int col_groups) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t r = blockIdx.x / (unsigned)col_groups;
    const int64_t n0 = ((int64_t)(blockIdx.x % (unsigned)col_groups) * kSlotWaves + wave) * COLS;
    if (n0 >= g.N) return;                             // N is a multiple of COLS
    const int slot = slots[r];
    float sum[COLS] = {};
    if (slot >= 0 && slot < g.n_experts) {
        const char* x = g.a + (r / a_row_div) * g.a_stride;
        const char* w = g.w + slot * g.w_stride_e + n0 * g.w_stride_r;
        // UNROLL chunks from k0; in the last ones lanes past K read the last piece and count it as zero on both sides
        auto chunks = [&](int64_t k0, auto tail) {
            uint4 xv[UNROLL], wv[COLS][UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; u++) {
                int64_t k = k0 + u * (kWave * 8) + lane * 8;
                if (tail) k = k < g.K ? k : g.K - 8;
                xv[u] = *reinterpret_cast<const uint4*>(x + k * 2);
#pragma unroll
                for (int c = 0; c < COLS; c++) wv[c][u] = *reinterpret_cast<const uint4*>(w + c * g.w_stride_r + k * 2);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; u++) {
                const bool in = !tail || k0 + u * (kWave * 8) + lane * 8 < g.K;
                float xf[8];
                unpack8<F16>(in ? xv[u] : make_uint4(0u, 0u, 0u, 0u), xf);
#pragma unroll
                for (int c = 0; c < COLS; c++) {
                    float wf[8];
                    unpack8<F16>(in ? wv[c][u] : make_uint4(0u, 0u, 0u, 0u), wf);
#pragma unroll
                    for (int i = 0; i < 8; i++) sum[c] = __builtin_fmaf(wf[i], xf[i], sum[c]);
                }
            }
        };
        int64_t k0 = 0;
        for (; k0 + UNROLL * kWave * 8 <= g.K; k0 += UNROLL * kWave * 8) chunks(k0, std::false_type{});
        if (k0 < g.K) chunks(k0, std::true_type{});
#pragma unroll
        for (int c = 0; c < COLS; c++)
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum[c] += __shfl_xor(sum[c], d, kWave);
    }
    if (lane < COLS) {
        float v = sum[0];
#pragma unroll
        for (int c = 1; c < COLS; c++) v = lane == c ? sum[c] : v;
        const int64_t o = r * g.out_stride + n0 + lane;
        if (g.out_dt == MOE_F32) store_from_f32<kF32>(g.out, o, v);
        else if (g.out_dt == MOE_BF16) store_from_f32<kBF16>(g.out, o, v);
        else store_from_f32<kF16>(g.out, o, v);
    }
}

template <bool F16, int COLS, int UNROLL>
int slot_launch_cols(hipStream_t st, const GemmArgs& g, const int32_t* slots, int64_t a_row_div) {
    const int64_t groups = ceil_div(g.N, COLS * kSlotWaves);
    if (groups * g.m_rows >= ((int64_t)1 << 32) / (64 * kSlotWaves)) return MOE_ERR_SHAPE;   // a grid's threads fit 32 bits
    hipLaunchKernelGGL((b16_slot_kernel<F16, COLS, UNROLL>), dim3((unsigned)(groups * g.m_rows)), dim3(64 * kSlotWaves), 0, st, g,
                       slots, a_row_div, (int)groups);
    return launch_status();
}

// Up to 1024 k a row is two chunks, so a wave takes four columns of them; beyond, two columns of four chunks.
int slot_launch(hipStream_t st, bool f16, const GemmArgs& g, const int32_t* slots, int64_t a_row_div) {
    if (g.K <= 1024)
        return f16 ? slot_launch_cols<true, 4, 2>(st, g, slots, a_row_div) : slot_launch_cols<false, 4, 2>(st, g, slots, a_row_div);
    return f16 ? slot_launch_cols<true, 2, 4>(st, g, slots, a_row_div) : slot_launch_cols<false, 2, 4>(st, g, slots, a_row_div);
}

}  // namespace b16
}  // namespace moe

using namespace moe;

extern "C" int moe_b16_grouped_tile(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K, int32_t tile[2]) {
    if (!tile) return MOE_ERR_NULL;
    if (m_rows < 1 || m_rows > 0x7FFFFFFF || n_experts < 1 || n_experts > b16::kMaxExperts || N < 8 || N > b16::kMaxWidth ||
        N % 8 || K < 8 || K > b16::kMaxWidth || K % 8)
        return MOE_ERR_SHAPE;
    const b16::TileCost& c = b16::kCosts[b16::pick_tile(m_rows, n_experts, N, K)];
    tile[0] = c.bp;
    tile[1] = c.bq;
    return MOE_OK;
}

extern "C" int moe_b16_grouped_gemm(const void* a, int64_t a_stride, const void* w, int64_t w_stride_e,
                                    int64_t w_stride_r, int64_t n_experts, int64_t N, int64_t K, int dt, int w_trans,
                                    int mode, const int32_t* expert_offsets, const int32_t* slot_ids, int64_t m_rows,
                                    int64_t a_row_div, void* out, int out_dt, int64_t out_stride, void* stream) {
    if (mode != MOE_MODE_GROUPED && mode != MOE_MODE_SLOT) return MOE_ERR_SHAPE;
    if (w_trans != 0 && (w_trans != 1 || mode == MOE_MODE_SLOT)) return MOE_ERR_SHAPE;
    if ((dt != MOE_BF16 && dt != MOE_F16) || !dtype_ok(out_dt)) return MOE_ERR_DTYPE;
    if (m_rows < 0 || m_rows > 0x7FFFFFFF || n_experts < 0 || n_experts > 0x7FFFFFFF) return MOE_ERR_SHAPE;
    if (N < 8 || N > b16::kMaxWidth || N % 8 || K < 8 || K > b16::kMaxWidth || K % 8) return MOE_ERR_SHAPE;
    if (m_rows == 0) return MOE_OK;
    if (!out) return MOE_ERR_NULL;
    if (out_stride < N) return MOE_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(out) % (out_dt == MOE_F32 ? 4 : 2)) return MOE_ERR_ALIGN;
    if (n_experts > 0) {
        if (!a || !w) return MOE_ERR_NULL;
        const int64_t rows = w_trans ? K : N, width = w_trans ? N : K;
        if (a_stride < K || w_stride_r < width || (n_experts > 1 && w_stride_e / w_stride_r < rows)) return MOE_ERR_SHAPE;
        if (!aligned16(a) || !aligned16(w) || a_stride % 8 || w_stride_r % 8 || w_stride_e % 8) return MOE_ERR_ALIGN;
    }
    b16::GemmArgs g{};
    g.a = (const char*)a; g.a_stride = a_stride * 2;
    g.w = (const char*)w; g.w_stride_e = w_stride_e * 2; g.w_stride_r = w_stride_r * 2;
    g.n_experts = (int)n_experts; g.N = N; g.K = K; g.offsets = expert_offsets; g.m_rows = (int)m_rows;
    g.out = out; g.out_dt = out_dt; g.out_stride = out_stride;
    if (mode == MOE_MODE_SLOT) {
        if (!slot_ids) return MOE_ERR_NULL;
        if (a_row_div < 1) return MOE_ERR_SHAPE;
        return b16::slot_launch(as_stream(stream), dt == MOE_F16, g, slot_ids, a_row_div);
    }
    if (n_experts < 1 || n_experts > b16::kMaxExperts) return MOE_ERR_SHAPE;
    if (!expert_offsets) return MOE_ERR_NULL;
    return b16::grouped_launch(as_stream(stream), w_trans == 1, dt == MOE_F16, g);
}
