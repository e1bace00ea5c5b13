// Routing to experts in its general form, and the gradient of its logits.
//
// Per token: scores s_e (softmax over the experts, or the sigmoid of each logit), choices c_e = s_e + bias_e, the best
// groups of consecutive experts, the top-k of the choices among them, and the weights s_e of the chosen ones, renormalised
// or not, times a factor.  A logit of -inf (or NaN) masks its expert for that token.  Then the (expert, token)-ordered
// route maps of route_prep.hip over the routes there are.
//
// MI355X design.
//  * Choices are ranked as 64-bit keys: the order-preserving bits of the value above the inverted expert index, so one
//    unsigned compare is "larger value, ties to the lower index".  Without a bias the order is the logits' own, which needs
//    no exponential and is exact.  With one (or with group values that are sums) the scores are formed in 64 bits: in 32
//    bits about one token in ten thousand has two choices next to each other that round to the wrong order.
//  * Up to 64 experts a token takes 16 lanes of a wave, beyond a whole wave; lanes hold experts lane, lane + LPT, ... .
//    Round j takes the largest key below round j - 1's winner by DPP moves.
//  * A workgroup takes 16 tokens at a time and sets one bit per (expert, token) in LDS, whose counts are the chunk's loads.
//    Up to 64 tokens one workgroup does everything, maps included, in one launch.  Beyond, a second launch scatters: each of
//    its workgroups adds up the counts of all chunks (bytes) for the experts' offsets and of the chunks before its own
//    for its rows.  With more than kSumChunks chunks those sums come from a scan launched between.
#include <algorithm>

#include "device.h"
#include "host.h"

namespace moe {
namespace router {
namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxTopk = 64;
constexpr int kMaxGroups = 64;
constexpr int kTok = 16;                        // tokens of a workgroup at one time
constexpr int kSingle = 64;                     // tokens that one workgroup routes alone
constexpr int kSumChunks = 512;                 // chunks whose counts every scattering workgroup adds up itself
constexpr int kScatterThreads = 512;
constexpr int64_t kMaxT = 1 << 27;              // a chunk of 64 tokens is 1024 threads of a grid, which fit 32 bits

struct Args {
    const void* logits;
    int dt;
    int64_t stride;
    int T, E, topk, score;
    const float* bias;
    int n_group, keep, group_top, renorm;
    float scale;
    int32_t* ids;
    float* weights;
    float* scores;
    int32_t* dst2src;                           // all three maps or none
    int32_t* route_rows;
    int32_t* offsets;
    uint8_t* counts;                            // [chunk][experts rounded up to 16]
    int32_t* before;                            // [chunk][experts]: rows in earlier chunks; then [experts]: totals
    int chunk;                                  // tokens of a chunk
    int nc;
};

__host__ __device__ inline int row_bytes(int E) { return (E + 15) / 16 * 16; }

// A logit as the formulas take it: NaN masks as -inf does, +inf is the largest value.
__device__ __forceinline__ float shown(float v) { return v != v ? -__builtin_inff() : __builtin_fminf(v, 3.402823466e38f); }

__device__ __forceinline__ float load_logit(const Args& a, int64_t i) {
    if (a.dt == MOE_F32) return shown(load_as_f32<kF32>(a.logits, i));
    return shown(a.dt == MOE_BF16 ? load_as_f32<kBF16>(a.logits, i) : load_as_f32<kF16>(a.logits, i));
}

// Logits i * LPT + l of a row, -inf past the last expert (the row's last one is read there).
template <int DT, int LPT, int VPL>
__device__ __forceinline__ void load_row(const Args& a, int64_t row, int l, float (&v)[VPL]) {
    float x[VPL];
#pragma unroll
    for (int i = 0; i < VPL; i++) x[i] = load_as_f32<DT>(a.logits, row + min(i * LPT + l, a.E - 1));
#pragma unroll
    for (int i = 0; i < VPL; i++) v[i] = i * LPT + l < a.E ? shown(x[i]) : -__builtin_inff();
}

// Order-preserving maps to unsigned, larger value -> larger code; -0 as +0.
__device__ __forceinline__ uint32_t mono32(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t mono64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
// The ten lowest bits of a 64-bit value give way to the index, the others rounded to nearest: 43 significant bits.  (Cut off,
// values that are equal but for their last rounding, such as sums s(x) + s(-x) = 1, would fall on either side of 1.)
constexpr uint64_t kLow = 1023;
__device__ __forceinline__ uint64_t value_key(double c, int i) { return ((mono64(c) + (kLow + 1) / 2) & ~kLow) | (kLow - (uint64_t)i); }
__device__ __forceinline__ uint64_t logit_key(float v, int e) { return ((uint64_t)mono32(v) << 32) | (kLow - (uint64_t)e); }
__device__ __forceinline__ int key_index(uint64_t key) { return (int)(kLow - (key & kLow)); }

template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)x, CTRL, ROW_MASK, 0xF, false);
}
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint64_t max_step(uint64_t k) {
    const uint64_t o = ((uint64_t)dpp<CTRL, ROW_MASK>((uint32_t)(k >> 32), (uint32_t)(k >> 32)) << 32) |
                       dpp<CTRL, ROW_MASK>((uint32_t)k, (uint32_t)k);
    return o > k ? o : k;
}
// The largest key over the LPT lanes of a token, in every one of them.
template <int LPT>
__device__ __forceinline__ uint64_t token_max(uint64_t k) {
    k = max_step<0xB1>(k);                      // quad_perm [1,0,3,2], [2,3,0,1], half-mirror, mirror: a row of 16
    k = max_step<0x4E>(k);
    k = max_step<0x141>(k);
    k = max_step<0x140>(k);
    if constexpr (LPT == 64) {
        k = max_step<0x142, 0xA>(k);            // row_bcast:15, row_bcast:31: the wave's in lane 63
        k = max_step<0x143, 0xC>(k);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), 63);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, 63);
        k = ((uint64_t)hi << 32) | lo;
    }
    return k;
}
template <int LPT, class T>
__device__ __forceinline__ T token_sum(T x) {
#pragma unroll
    for (int m = 1; m < LPT; m <<= 1) x += __shfl_xor(x, m, kWave);
    return x;
}
template <int LPT>
__device__ __forceinline__ float token_fmax(float x) {
#pragma unroll
    for (int m = 1; m < LPT; m <<= 1) x = __builtin_fmaxf(x, __shfl_xor(x, m, kWave));
    return x;
}

__device__ __forceinline__ double sigmoid64(double l) {
    const double t = exp(-fabs(l)), r = 1.0 / (1.0 + t);
    return l >= 0.0 ? r : t * r;
}
__device__ __forceinline__ float sigmoid32(float l) {
    const float t = expf(-__builtin_fabsf(l)), r = 1.0f / (1.0f + t);
    return l >= 0.0f ? r : t * r;
}

// LDS of a token while it is routed.
struct TokenLds {
    uint64_t top1[kMaxGroups], top2[kMaxGroups];     // keys of each group's two largest choices
    double val1[kMaxGroups], val2[kMaxGroups];       // and, for their sum, the choices
    int32_t id[kMaxTopk];
};

// Routes token t with the LPT lanes of which this is `l`; ids go to lds.id and, with the weights, to memory.
template <int LPT, int VPL, bool WIDE>
__device__ __forceinline__ void route_token(const Args& a, int t, int l, TokenLds& lds) {
    constexpr float kInf = __builtin_inff();
    const int64_t row = (int64_t)t * a.stride;
    float v[VPL];
    if (a.dt == MOE_F32) load_row<kF32, LPT>(a, row, l, v);
    else if (a.dt == MOE_BF16) load_row<kBF16, LPT>(a, row, l, v);
    else load_row<kF16, LPT>(a, row, l, v);
    float top = v[0];
#pragma unroll
    for (int i = 1; i < VPL; i++) top = __builtin_fmaxf(top, v[i]);
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    double z64 = 0.0;
    float z = 0.0f;
    if (softmax) {
        top = token_fmax<LPT>(top);
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < VPL; i++) z64 += v[i] > -kInf ? exp((double)v[i] - (double)top) : 0.0;
            z64 = token_sum<LPT>(z64);
            z = (float)z64;
        } else if (a.scores || !a.renorm) {
#pragma unroll
            for (int i = 0; i < VPL; i++) z += v[i] > -kInf ? expf(v[i] - top) : 0.0f;
            z = token_sum<LPT>(z);
        }
    }
    if (a.scores) {
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = i * LPT + l;
            const float s = v[i] > -kInf ? (softmax ? expf(v[i] - top) / z : sigmoid32(v[i])) : 0.0f;
            if (e < a.E) a.scores[(int64_t)t * a.E + e] = s;
        }
    }
    uint64_t key[VPL];
    double choice[WIDE ? VPL : 1];
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = i * LPT + l;
        if constexpr (WIDE) {
            double c = softmax ? exp((double)v[i] - (double)top) / z64 : sigmoid64((double)v[i]);
            if (a.bias) c += (double)a.bias[e < a.E ? e : a.E - 1];
            const bool there = v[i] > -kInf && c > -(double)kInf;            // false for NaN too
            key[i] = there ? value_key(c, e) : 0ull;
            choice[i] = c;
        } else {
            key[i] = v[i] > -kInf ? logit_key(v[i], e) : 0ull;
        }
    }
    if (a.n_group > 1) {                        // the best groups stay
        const int size = a.E / a.n_group;
        for (int g = l; g < a.n_group; g += LPT) lds.top1[g] = lds.top2[g] = 0ull;
        wave_lds_fence();
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (key[i]) atomicMax((unsigned long long*)&lds.top1[(i * LPT + l) / size], (unsigned long long)key[i]);
        wave_lds_fence();
        if constexpr (WIDE) {
            if (a.group_top == 2) {
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    const int g = (i * LPT + l) / size;
                    if (key[i] && key[i] == lds.top1[g]) lds.val1[g] = choice[i];
                    else if (key[i]) atomicMax((unsigned long long*)&lds.top2[g], (unsigned long long)key[i]);
                }
                wave_lds_fence();
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    const int g = (i * LPT + l) / size;
                    if (key[i] && key[i] == lds.top2[g]) lds.val2[g] = choice[i];
                }
                wave_lds_fence();
            }
        }
        uint64_t gk[kMaxGroups / LPT];
#pragma unroll
        for (int j = 0; j < kMaxGroups / LPT; j++) {
            const int g = j * LPT + l;
            gk[j] = 0ull;
            if (g < a.n_group && lds.top1[g]) {
                gk[j] = lds.top1[g];            // its index orders ties by group as well
                if (WIDE && a.group_top == 2) gk[j] = value_key(lds.top2[g] ? lds.val1[g] + lds.val2[g] : lds.val1[g], g);
            }
        }
        uint64_t kept = 0ull, prev = ~0ull;
        for (int n = 0; n < a.keep; n++) {
            uint64_t best = 0ull;
#pragma unroll
            for (int j = 0; j < kMaxGroups / LPT; j++) best = gk[j] < prev && gk[j] > best ? gk[j] : best;
            best = token_max<LPT>(best);
            if (best == 0ull) break;            // the same in the token's lanes; other tokens of the wave go on
            prev = best;
            kept |= 1ull << (WIDE && a.group_top == 2 ? key_index(best) : key_index(best) / size);
        }
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (!((kept >> ((i * LPT + l) / size & 63)) & 1ull)) key[i] = 0ull;
        if constexpr (WIDE) {
            if (!a.bias) {                      // the groups went by scores, the order within them is the logits' own
#pragma unroll
                for (int i = 0; i < VPL; i++) key[i] = key[i] ? logit_key(v[i], i * LPT + l) : 0ull;
            }
        }
        wave_lds_fence();
    }
    uint64_t prev = ~0ull;
    for (int j = 0; j < a.topk; j++) {
        uint64_t f[VPL];                        // candidates of this round, then a depth-log2(VPL) max tree
#pragma unroll
        for (int i = 0; i < VPL; i++) f[i] = key[i] < prev ? key[i] : 0ull;
#pragma unroll
        for (int w = VPL / 2; w >= 1; w /= 2)
#pragma unroll
            for (int i = 0; i < w; i++) f[i] = f[i] > f[i + w] ? f[i] : f[i + w];
        const uint64_t best = token_max<LPT>(f[0]);
        prev = best ? best : 1ull;              // none left: every later round finds none
        if (l == 0) lds.id[j] = best == 0ull ? -1 : key_index(best);
    }
    wave_lds_fence();
    // the weights, in 64 bits: lane l takes routes l, l + LPT, ...
    constexpr int RPL = kMaxTopk / LPT;
    float lg[RPL];
    double w[RPL], sum = 0.0;
    float most = -kInf;
#pragma unroll
    for (int j = 0; j < RPL; j++) {
        const int r = j * LPT + l;
        const int id = r < a.topk ? lds.id[r] : -1;
        lg[j] = id >= 0 ? load_logit(a, row + id) : -kInf;
        most = __builtin_fmaxf(most, lg[j]);
    }
    if (a.renorm) {                             // ratios of scores: scaled by the largest one, nothing underflows as a whole
        most = token_fmax<LPT>(most);
        const float low = softmax ? most : __builtin_fminf(most, 0.0f);
#pragma unroll
        for (int j = 0; j < RPL; j++) {
            const double x = (double)lg[j];
            w[j] = 0.0;
            if (lg[j] > -kInf) {
                w[j] = exp(lg[j] >= 0.0f && !softmax ? 0.0 : x - (double)low);
                if (!softmax) w[j] /= 1.0 + exp(-fabs(x));
            }
            sum += w[j];
        }
        sum = token_sum<LPT>(sum);
    } else {
#pragma unroll
        for (int j = 0; j < RPL; j++) {
            const double x = (double)lg[j];
            w[j] = lg[j] > -kInf ? (softmax ? exp(x - (double)top) : sigmoid64(x)) : 0.0;
        }
        sum = softmax ? (WIDE ? z64 : (double)z) : 1.0;
    }
#pragma unroll
    for (int j = 0; j < RPL; j++) {
        const int r = j * LPT + l;
        if (r < a.topk) {
            a.ids[(int64_t)t * a.topk + r] = lds.id[r];
            a.weights[(int64_t)t * a.topk + r] = lg[j] > -kInf ? (float)((double)a.scale * w[j] / sum) : 0.0f;
        }
    }
}

// Exclusive scan of one int per thread over a block of THREADS; every thread gets the total too.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* lds, int& total) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    int x = v;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int y = __shfl_up(x, d, kWave);
        if (lane >= d) x += y;
    }
    if (lane == kWave - 1) lds[wave] = x;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWave; w++) {
        if (w < wave) base += lds[w];
        total += lds[w];
    }
    __syncthreads();
    return base + x - v;
}

// SINGLE: one workgroup, T <= kSingle, maps too.  Else chunk blockIdx.x, whose counts are written when maps are wanted.
template <int LPT, int VPL, bool WIDE, bool SINGLE>
__global__ void __launch_bounds__(kTok * LPT) route_kernel(const Args a) {
    constexpr int THREADS = kTok * LPT;
    __shared__ TokenLds tok[kTok];
    __shared__ uint64_t mask[SINGLE ? kMaxE : 1];      // the tokens of each expert
    __shared__ uint32_t count[SINGLE ? 1 : kMaxE];
    __shared__ int32_t all_ids[SINGLE ? kSingle * kMaxTopk : 1];
    __shared__ int32_t first[SINGLE ? kMaxE : 1];
    __shared__ int sums[THREADS / kWave];
    const int l = threadIdx.x % LPT, w = threadIdx.x / LPT;
    const int t0 = blockIdx.x * a.chunk;
    const int n_tok = min(a.chunk, a.T - t0);
    for (int i = threadIdx.x; i < a.E; i += THREADS) {
        if constexpr (SINGLE) mask[i] = 0ull;
        else count[i] = 0u;
    }
    __syncthreads();
    for (int i = 0; i < n_tok; i += kTok) {
        if (i + w < n_tok) {                           // whole tokens are active or idle together
            const int t = t0 + i + w;
            route_token<LPT, VPL, WIDE>(a, t, l, tok[w]);
            for (int j = l; j < a.topk; j += LPT) {
                const int e = tok[w].id[j];
                if constexpr (SINGLE) {
                    all_ids[t * a.topk + j] = e;
                    if (e >= 0) atomicOr((unsigned long long*)&mask[e], 1ull << t);
                } else if (e >= 0) {
                    atomicAdd(&count[e], 1u);
                }
            }
            wave_lds_fence();                          // the ids are read before the next token's
        }
    }
    if (!a.dst2src) return;
    __syncthreads();
    if constexpr (!SINGLE) {
        uint8_t* out = a.counts + (int64_t)blockIdx.x * row_bytes(a.E);
        for (int i = threadIdx.x; i < row_bytes(a.E); i += THREADS) out[i] = i < a.E ? (uint8_t)count[i] : 0;
    } else {
        int base = 0;
        for (int e0 = 0; e0 < a.E; e0 += THREADS) {
            const int e = e0 + threadIdx.x;
            const int mine = e < a.E ? __popcll(mask[e]) : 0;
            int total;
            const int at = base + block_scan<THREADS>(mine, sums, total);
            if (e < a.E) {
                first[e] = at;
                a.offsets[e] = at;
            }
            base += total;
        }
        if (threadIdx.x == 0) a.offsets[a.E] = base;
        __syncthreads();
        for (int i = threadIdx.x; i < a.T * a.topk; i += THREADS) {
            const int t = i / a.topk, e = all_ids[i];
            int row = -1;
            if (e >= 0) {
                row = first[e] + __popcll(mask[e] & ((1ull << t) - 1ull));
                a.dst2src[row] = t;
            }
            a.route_rows[i] = row;
            if (i >= base) a.dst2src[i] = -1;
        }
    }
}

// Column sums over the chunks for many chunks: four experts a thread, one workgroup per 64 threads' experts.
__global__ void __launch_bounds__(256) scan_kernel(const Args a) {
    __shared__ int4 part[4][kWave];
    const int rw = row_bytes(a.E);
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int e = (blockIdx.x * kWave + lane) * 4;
    const int per = (a.nc + 3) / 4, c0 = wave * per, c1 = min(c0 + per, a.nc);
    int4 s = make_int4(0, 0, 0, 0);
    if (e < rw)
        for (int c = c0; c < c1; c++) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(a.counts + (int64_t)c * rw + e);
            s.x += v & 255u; s.y += v >> 8 & 255u; s.z += v >> 16 & 255u; s.w += v >> 24;
        }
    part[wave][lane] = s;
    __syncthreads();
    int4 run = make_int4(0, 0, 0, 0);
    for (int w = 0; w < wave; w++) {
        const int4 p = part[w][lane];
        run.x += p.x; run.y += p.y; run.z += p.z; run.w += p.w;
    }
    if (e >= rw) return;
    for (int c = c0; c < c1; c++) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(a.counts + (int64_t)c * rw + e);
        *reinterpret_cast<int4*>(a.before + (int64_t)c * rw + e) = run;
        run.x += v & 255u; run.y += v >> 8 & 255u; run.z += v >> 16 & 255u; run.w += v >> 24;
    }
    if (wave == 3) *reinterpret_cast<int4*>(a.before + (int64_t)a.nc * rw + e) = run;
}

// Chunk blockIdx.x's routes to their rows.
template <bool SCANNED>
__global__ void __launch_bounds__(kScatterThreads) scatter_kernel(const Args a) {
    __shared__ int total[kMaxE], base[kMaxE];
    __shared__ uint64_t mask[kMaxE];
    __shared__ int sums[kScatterThreads / kWave];
    const int rw = row_bytes(a.E), c = blockIdx.x;
    const int t0 = c * a.chunk, n_tok = min(a.chunk, a.T - t0), n = n_tok * a.topk;
    const int32_t* ids = a.ids + (int64_t)t0 * a.topk;
    for (int e = threadIdx.x; e < a.E; e += kScatterThreads) {
        total[e] = SCANNED ? a.before[(int64_t)a.nc * rw + e] : 0;
        base[e] = SCANNED ? a.before[(int64_t)c * rw + e] : 0;
        mask[e] = 0ull;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kScatterThreads) {
        const int e = ids[i];
        if (e >= 0) atomicOr((unsigned long long*)&mask[e], 1ull << (i / a.topk));
    }
    if constexpr (!SCANNED) {
        // 16 experts a thread and load; sums of bytes as 16-bit pairs (at most 512 chunks of at most 64 tokens)
        const int quads = rw / 16, parts = kScatterThreads / quads;
        const int qd = threadIdx.x % quads, part = threadIdx.x / quads;
        if (part < parts) {
            uint32_t lo[4] = {}, hi[4] = {}, blo[4] = {}, bhi[4] = {};
            for (int cc = part; cc < a.nc; cc += parts) {
                const uint4 x = *reinterpret_cast<const uint4*>(a.counts + (int64_t)cc * rw + qd * 16);
                const uint32_t v[4] = {x.x, x.y, x.z, x.w};
                const uint32_t early = cc < c ? 0xFFFFFFFFu : 0u;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint32_t even = v[k] & 0x00FF00FFu, odd = v[k] >> 8 & 0x00FF00FFu;
                    lo[k] += even;
                    hi[k] += odd;
                    blo[k] += even & early;
                    bhi[k] += odd & early;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int e = qd * 16 + 4 * k;
#pragma unroll
                for (int b = 0; b < 4; b++) {
                    const uint32_t s = (b & 1 ? hi[k] : lo[k]) >> (b & 2 ? 16 : 0) & 0xFFFFu;
                    const uint32_t f = (b & 1 ? bhi[k] : blo[k]) >> (b & 2 ? 16 : 0) & 0xFFFFu;
                    if (e + b < a.E && s) {
                        atomicAdd(&total[e + b], (int)s);
                        if (f) atomicAdd(&base[e + b], (int)f);
                    }
                }
            }
        }
    }
    __syncthreads();
    int run = 0;
    for (int e0 = 0; e0 < a.E; e0 += kScatterThreads) {
        const int e = e0 + threadIdx.x;
        const int mine = e < a.E ? total[e] : 0;
        int sum;
        const int at = run + block_scan<kScatterThreads>(mine, sums, sum);
        if (e < a.E) {
            base[e] += at;
            if (c == 0) a.offsets[e] = at;
        }
        run += sum;
    }
    if (c == 0 && threadIdx.x == 0) a.offsets[a.E] = run;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kScatterThreads) {
        const int tt = i / a.topk, e = ids[i];
        int row = -1;
        if (e >= 0) {
            row = base[e] + __popcll(mask[e] & ((1ull << tt) - 1ull));
            a.dst2src[row] = t0 + tt;
        }
        a.route_rows[(int64_t)t0 * a.topk + i] = row;
    }
    // the rows behind the last route name no token
    const int64_t all = (int64_t)a.T * a.topk;
    for (int64_t i = run + (int64_t)c * kScatterThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kScatterThreads)
        a.dst2src[i] = -1;
}

__global__ void zero_offsets_kernel(int E, int32_t* offsets) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

int chunk_of(int64_t T) { return T <= kSingle ? kSingle : T <= (int64_t)kTok * kSumChunks ? kTok : 64; }

template <int LPT, int VPL, bool WIDE>
void launch_route(hipStream_t st, const Args& a) {
    const dim3 block(kTok * LPT);
    if (a.T <= kSingle) hipLaunchKernelGGL((route_kernel<LPT, VPL, WIDE, true>), dim3(1), block, 0, st, a);
    else hipLaunchKernelGGL((route_kernel<LPT, VPL, WIDE, false>), dim3((unsigned)a.nc), block, 0, st, a);
}

template <bool WIDE>
void launch_route_e(hipStream_t st, const Args& a) {
    if (a.E <= 64) launch_route<16, 4, WIDE>(st, a);
    else if (a.E <= 256) launch_route<64, 4, WIDE>(st, a);
    else if (a.E <= 512) launch_route<64, 8, WIDE>(st, a);
    else launch_route<64, 16, WIDE>(st, a);
}

// ------------------------------------------------------------------ the gradient
struct BackArgs {
    const void* logits;
    int dt;
    int64_t stride;
    const int32_t* ids;
    const float* weights;
    const float* dweights;
    const float* dscores;
    int64_t dscores_stride;
    int64_t T;
    int E, topk, score, renorm;
    float scale;
    void* dlogits;
    int64_t dlogits_stride;
};

// One wave per token; lane j holds route j, lanes hold experts lane, lane + 64, ... .  With u_e = dL/ds_e (the weights'
// part of a form that is not renormalised, and the auxiliary loss's), d l_e = s_e (u_e - sum s u) for the softmax and
// u_e s_e (1 - s_e) for the sigmoid.  A renormalised weight w_j = scale n_j, n_j = s_j / sum s, adds
// scale n_j (dw_j - sum n dw), times 1 - s_j for the sigmoid: the sum of the scores cancels.
// DENSE: every entry has a gradient, so all logits are read; else only the chosen ones' (sigmoid).
template <int DT, int VPL, bool DENSE>
__global__ void __launch_bounds__(256) route_back_kernel(const BackArgs a) {
    constexpr float kInf = __builtin_inff();
    const int lane = threadIdx.x & (kWave - 1);
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    for (int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; t < a.T; t += (int64_t)gridDim.x * 4) {
        const int64_t row = t * a.stride;
        auto logit = [&](int e) { return shown(load_as_f32<DT>(a.logits, row + e)); };
        const int id = lane < a.topk ? a.ids[t * a.topk + lane] : -1;
        const bool on = id >= 0 && id < a.E;
        const float dw = on ? a.dweights[t * a.topk + lane] : 0.0f;
        float give = 0.0f;                             // this route's part: of d l (renormalised), else of u
        if (a.renorm) {
            const float nj = on ? a.weights[t * a.topk + lane] / a.scale : 0.0f;
            const float mean = nj * dw;
            float sum = mean;
#pragma unroll
            for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m, kWave);
            give = a.scale * nj * (dw - sum);
            if (!softmax && on) {
                const float x = logit(id), tt = expf(-__builtin_fabsf(x)), r = 1.0f / (1.0f + tt);
                give *= x >= 0.0f ? tt * r : r;
            }
        } else {
            give = a.scale * dw;
            if (!DENSE && on) {                        // a sigmoid without an auxiliary loss
                const float tt = expf(-__builtin_fabsf(logit(id))), r = 1.0f / (1.0f + tt);
                give *= tt * r * r;
            }
        }
        float part[VPL];
#pragma unroll
        for (int i = 0; i < VPL; i++) part[i] = 0.0f;
        for (int j = 0; j < a.topk; j++) {
            const int idj = __builtin_amdgcn_readlane(id, j);
            const float gj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, give), j));
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (idj == i * kWave + lane) part[i] += gj;
        }
        float d[VPL];
        if constexpr (DENSE) {
            float v[VPL], u[VPL], top = -kInf;
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int e = i * kWave + lane;
                v[i] = e < a.E ? logit(e) : -kInf;
                u[i] = a.dscores && e < a.E ? a.dscores[t * a.dscores_stride + e] : 0.0f;
                if (!a.renorm) u[i] += part[i];
                top = __builtin_fmaxf(top, v[i]);
            }
            if (softmax) {
#pragma unroll
                for (int m = 32; m > 0; m >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, m, kWave));
                float z = 0.0f, zu = 0.0f;
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    v[i] = v[i] > -kInf ? expf(v[i] - top) : 0.0f;
                    z += v[i];
                    zu += v[i] > 0.0f ? v[i] * u[i] : 0.0f;
                }
#pragma unroll
                for (int m = 32; m > 0; m >>= 1) {
                    z += __shfl_xor(z, m, kWave);
                    zu += __shfl_xor(zu, m, kWave);
                }
                const float inv = z > 0.0f ? 1.0f / z : 0.0f, mean = zu * inv;
#pragma unroll
                for (int i = 0; i < VPL; i++) d[i] = v[i] > 0.0f ? v[i] * inv * (u[i] - mean) : 0.0f;
            } else {
#pragma unroll
                for (int i = 0; i < VPL; i++) {
                    const float tt = expf(-__builtin_fabsf(v[i])), r = 1.0f / (1.0f + tt);
                    d[i] = v[i] > -kInf ? u[i] * (tt * r * r) : 0.0f;
                }
            }
            if (a.renorm) {
#pragma unroll
                for (int i = 0; i < VPL; i++) d[i] += part[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < VPL; i++) d[i] = part[i];
        }
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = i * kWave + lane;
            if (e < a.E) store_from_f32<DT>(a.dlogits, t * a.dlogits_stride + e, d[i]);
        }
    }
}

template <int DT, bool DENSE>
void launch_back_e(hipStream_t st, const BackArgs& a) {
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div(a.T, 4), 1 << 20)), block(256);
    if (a.E <= 256) hipLaunchKernelGGL((route_back_kernel<DT, 4, DENSE>), grid, block, 0, st, a);
    else if (a.E <= 512) hipLaunchKernelGGL((route_back_kernel<DT, 8, DENSE>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((route_back_kernel<DT, 16, DENSE>), grid, block, 0, st, a);
}

template <int DT>
void launch_back(hipStream_t st, const BackArgs& a) {
    const bool dense = a.dscores || (!a.renorm && a.score == MOE_SCORE_SOFTMAX);
    if (dense) launch_back_e<DT, true>(st, a);
    else launch_back_e<DT, false>(st, a);
}

bool sizes_ok(int64_t T, int64_t E, int64_t topk) {
    return T >= 0 && T <= kMaxT && E >= 1 && E <= kMaxE && topk >= 1 && topk <= std::min<int64_t>(E, kMaxTopk) && T <= 0x7FFFFFFF / topk;
}

bool scale_ok(float scale) { return scale > 0.0f && scale <= 3.402823466e38f; }

bool natural(const void* p, int dt) { return reinterpret_cast<uintptr_t>(p) % (dt == MOE_F32 ? 4 : 2) == 0; }

}  // namespace
}  // namespace router
}  // namespace moe

using namespace moe;

extern "C" size_t moe_router_workspace_size(int64_t T, int64_t E) {
    if (T <= router::kSingle || T > router::kMaxT || E < 1 || E > router::kMaxE) return 0;
    const int64_t nc = ceil_div(T, router::chunk_of(T)), rw = router::row_bytes((int)E);
    const int64_t bytes = nc * rw + (nc > router::kSumChunks ? (nc + 1) * rw * 4 : 0);
    return (size_t)ceil_div(bytes, 256) * 256;
}

extern "C" int moe_router(const void* logits, int dt, int64_t logits_stride, int64_t T, int64_t E, int64_t topk, int score,
                          const float* bias, int64_t n_group, int64_t topk_group, int group_top, int renorm, float scale,
                          int32_t* expert_ids, float* weights, float* scores, int32_t* dst2src, int32_t* route_rows,
                          int32_t* expert_offsets, void* workspace, size_t ws_bytes, void* stream) {
    if (!dtype_ok(dt)) return MOE_ERR_DTYPE;
    if (!router::sizes_ok(T, E, topk) || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)) return MOE_ERR_SHAPE;
    if (n_group < 1 || n_group > std::min<int64_t>(E, router::kMaxGroups) || E % n_group || topk_group < 1 || topk_group > n_group ||
        topk > topk_group * (E / n_group) || (group_top != 1 && group_top != 2) || (renorm != 0 && renorm != 1) || !router::scale_ok(scale))
        return MOE_ERR_SHAPE;
    const bool maps = dst2src || route_rows || expert_offsets;
    if (maps && (!expert_offsets || (T > 0 && (!dst2src || !route_rows)))) return MOE_ERR_NULL;
    auto st = as_stream(stream);
    if (T == 0) {
        if (!maps) return MOE_OK;
        hipLaunchKernelGGL(router::zero_offsets_kernel, dim3(1), dim3(1024), 0, st, (int)E, expert_offsets);
        return launch_status();
    }
    if (!logits || !expert_ids || !weights) return MOE_ERR_NULL;
    if (logits_stride < E) return MOE_ERR_SHAPE;
    if (!router::natural(logits, dt)) return MOE_ERR_ALIGN;
    router::Args a{};
    a.logits = logits; a.dt = dt; a.stride = logits_stride;
    a.T = (int)T; a.E = (int)E; a.topk = (int)topk; a.score = score; a.bias = bias;
    a.n_group = topk_group < n_group ? (int)n_group : 1;
    a.keep = (int)topk_group; a.group_top = group_top; a.renorm = renorm; a.scale = scale;
    a.ids = expert_ids; a.weights = weights; a.scores = scores; a.dst2src = dst2src; a.route_rows = route_rows; a.offsets = expert_offsets;
    a.chunk = router::chunk_of(T);
    a.nc = (int)ceil_div(T, a.chunk);
    if (maps && T > router::kSingle) {
        if (!workspace) return MOE_ERR_NULL;
        if (ws_bytes < moe_router_workspace_size(T, E)) return MOE_ERR_WORKSPACE;
        if (!aligned16(workspace)) return MOE_ERR_ALIGN;
        a.counts = (uint8_t*)workspace;
        a.before = (int32_t*)(a.counts + (int64_t)a.nc * router::row_bytes((int)E));
    }
    if (bias || (a.n_group > 1 && group_top == 2)) router::launch_route_e<true>(st, a);
    else router::launch_route_e<false>(st, a);
    if (maps && T > router::kSingle) {
        const dim3 grid((unsigned)a.nc), block(router::kScatterThreads);
        if (a.nc > router::kSumChunks) {
            hipLaunchKernelGGL(router::scan_kernel, dim3((unsigned)ceil_div(router::row_bytes((int)E), 4 * kWave)), dim3(256), 0, st, a);
            hipLaunchKernelGGL((router::scatter_kernel<true>), grid, block, 0, st, a);
        } else {
            hipLaunchKernelGGL((router::scatter_kernel<false>), grid, block, 0, st, a);
        }
    }
    return launch_status();
}

extern "C" int moe_router_backward(const void* logits, int dt, int64_t logits_stride, const int32_t* expert_ids, const float* weights,
                                   const float* dweights, const float* dscores, int64_t dscores_stride, int64_t T, int64_t E,
                                   int64_t topk, int score, int renorm, float scale, void* dlogits, int64_t dlogits_stride,
                                   void* stream) {
    if (!dtype_ok(dt)) return MOE_ERR_DTYPE;
    if (!router::sizes_ok(T, E, topk) || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) || (renorm != 0 && renorm != 1) ||
        !router::scale_ok(scale))
        return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!logits || !expert_ids || !weights || !dweights || !dlogits) return MOE_ERR_NULL;
    if (logits_stride < E || dlogits_stride < E || (dscores && dscores_stride != 0 && dscores_stride < E)) return MOE_ERR_SHAPE;
    if (!router::natural(logits, dt) || !router::natural(dlogits, dt)) return MOE_ERR_ALIGN;
    const router::BackArgs a{logits, dt, logits_stride, expert_ids, weights, dweights, dscores, dscores_stride, T, (int)E, (int)topk, score,
                             renorm, scale, dlogits, dlogits_stride};
    auto st = as_stream(stream);
    if (dt == MOE_F32) router::launch_back<kF32>(st, a);
    else if (dt == MOE_BF16) router::launch_back<kBF16>(st, a);
    else router::launch_back<kF16>(st, a);
    return launch_status();
}
