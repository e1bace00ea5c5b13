// Routing to experts in its general form, and the gradient of its logits.
//
// Per token: scores s_e (softmax over the experts, or the sigmoid of each logit), choices c_e = s_e + bias_e, the best
// groups of consecutive experts, the top-k of the choices among them, and the weights s_e of the chosen ones, renormalised
// or not, times a factor.  A logit of -inf (or NaN) masks its expert for that token.  Then the (expert, token)-ordered
// route maps of route_prep.hip over the routes there are.
//
// MI355X design.
//  * What is ranked: the choice's order-preserving bits above the inverted expert index, so one unsigned compare is "larger
//    value, ties to the lower index".  Without a bias the order is the logits' own, which needs no exponential.  With one (or
//    with group values that are sums) scores have to be formed in 64 bits, for in 32 about one token in ten thousand has two
//    choices next to each other that round to the wrong order; but 64-bit exponentials and 64-bit keys for every expert took
//    86 us where this takes 39 (16384 tokens, 512 experts).  So keys are 32 bits: 22-bit steps over the token's own range, formed
//    with 32-bit scores whose error is known in steps.  Where two keys that matter are closer than that, the candidates alone
//    are ranked again in 64 bits: of experts (refine, one token in a hundred) or groups (exact_groups, one in ten thousand).
//    What even that leaves open, and tokens whose range has no such steps, are ranked as a whole, one after the other
//    (rank_exact).  16-bit logits fit a key as they are.
//  * Up to 64 experts a token takes 16 lanes of a wave, beyond a whole wave; lanes hold experts lane, lane + LPT, ... .
//    Every round's largest key is found by lane moves folded into the maximum, then struck out.
//  * A workgroup takes 16 tokens at a time and counts its routes in LDS, the chunk's loads.  Up to 64 tokens (32 of more than
//    64 experts) one workgroup does everything, maps included, in one launch.  Beyond, a second launch scatters: each of its
//    workgroups adds up the counts of all chunks (bytes) for the experts' offsets and of the chunks before its own for its
//    rows.  With more than kSumChunks chunks those sums come from a scan launched between.
//  * Bound by instruction issue and the latency of the rounds, not by bytes: 4096 tokens of 256 fp32 logits in 8 groups with
//    maps take 16.4 us in two launches (790 vector instructions a token), 16384 of 512 bf16 ones with their
//    scores 39 us in two (50 MB: 1.3 TB/s), eight of 64 experts 7.3 us, which is the call (5.9 in a graph).
#include <algorithm>
#include <type_traits>

#include "device.h"
#include "host.h"

namespace moe {
namespace router {
namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxTopk = 64;
constexpr int kMaxGroups = 64;
constexpr int kTok = 16;                        // tokens of a workgroup at one time (TOK: of the only one, where a token takes 16 lanes)
constexpr int kWaves = 16;                      // of a workgroup at most
constexpr int kSingle = 64;                     // tokens that one workgroup routes alone, with up to 64 experts
constexpr int kSingleWide = 32;                 // with more, a wave a token
constexpr int kSumChunks = 512;                 // chunks whose counts every scattering workgroup adds up itself
constexpr int kScatterThreads = 1024;
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

// Logits i * LPT + l of a row as they are; past the last expert the row's last one.
template <int LPT, int VPL>
__device__ __forceinline__ void load_row(const Args& a, int t, int l, float (&v)[VPL]) {
    const int64_t row = (int64_t)t * a.stride;
    auto as = [&](auto type) {
#pragma unroll
        for (int i = 0; i < VPL; i++) v[i] = load_as_f32<decltype(type)::value>(a.logits, row + min(i * LPT + l, a.E - 1));
    };
    if (a.dt == MOE_F32) as(std::integral_constant<int, kF32>{});
    else if (a.dt == MOE_BF16) as(std::integral_constant<int, kBF16>{});
    else as(std::integral_constant<int, kF16>{});
}

__device__ __forceinline__ float load_logit(const Args& a, int64_t i) {
    if (a.dt == MOE_F32) return load_as_f32<kF32>(a.logits, i);
    return a.dt == MOE_BF16 ? load_as_f32<kBF16>(a.logits, i) : load_as_f32<kF16>(a.logits, i);
}

// Order-preserving maps to unsigned, larger value -> larger code; -0 as +0.
__device__ __forceinline__ uint32_t mono32(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_mono32(uint32_t u) { return __uint_as_float(u >> 31 ? u & 0x7FFFFFFFu : ~u); }
__device__ __forceinline__ uint64_t mono64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double from_mono64(uint64_t u) {
    return __longlong_as_double((long long)(u >> 63 ? u & 0x7FFFFFFFFFFFFFFFull : ~u));
}
// The ten lowest bits of a 64-bit value give way to the index, the others rounded to nearest: 43 significant bits.  (Cut off,
// values that are equal but for their last rounding, such as sums s(x) + s(-x) = 1, would fall on either side of 1.)
constexpr uint64_t kLow = 1023;
__device__ __forceinline__ uint64_t value_key(double c, int i) { return ((mono64(c) + (kLow + 1) / 2) & ~kLow) | (kLow - (uint64_t)i); }
__device__ __forceinline__ uint64_t logit_key(float v, int e) { return ((uint64_t)mono32(v) << 32) | (kLow - (uint64_t)e); }
__device__ __forceinline__ int key_index(uint64_t key) { return (int)(kLow - (key & kLow)); }

// Lane moves; a lane that a move leaves out (ROW_MASK) keeps `old`.  (Told that nothing is out of bounds, the compiler folds a
// move into the operation that uses it.)
template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t old, uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)x, CTRL, ROW_MASK, 0xF, ROW_MASK == 0xF);
}
// f over the LPT lanes of a token, f commutative with the neutral word `none`; in every one of them.
template <int LPT, class F>
__device__ __forceinline__ uint32_t token_reduce(uint32_t x, uint32_t none, const F& f) {
    x = f(x, dpp<0xB1>(none, x));               // quad_perm [1,0,3,2], [2,3,0,1], half-mirror, mirror: a row of 16
    x = f(x, dpp<0x4E>(none, x));
    x = f(x, dpp<0x141>(none, x));
    x = f(x, dpp<0x140>(none, x));
    if constexpr (LPT == 64) {
        x = f(x, dpp<0x142, 0xA>(none, x));     // row_bcast:15, row_bcast:31: the wave's in lane 63
        x = f(x, dpp<0x143, 0xC>(none, x));
        x = (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
    }
    return x;
}
template <int LPT>
__device__ __forceinline__ uint32_t token_umax(uint32_t x) {
    return token_reduce<LPT>(x, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LPT>
__device__ __forceinline__ float token_fmax(float x) { return from_mono32(token_umax<LPT>(mono32(x))); }
template <int LPT>
__device__ __forceinline__ float token_fsum(float x) {
    return __uint_as_float(token_reduce<LPT>(__float_as_uint(x), 0u, [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
// The larger and the smaller of two numbers that are no NaN, in one instruction each.
__device__ __forceinline__ float larger(float x, float y) { return __builtin_amdgcn_fmed3f(x, y, __builtin_inff()); }
__device__ __forceinline__ float smaller(float x, float y) { return __builtin_amdgcn_fmed3f(x, y, -__builtin_inff()); }

__device__ __forceinline__ double sigmoid64(double l) {
    const double t = exp(-fabs(l)), r = 1.0 / (1.0 + t);
    return l >= 0.0 ? r : t * r;
}
// From the hardware exp2 and reciprocal, within an ulp each: e^x for x <= 0 is within (1.25 |x| + 2) 2^-24 of itself (a
// difference as x adds |x| by its rounding).
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }
__device__ __forceinline__ float fast_score(float l) {
    const float t = fast_exp(-__builtin_fabsf(l)), r = __builtin_amdgcn_rcpf(1.0f + t);
    return l >= 0.0f ? r : t * r;
}
__device__ __forceinline__ float sigmoid32(float l) {
    const float t = expf(-__builtin_fabsf(l)), r = 1.0f / (1.0f + t);
    return l >= 0.0f ? r : t * r;
}

// e^(x - y) for x <= y, the difference as an exact sum of two floats, so that its rounding does not scale with it.  Below -104
// (half a step of 2^-149 is e^-103.97) it is 0 by itself: d may have overflowed there, which leaves no number in `rest`.
__device__ __forceinline__ float exp_of_difference(float x, float y) {
    const float d = x - y, yy = x - d, xx = d + yy;
    const float rest = (x - xx) + (yy - y);
    return d < -104.0f ? 0.0f : expf(d) * (1.0f + rest);
}

// What a lane needs of its experts for every token: their biases and groups.
template <int VPL>
struct LaneExperts {
    float bias[VPL];
    int group[VPL];
};

template <int LPT, int VPL>
__device__ __forceinline__ LaneExperts<VPL> lane_experts(const Args& a, int l) {
    LaneExperts<VPL> x;
#pragma unroll
    for (int i = 0; i < VPL; i++) x.bias[i] = a.bias ? a.bias[min(i * LPT + l, a.E - 1)] : 0.0f;
    // (e + 1/2) / size is at least 1/2048 away from a whole number and below 64, 1 / size within 2^-22 of itself
    const float per = __builtin_amdgcn_rcpf((float)(a.E / a.n_group));
#pragma unroll
    for (int i = 0; i < VPL; i++) x.group[i] = min((int)(((float)(i * LPT + l) + 0.5f) * per), kMaxGroups - 1);   // (past E: no key)
    return x;
}

// The groups' largest choices while a token is ranked, and their values' keys where 32 bits are too few.
struct GroupLds {
    uint32_t top1[kMaxGroups], top2[kMaxGroups], top3[kMaxGroups];
    uint64_t key[kMaxGroups];
};

// What a token's scores are made of: its logits in this lane (-inf: masked), their largest, and the softmax's sum.
template <int VPL>
struct TokenScores {
    float v[VPL];
    float top, z;
};

// ---------------------------------------------------------------- ranking in 32 bits
// Values as 22-bit steps over the token's range, the index below: ranks are one unsigned compare and two values closer than
// `near` steps may stand in the wrong order.  Where that is so the token is ranked again in 64 bits (rank_wide).
struct Steps {
    float lo, inv;
    uint32_t near;
    bool fine;
};

// lo is the smallest value (`all`: groups add values up, or few lanes), else the smallest of the lanes' largest: those below it,
// cut to step 0, are hardly ever among the first.  A value x may be off by tol + 2^-23 |x|.
template <int LPT, int VPL>
__device__ __forceinline__ Steps steps_of(const float (&c)[VPL], bool all, float tol) {
    constexpr float kInf = __builtin_inff();
    float most = c[0], least = kInf;
#pragma unroll
    for (int i = 1; i < VPL; i++) most = larger(most, c[i]);
    if (all) {
#pragma unroll
        for (int i = 0; i < VPL; i++) least = smaller(least, c[i] > -kInf ? c[i] : kInf);
    } else {
        least = most > -kInf ? most : kInf;
    }
    const float hi = token_fmax<LPT>(most);
    Steps s;
    s.lo = -token_fmax<LPT>(-least);
    const float range = hi - s.lo;
    s.inv = 4194301.0f * __builtin_amdgcn_rcpf(range);                 // (a step's width need not be exact)
    s.fine = (range > 1e-30f && range < 1e30f) || hi == -kInf;         // no expert at all: nothing to rank
    tol = 2.0f * (tol + 0x1p-23f * larger(__builtin_fabsf(hi), __builtin_fabsf(s.lo)));
    s.near = hi > -kInf ? (uint32_t)smaller(tol * s.inv, 1e9f) + 3u : 0u;
    return s;
}
__device__ __forceinline__ uint32_t step_key(const Steps& s, float c, int e) {
    const float q = (c - s.lo) * s.inv;
    return c > -__builtin_inff() ? (((uint32_t)larger(q, 0.0f) + 1u) << 10) | (1023u - (uint32_t)e) : 0u;
}
// A 16-bit logit's own order, exact: equal logits are true ties.  (+inf, fp32's largest value here, is above each type's largest
// finite one: the conversions round it up to the type's infinity, bf16's by half a step, which changes no other value.)
__device__ __forceinline__ uint32_t half_key(float v, bool bf16, int e) {
    uint32_t u;
    if (bf16) u = (__float_as_uint(v + 0.0f) + 0x8000u) >> 16;
    else u = f32_to_f16(v + 0.0f);
    u = u >> 15 ? 0xFFFFu & ~u : u | 0x8000u;
    return v > -__builtin_inff() ? ((u + 1u) << 10) | (1023u - (uint32_t)e) : 0u;
}

// In 64 bits: the softmax's sum over all of a token's experts, and the choice of expert e with logit v (without a bias: its score).
template <int LPT>
__device__ __forceinline__ double exact_sum(const Args& a, int64_t row, int l, float top) {
    double z = 0.0;
#pragma unroll 1
    for (int e = l; e < a.E; e += LPT) {
        const float v = shown(load_logit(a, row + e));
        z += v > -__builtin_inff() ? exp((double)v - (double)top) : 0.0;
    }
#pragma unroll
    for (int m = 1; m < LPT; m <<= 1) z += __shfl_xor(z, m, kWave);
    return z;
}
template <bool SOFT>
__device__ __forceinline__ double exact_choice(const Args& a, int e, float v, float top, double z) {
    const double s = SOFT ? exp((double)v - (double)top) / z : sigmoid64((double)v);
    return a.bias ? s + (double)a.bias[e] : s;
}

// The groups that stay, by sums of two choices in 64 bits (0: a third choice of some group may be one of its two largest).
// One pass more over the keys finds the third ones: `largest`.
template <int LPT, bool SOFT, class Largest>
__device__ __forceinline__ uint64_t exact_groups(const Args& a, int64_t row, int l, float top, uint32_t near, GroupLds& lds, const Largest& largest) {
    for (int g = l; g < a.n_group; g += LPT) lds.top3[g] = 0u;
    wave_lds_fence();
    largest(lds.top3, 2);
    const double z = SOFT ? exact_sum<LPT>(a, row, l, top) : 1.0;
    uint32_t unsure = 0u;
#pragma unroll 1
    for (int g = l; g < a.n_group; g += LPT) {
        const uint32_t k2 = lds.top2[g], k3 = lds.top3[g];
        if (k3 && (k2 >> 10) - (k3 >> 10) <= near) unsure = 1u;
        double sum = 0.0;
        uint32_t k = lds.top1[g];
        const bool some = k != 0u;
#pragma unroll 1
        for (int i = 0; i < 2 && k; i++, k = k2) {
            const int e = (int)(1023u - (k & 1023u));
            sum += exact_choice<SOFT>(a, e, shown(load_logit(a, row + e)), top, z);
        }
        lds.key[g] = some ? value_key(sum, g) : 0ull;
    }
    wave_lds_fence();
    if (token_umax<LPT>(unsure)) return 0ull;
    uint64_t kept = 0ull, prev = ~0ull;
    for (int n = 0; n < a.keep; n++) {
        uint64_t best = 0ull;
        for (int g = l; g < a.n_group; g += LPT) {
            const uint64_t k = lds.key[g];
            best = k < prev && k > best ? k : best;
        }
        const uint32_t hi = token_umax<LPT>((uint32_t)(best >> 32));
        const uint32_t lo = token_umax<LPT>((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        prev = (uint64_t)hi << 32 | lo;
        if (!prev) break;
        kept |= 1ull << key_index(prev);
    }
    return kept;
}

// Ranks the token's experts by 32-bit keys: lane l gets the keys of ranks l, l + LPT, ... (0: none).  Of the n keys every other
// expert is surely below; `close` if some of them may stand in the wrong order.  False if the groups, or more than 64 values,
// are too near.
template <int LPT, int VPL, bool WIDE, bool SOFT, bool GROUPS>
__device__ __forceinline__ bool rank_fast(const Args& a, int64_t row, const LaneExperts<VPL>& x, const TokenScores<VPL>& s, int l, GroupLds& lds,
                                          uint32_t (&mine)[kMaxTopk / LPT], int& n, bool& close) {
    constexpr float kInf = __builtin_inff();
    const bool halves = a.dt != MOE_F32;
    uint32_t key[VPL];
    uint32_t near = 0u;
    bool fine = true;
    auto by_logit = [&]() {
        if (halves) {
#pragma unroll
            for (int i = 0; i < VPL; i++) key[i] = half_key(s.v[i], a.dt == MOE_BF16, i * LPT + l);
            near = 0u;
        } else {
            const Steps st = steps_of<LPT, VPL>(s.v, LPT == 16, 0.0f);
#pragma unroll
            for (int i = 0; i < VPL; i++) key[i] = step_key(st, s.v[i], i * LPT + l);
            near = st.near;
            fine = fine && st.fine;
        }
    };
    if constexpr (WIDE) {
        constexpr bool softmax = SOFT;
        const float inv = softmax ? __builtin_amdgcn_rcpf(s.z) : 1.0f;
        float c[VPL];
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            c[i] = (softmax ? fast_exp(s.v[i] - s.top) * inv : fast_score(s.v[i])) + x.bias[i];
            c[i] = s.v[i] > -kInf && c[i] > -kInf ? c[i] : -kInf;
        }
        // In units of 2^-24, with the hardware exp2 and reciprocal: a sigmoid is off by t (1.25 |x| + 2) / (1 + t)^2 < 1 for t, 1
        // for 1 + t, 2 for its reciprocal, 1 for the product.  A softmax score is inv at most and off by inv times: e^-d (2.25 d +
        // 2) < 3, 2 for the reciprocal, 1 for the product, and for the sum 2.25 ln E + 2 < 18 and 22 additions: 46 of the 64 that
        // are allowed.  Then the bias's addition rounds.
        const Steps st = steps_of<LPT, VPL>(c, GROUPS || LPT == 16, softmax ? 0x1p-18f * inv : 0x1p-21f);
#pragma unroll
        for (int i = 0; i < VPL; i++) key[i] = step_key(st, c[i], i * LPT + l);
        near = st.near;
        fine = st.fine;
    } else {
        by_logit();
    }
    if constexpr (GROUPS) {
        const int size = a.E / a.n_group;
        uint32_t* top1 = lds.top1;
        uint32_t* top2 = lds.top2;
        for (int g = l; g < a.n_group; g += LPT) top1[g] = top2[g] = 0u;
        wave_lds_fence();
        // groups of whole rows of 16 lanes: a row's largest by lane moves, then one lane of it goes to LDS
        const bool rows = LPT == 64 && size % 16 == 0;
        auto largest = [&](uint32_t* to, int rank) {            // of what is left without the `rank` larger ones
#pragma unroll
            for (int i = 0; i < VPL; i++) {
                const int g = x.group[i];
                uint32_t k = key[i];
                if (rank > 0) k = k == top1[g] ? 0u : k;
                if (rank > 1) k = k == top2[g] ? 0u : k;
                if (rows) {
                    k = token_reduce<16>(k, 0u, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
                    if ((l & 15) == 0 && k) atomicMax(&to[g], k);
                } else if (k) {
                    atomicMax(&to[g], k);
                }
            }
            wave_lds_fence();
        };
        largest(top1, 0);
        const bool two = WIDE && a.group_top == 2;
        if (two) largest(top2, 1);
        uint32_t gk[kMaxGroups / LPT];
        bool lone = false;
#pragma unroll
        for (int j = 0; j < kMaxGroups / LPT; j++) {
            const int g = j * LPT + l;
            const uint32_t k1 = g < a.n_group ? top1[g] : 0u;
            if (two) {
                const uint32_t k2 = g < a.n_group ? top2[g] : 0u;
                lone = lone || (k1 && !k2);                       // a group with one expert: its value is no sum
                gk[j] = k1 ? (((k1 >> 10) + (k2 >> 10)) << 6) | (63u - (uint32_t)g) : 0u;
            } else {
                // (the group's index in the low six bits; its first expert's orders ties the same way)
                gk[j] = k1 ? (k1 >> 10 << 6) | (63u - (uint32_t)g) : 0u;
            }
        }
        bool unsure = token_umax<LPT>(lone ? 1u : 0u) != 0u;
        uint64_t kept = 0ull;
        uint32_t last = 0u;
        for (int n = 0; n <= a.keep; n++) {
            uint32_t best = 0u;
#pragma unroll
            for (int j = 0; j < kMaxGroups / LPT; j++) best = gk[j] > best ? gk[j] : best;
            best = token_umax<LPT>(best);
            if (n == a.keep) {
                if (near && best && last && (last >> 6) - (best >> 6) <= 2u * near) unsure = true;
            } else {
                if (best) kept |= 1ull << (63u - (best & 63u));
                last = best;
#pragma unroll
                for (int j = 0; j < kMaxGroups / LPT; j++) gk[j] = gk[j] == best ? 0u : gk[j];
            }
        }
        if (unsure) {
            kept = 0ull;
            if constexpr (WIDE) {
                if (two && fine) kept = exact_groups<LPT, SOFT>(a, row, l, s.top, near, lds, largest);
            }
            fine = fine && kept != 0ull;
        }
        if constexpr (WIDE) {
            if (!a.bias) {                      // the groups went by scores, the order within them is the logits' own
                uint32_t there = 0u;
#pragma unroll
                for (int i = 0; i < VPL; i++) there |= key[i] ? 1u << i : 0u;
                by_logit();
#pragma unroll
                for (int i = 0; i < VPL; i++) key[i] = there >> i & 1u ? key[i] : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if (!((kept >> x.group[i]) & 1ull)) key[i] = 0u;
        wave_lds_fence();
    }
#pragma unroll
    for (int q = 0; q < kMaxTopk / LPT; q++) mine[q] = 0u;
    uint32_t last = 0u;
    close = false;
    for (n = 0; n < a.topk || near; n++) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < VPL; i++) best = key[i] > best ? key[i] : best;
        best = token_umax<LPT>(best);
        const bool same = near && best && last && (last >> 10) - (best >> 10) <= near;
        if (n >= a.topk && !same) break;
        if (n >= kMaxTopk) return false;
        close = close || same;
        last = best;
#pragma unroll
        for (int i = 0; i < VPL; i++) key[i] = key[i] == best ? 0u : key[i];
#pragma unroll
        for (int q = 0; q < kMaxTopk / LPT; q++) mine[q] = n == q * LPT + l ? best : mine[q];
    }
    return fine;
}

// ---------------------------------------------------------------- ranking in 64 bits
// Puts the first n keys of a token into their right order (about one token in a hundred has two that stand too close).
template <int LPT, bool WIDE, bool SOFT>
__device__ __forceinline__ void refine(const Args& a, int64_t row, int l, float top, int n, GroupLds& lds, uint32_t (&mine)[kMaxTopk / LPT]) {
    constexpr int RPL = kMaxTopk / LPT;
    const bool by_choice = WIDE && a.bias;
    const double z = by_choice && SOFT ? exact_sum<LPT>(a, row, l, top) : 1.0;
    uint64_t key[RPL];
    int rank[RPL];
#pragma unroll
    for (int q = 0; q < RPL; q++) {
        const int e = (int)(1023u - (mine[q] & 1023u));
        key[q] = 0ull;
        if (mine[q]) {
            const float v = shown(load_logit(a, row + e));
            key[q] = by_choice ? value_key(exact_choice<SOFT>(a, e, v, top, z), e) : logit_key(v, e);
        }
        rank[q] = 0;
    }
#pragma unroll
    for (int q = 0; q < RPL; q++)
        for (int j = 0; j < LPT && q * LPT + j < n; j++) {
            uint64_t k;
            if constexpr (LPT == kWave)
                k = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(key[q] >> 32), j) << 32 |
                    (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key[q], j);
            else
                k = (uint64_t)__shfl((long long)key[q], j, LPT);
#pragma unroll
            for (int p = 0; p < RPL; p++) rank[p] += k > key[p] ? 1 : 0;
        }
#pragma unroll
    for (int q = 0; q < RPL; q++)
        if (mine[q]) lds.top1[rank[q]] = mine[q];
    wave_lds_fence();
#pragma unroll
    for (int q = 0; q < RPL; q++)
        if (mine[q]) mine[q] = lds.top1[q * LPT + l];   // (the keys there are lead)
}

// All of a token in 64 bits, where it has a great many close candidates or its range has no 22-bit steps: the workgroup takes one
// at a time, an expert a thread, 6 to 8 us each.  Hardly a token of random logits needs it, but whole batches can:
// fp32 logits (or biased scores) that are all equal, one choosable expert a token, and fp32 logits ranked without a bias, or
// biases, among which some are the type's lowest value in place of -inf.  Then 4096 tokens of 256 experts take 96 to 135 us
// instead of 14, 64 of 64 (one workgroup) 340 to 460 instead of 10; -inf as the mask, and 16-bit logits without a bias, stay with
// the 32-bit keys.
struct ExactLds {
    uint64_t top1[kMaxGroups], top2[kMaxGroups];     // each group's largest key; for sums its two largest choices, all their bits
    int32_t owner[kMaxGroups];                       // the expert whose choice the largest is
    uint64_t part[2][kWaves];
    int32_t id[kMaxTopk];
    float logit[kMaxTopk];                           // of the chosen experts
};

// The largest key of the workgroup.  `turn` alternates, so that the parts of one call are read before the next but one's.
template <int THREADS>
__device__ __forceinline__ uint64_t block_max(uint64_t k, ExactLds& lds, int& turn) {
    // the largest upper half, then the largest lower half among those that have it
    auto wave_max = [](uint64_t k) {
        const uint32_t hi = token_umax<kWave>((uint32_t)(k >> 32));
        const uint32_t lo = token_umax<kWave>((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
        return (uint64_t)hi << 32 | lo;
    };
    uint64_t* part = lds.part[turn];
    turn ^= 1;
    k = wave_max(k);
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = k;
    __syncthreads();
    return wave_max(part[threadIdx.x % (THREADS / kWave)]);
}

// Ranks token t: ids and logits of the ranks to lds.id and lds.logit, the softmax's largest logit and sum to top and z.
template <int THREADS, bool WIDE>
__device__ __forceinline__ void rank_exact(const Args& a, int t, ExactLds& lds, float& top, float& z) {
    constexpr float kInf = __builtin_inff();
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    const int e = threadIdx.x, wave = threadIdx.x / kWave;
    const float v = e < a.E ? shown(load_logit(a, (int64_t)t * a.stride + e)) : -kInf;
    int turn = 0;
    double sum = 1.0;
    top = 0.0f;
    if (softmax) {
        top = from_mono32((uint32_t)block_max<THREADS>(mono32(v), lds, turn));
        double part = v > -kInf ? exp((double)v - (double)top) : 0.0;
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1) part += __shfl_xor(part, m, kWave);
        uint64_t* parts = lds.part[turn];
        turn ^= 1;
        if (threadIdx.x % kWave == 0) parts[wave] = (uint64_t)__double_as_longlong(part);
        __syncthreads();
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < THREADS / kWave; w++) sum += __longlong_as_double((long long)parts[w]);
    }
    z = (float)sum;
    double c = 0.0;                             // the choice
    uint64_t key = 0ull;
    if (v > -kInf) {
        if constexpr (WIDE) {
            c = softmax ? exp((double)v - (double)top) / sum : sigmoid64((double)v);
            if (a.bias) c += (double)a.bias[e];
            key = c > -(double)kInf ? value_key(c, e) : 0ull;                       // (no key for NaN either)
        } else {
            key = logit_key(v, e);
        }
    }
    if (a.n_group > 1) {                        // the best groups stay
        const int size = a.E / a.n_group, g = min(e / size, kMaxGroups - 1);
        const bool two = WIDE && a.group_top == 2;
        if (e < a.n_group) {
            lds.top1[e] = lds.top2[e] = 0ull;
            lds.owner[e] = kMaxE;
        }
        __syncthreads();
        // (a key would leave it to the index which of two choices that are one value in 43 bits enters the sum)
        const uint64_t entry = key ? (two ? mono64(c) : key) : 0ull;
        if (entry) atomicMax((unsigned long long*)&lds.top1[g], (unsigned long long)entry);
        __syncthreads();
        if (two) {
            if (entry && entry == lds.top1[g]) atomicMin(&lds.owner[g], e);
            __syncthreads();
            if (entry && lds.owner[g] != e) atomicMax((unsigned long long*)&lds.top2[g], (unsigned long long)entry);
            __syncthreads();
        }
        uint64_t gk = 0ull;
        if (e < a.n_group && lds.top1[e]) {
            gk = lds.top1[e];                   // its index orders ties by group as well
            if (two) gk = value_key(lds.top2[e] ? from_mono64(lds.top1[e]) + from_mono64(lds.top2[e]) : from_mono64(lds.top1[e]), e);
        }
        uint64_t kept = 0ull;
        for (int n = 0; n < a.keep; n++) {
            const uint64_t best = block_max<THREADS>(gk, lds, turn);
            if (best == 0ull) break;
            gk = gk == best ? 0ull : gk;
            kept |= 1ull << (two ? key_index(best) : key_index(best) / size);
        }
        if (!(kept >> g & 1ull)) key = 0ull;
        if constexpr (WIDE) {
            if (!a.bias && key) key = logit_key(v, e);   // the groups went by scores, the order within them is the logits' own
        }
    }
    for (int j = 0; j < a.topk; j++) {
        const uint64_t best = block_max<THREADS>(key, lds, turn);
        if (best ? key == best : e == 0) {
            lds.id[j] = best ? e : -1;
            lds.logit[j] = v;
            key = 0ull;
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- a token
// Scores' statistics of a token's logits in its lanes; the scores to memory where they are wanted.
template <int LPT, int VPL, bool WIDE, bool SOFT>
__device__ __forceinline__ void score_token(const Args& a, const float (&v)[VPL], int t, int l, TokenScores<VPL>& s) {
    constexpr float kInf = __builtin_inff();
#pragma unroll
    for (int i = 0; i < VPL; i++) s.v[i] = i * LPT + l < a.E ? shown(v[i]) : -kInf;
    constexpr bool softmax = SOFT;
    s.top = 0.0f;
    s.z = 1.0f;
    if (softmax && (WIDE || a.scores || !a.renorm)) {
        float top = s.v[0];
#pragma unroll
        for (int i = 1; i < VPL; i++) top = larger(top, s.v[i]);
        s.top = token_fmax<LPT>(top);
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; i++) z += s.v[i] > -kInf ? fast_exp(s.v[i] - s.top) : 0.0f;
        s.z = token_fsum<LPT>(z);
    }
    if (a.scores) {
        const float inv = 1.0f / s.z;
#pragma unroll
        for (int i = 0; i < VPL; i++) {
            const int e = i * LPT + l;
            const float p = s.v[i] > -kInf ? (softmax ? fast_exp(s.v[i] - s.top) * inv : fast_score(s.v[i])) : 0.0f;
            if (e < a.E) a.scores[(int64_t)t * a.E + e] = p;
        }
    }
}

// Ids and weights of token t to memory: lane l has the ids (-1: none) and logits (-inf then) of routes l, l + LPT, ... .
template <int LPT, bool SOFT>
__device__ __forceinline__ void weigh_token(const Args& a, int t, int l, const int (&id)[kMaxTopk / LPT], const float (&lg)[kMaxTopk / LPT],
                                            float top, float z) {
    constexpr float kInf = __builtin_inff();
    constexpr int RPL = kMaxTopk / LPT;
    constexpr bool softmax = SOFT;
    float w[RPL], sum = 0.0f;
    if (a.renorm) {                             // ratios of scores: scaled by the largest one, nothing underflows as a whole
        float most = lg[0];
#pragma unroll
        for (int j = 1; j < RPL; j++) most = larger(most, lg[j]);
        most = token_fmax<LPT>(most);
        const float low = softmax ? most : smaller(most, 0.0f);
#pragma unroll
        for (int j = 0; j < RPL; j++) {
            w[j] = 0.0f;
            if (lg[j] > -kInf) {
                w[j] = lg[j] >= 0.0f && !softmax ? 1.0f : exp_of_difference(lg[j], low);
                if (!softmax) w[j] /= 1.0f + expf(-__builtin_fabsf(lg[j]));
            }
            sum += w[j];
        }
        sum = token_fsum<LPT>(sum);
    } else {
#pragma unroll
        for (int j = 0; j < RPL; j++) w[j] = lg[j] > -kInf ? (softmax ? exp_of_difference(lg[j], top) : sigmoid32(lg[j])) : 0.0f;
        sum = softmax ? z : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < RPL; j++) {
        const int r = j * LPT + l;
        if (r < a.topk) {
            a.ids[(int64_t)t * a.topk + r] = id[j];
            a.weights[(int64_t)t * a.topk + r] = lg[j] > -kInf ? a.scale * (w[j] / sum) : 0.0f;
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

// SINGLE: one workgroup, maps too.  Else chunk blockIdx.x, whose counts are written when maps are wanted.
template <int LPT, int VPL, bool WIDE, bool SOFT, bool GROUPS, bool SINGLE, int TOK>
__global__ void __launch_bounds__((TOK * LPT)) route_kernel(const Args a) {
    constexpr int THREADS = TOK * LPT;
    constexpr int RPL = kMaxTopk / LPT;
    __shared__ GroupLds groups[TOK];
    __shared__ ExactLds exact;
    __shared__ int n_left, left[kSingle];              // tokens that 32 bits do not rank (a chunk has kSingle at most)
    __shared__ uint64_t mask[SINGLE ? kMaxE : 1];      // the tokens of each expert
    __shared__ uint32_t count[SINGLE ? 1 : kMaxE];
    __shared__ int32_t all_ids[SINGLE ? kSingle * kMaxTopk : 1];
    __shared__ int32_t first[SINGLE ? kMaxE : 1];
    __shared__ int sums[THREADS / kWave];
    const int l = threadIdx.x % LPT, w = threadIdx.x / LPT;
    const int t0 = blockIdx.x * a.chunk;
    const int n_tok = min(a.chunk, a.T - t0);
    float next[VPL];                                   // the next token's logits are asked for before this one is ranked
    if (w < n_tok) load_row<LPT>(a, t0 + w, l, next);
    const LaneExperts<VPL> x = lane_experts<LPT, VPL>(a, l);
    for (int i = threadIdx.x; i < a.E; i += THREADS) {
        if constexpr (SINGLE) mask[i] = 0ull;
        else count[i] = 0u;
    }
    if (threadIdx.x == 0) n_left = 0;
    __syncthreads();
    auto count_routes = [&](int t, const int (&id)[RPL]) {
#pragma unroll
        for (int j = 0; j < RPL; j++) {
            const int r = j * LPT + l;
            if (r >= a.topk) continue;
            if constexpr (SINGLE) {
                all_ids[t * a.topk + r] = id[j];
                if (id[j] >= 0) atomicOr((unsigned long long*)&mask[id[j]], 1ull << t);
            } else {
                if (id[j] >= 0) atomicAdd(&count[id[j]], 1u);
            }
        }
    };
    for (int i = 0; i < n_tok; i += TOK) {
        if (i + w < n_tok) {                           // whole tokens are active or idle together
            const int t = t0 + i + w;
            TokenScores<VPL> s;
            score_token<LPT, VPL, WIDE, SOFT>(a, next, t, l, s);
            if (i + TOK + w < n_tok) load_row<LPT>(a, t + TOK, l, next);
            uint32_t mine[RPL];
            int n;
            bool close;
            if (rank_fast<LPT, VPL, WIDE, SOFT, GROUPS>(a, (int64_t)t * a.stride, x, s, l, groups[w], mine, n, close)) {
                if (close) refine<LPT, WIDE, SOFT>(a, (int64_t)t * a.stride, l, s.top, n, groups[w], mine);
                int id[RPL];
                float lg[RPL];
#pragma unroll
                for (int j = 0; j < RPL; j++) {
                    id[j] = mine[j] && j * LPT + l < a.topk ? (int)(1023u - (mine[j] & 1023u)) : -1;
                    lg[j] = -__builtin_inff();
                    if (j * LPT >= a.topk) continue;
#pragma unroll
                    for (int k = 0; k < VPL; k++) {
                        const float y = __shfl(s.v[k], id[j] & (LPT - 1), LPT);
                        lg[j] = id[j] >= 0 && id[j] / LPT == k ? y : lg[j];
                    }
                }
                weigh_token<LPT, SOFT>(a, t, l, id, lg, s.top, s.z);
                count_routes(t, id);
            } else if (l == 0) {
                left[atomicAdd(&n_left, 1)] = t;
            }
            wave_lds_fence();                          // the groups are read before the next token's
        }
    }
    __syncthreads();
    for (int i = 0; i < n_left; i++) {                 // (each by itself: their order changes nothing)
        const int t = left[i];
        float top, z;
        rank_exact<THREADS, WIDE>(a, t, exact, top, z);
        if (threadIdx.x < LPT) {
            int id[RPL];
            float lg[RPL];
#pragma unroll
            for (int j = 0; j < RPL; j++) {
                const int r = j * LPT + l;
                id[j] = r < a.topk ? exact.id[r] : -1;
                lg[j] = id[j] >= 0 ? exact.logit[r] : -__builtin_inff();
            }
            weigh_token<LPT, SOFT>(a, t, l, id, lg, top, z);
            count_routes(t, id);
        }
        __syncthreads();                               // before the next one's
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
    static_assert(kScatterThreads >= kMaxE, "a thread an expert");
    __shared__ int base[kMaxE];
    __shared__ uint64_t mask[kMaxE];
    __shared__ int sums[kScatterThreads / kWave];
    __shared__ uint4 sum4[SCANNED ? 1 : kScatterThreads];
    const int rw = row_bytes(a.E), c = blockIdx.x, e = threadIdx.x;
    const int t0 = c * a.chunk, n_tok = min(a.chunk, a.T - t0), n = n_tok * a.topk;
    const int32_t* ids = a.ids + (int64_t)t0 * a.topk;
    const int id0 = (int)threadIdx.x < n ? ids[threadIdx.x] : -1;      // asked for before the counts
    mask[e] = 0ull;
    int all = 0, early = 0;                            // expert e's routes, and those of the chunks before this one
    if constexpr (SCANNED) {
        if (e < a.E) {
            all = a.before[(int64_t)a.nc * rw + e];
            early = a.before[(int64_t)c * rw + e];
        }
        __syncthreads();
    } else {
        // Four experts a thread (a word of a chunk's counts), the chunks dealt over the parts of the workgroup, kAsk of them asked
        // for at once; sums of bytes as 16-bit pairs (at most 512 chunks of 64 tokens: 32768), added up over the parts through LDS.
        constexpr int kAsk = 16;
        const int quads = rw / 4, parts = kScatterThreads / quads;
        const int part = threadIdx.x / quads, qd = threadIdx.x - part * quads;
        uint32_t even = 0, odd = 0, even_b = 0, odd_b = 0;
        if (part < parts) {
            const uint8_t* counts = a.counts + qd * 4;
            for (int c0 = part; c0 < a.nc; c0 += kAsk * parts) {
                uint32_t w[kAsk];
#pragma unroll
                for (int k = 0; k < kAsk; k++) w[k] = *reinterpret_cast<const uint32_t*>(counts + (int64_t)min(c0 + k * parts, a.nc - 1) * rw);
#pragma unroll
                for (int k = 0; k < kAsk; k++) {
                    const int cc = c0 + k * parts;
                    const uint32_t v = cc < a.nc ? w[k] : 0u, before = cc < c ? v : 0u;
                    even += v & 0x00FF00FFu;
                    odd += v >> 8 & 0x00FF00FFu;
                    even_b += before & 0x00FF00FFu;
                    odd_b += before >> 8 & 0x00FF00FFu;
                }
            }
            sum4[threadIdx.x] = make_uint4(even, odd, even_b, odd_b);
        }
        __syncthreads();
        if (e < a.E) {
            const int sh = (e & 2) * 8;
            for (int p = 0; p < parts; p++) {
                const uint4 v = sum4[p * quads + e / 4];
                all += (e & 1 ? v.y : v.x) >> sh & 0xFFFFu;
                early += (e & 1 ? v.w : v.z) >> sh & 0xFFFFu;
            }
        }
    }
    auto mark = [&](int i, int id) {
        if (id >= 0) atomicOr((unsigned long long*)&mask[id], 1ull << (i / a.topk));
    };
    mark(threadIdx.x, id0);
    for (int i = threadIdx.x + kScatterThreads; i < n; i += kScatterThreads) mark(i, ids[i]);
    int run;
    const int at = block_scan<kScatterThreads>(all, sums, run);
    base[e] = early + at;
    if (c == 0 && e < a.E) a.offsets[e] = at;
    if (c == 0 && e == 0) a.offsets[a.E] = run;
    __syncthreads();
    auto place = [&](int i, int id) {
        const int tt = i / a.topk;
        int row = -1;
        if (id >= 0) {
            row = base[id] + __popcll(mask[id] & ((1ull << tt) - 1ull));
            a.dst2src[row] = t0 + tt;
        }
        a.route_rows[(int64_t)t0 * a.topk + i] = row;
    };
    if ((int)threadIdx.x < n) place(threadIdx.x, id0);
    for (int i = threadIdx.x + kScatterThreads; i < n; i += kScatterThreads) place(i, ids[i]);
    // the rows behind the last route name no token
    const int64_t routes = (int64_t)a.T * a.topk;
    for (int64_t i = run + (int64_t)c * kScatterThreads + threadIdx.x; i < routes; i += (int64_t)gridDim.x * kScatterThreads)
        a.dst2src[i] = -1;
}

__global__ void zero_offsets_kernel(int E, int32_t* offsets) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
}

// One workgroup, one launch.  (256 experts in 8 groups, in a graph: 64 tokens 29 us so and 13.6 in two launches of more, 32
// tokens 16.8 and 13.5, 16 tokens 10.6; outside of one the second launch costs the caller 4 us.  So 17 to 32 tokens of more than
// 64 experts are the quicker in one launch as eager calls, and up to 3 us slower in a graph.)
// Chunks: 16 tokens up to 512 chunks, then 64.  Without groups, over 256 experts, 8192 tokens take 25.0 us, 8193 25.7, 16384 26.9,
// 24576 49.8 and 32768 51.2; in 8 groups 31.1, 37.2, 36.1, 69.4 and 70.1.  A CU holds one workgroup, so chunks of 64 leave half of
// the card idle just past 8192.  Past 32768 the scan, one workgroup for 256 experts, takes nearly half of the time: 32769 tokens
// 93.7 us, 131072 344.
bool single(int64_t T, int64_t E) { return T <= (E <= 64 ? kSingle : kSingleWide); }
int chunk_of(int64_t T, int64_t E) { return single(T, E) ? kSingle : T <= (int64_t)kTok * kSumChunks ? kTok : 64; }

template <int LPT, int VPL, bool WIDE, bool SOFT, bool GROUPS>
void launch_route(hipStream_t st, const Args& a) {
    auto launch = [&](auto single, auto tok, int64_t blocks) {
        hipLaunchKernelGGL((route_kernel<LPT, VPL, WIDE, SOFT, GROUPS, decltype(single)::value, decltype(tok)::value>), dim3((unsigned)blocks),
                           dim3(decltype(tok)::value * LPT), 0, st, a);
    };
    constexpr std::integral_constant<int, kTok> some{};
    if (!single(a.T, a.E)) return launch(std::false_type{}, some, a.nc);
    // (64 tokens of 64 experts in 8 groups: 14.6 us all at once, 25.3 by sixteens; 8 tokens 6.6 and 5.9)
    if constexpr (LPT == 16) {
        if (a.T > kTok) return launch(std::true_type{}, std::integral_constant<int, kSingle>{}, 1);
    }
    launch(std::true_type{}, some, 1);
}

template <bool WIDE, bool SOFT, bool GROUPS>
void launch_route_e(hipStream_t st, const Args& a) {
    if (a.E <= 64) launch_route<16, 4, WIDE, SOFT, GROUPS>(st, a);
    else if (a.E <= 256) launch_route<64, 4, WIDE, SOFT, GROUPS>(st, a);
    else if (a.E <= 512) launch_route<64, 8, WIDE, SOFT, GROUPS>(st, a);
    else launch_route<64, 16, WIDE, SOFT, GROUPS>(st, a);
}

template <bool WIDE, bool SOFT>
void launch_route_groups(hipStream_t st, const Args& a) {
    if (a.n_group > 1) launch_route_e<WIDE, SOFT, true>(st, a);
    else launch_route_e<WIDE, SOFT, false>(st, a);
}

// The kernels of 513 to 1024 experts spill 96 to 113 vector registers with groups and choices, 55 with groups alone, 2 to 19
// without; those of 257 to 512 experts 8 to 20 with groups and choices, the others none.  (1024 experts, 4096 tokens: 24.2 us,
// with a bias and 32 groups 55.9.)
// What a kernel knows: whether choices (scores formed) or logits are ranked, the scores' form, whether there are groups.  (With
// all of it in one kernel the registers of the groups' part spill in the others': 16384 tokens over 512 experts 50.9 us
// instead of 46.)
template <bool WIDE>
void launch_route_score(hipStream_t st, const Args& a) {
    if (a.score == MOE_SCORE_SOFTMAX) launch_route_groups<WIDE, true>(st, a);
    else launch_route_groups<WIDE, false>(st, a);
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

// Bytes of workspace that T tokens take with maps: the chunks' counts, and their sums where a scan forms them.
int64_t workspace_need(int64_t T, int64_t E) {
    if (single(T, E)) return 0;
    const int64_t nc = ceil_div(T, chunk_of(T, E)), rw = row_bytes((int)E);
    return nc * rw + (nc > kSumChunks ? (nc + 1) * rw * 4 : 0);
}

bool scale_ok(float scale) { return scale > 0.0f && scale <= 3.402823466e38f; }

bool natural(const void* p, int dt) { return reinterpret_cast<uintptr_t>(p) % (dt == MOE_F32 ? 4 : 2) == 0; }

}  // namespace
}  // namespace router
}  // namespace moe

using namespace moe;

extern "C" size_t moe_router_workspace_size(int64_t T, int64_t E) {
    if (T > router::kMaxT || E < 1 || E > router::kMaxE) return 0;
    // Chunks grow from 16 tokens to 64 past kTok * kSumChunks tokens, which then need less: not fewer bytes than those.
    const int64_t bytes = std::max(router::workspace_need(T, E), router::workspace_need(std::min<int64_t>(T, router::kTok * router::kSumChunks), E));
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
    a.chunk = router::chunk_of(T, E);
    a.nc = (int)ceil_div(T, a.chunk);
    if (maps && !router::single(T, E)) {
        if (!workspace) return MOE_ERR_NULL;
        if (ws_bytes < (size_t)router::workspace_need(T, E)) return MOE_ERR_WORKSPACE;
        if (!aligned16(workspace)) return MOE_ERR_ALIGN;
        a.counts = (uint8_t*)workspace;
        a.before = (int32_t*)(a.counts + (int64_t)a.nc * router::row_bytes((int)E));
    }
    if (bias || (a.n_group > 1 && group_top == 2)) router::launch_route_score<true>(st, a);
    else router::launch_route_score<false>(st, a);
    if (maps && !router::single(T, E)) {
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
