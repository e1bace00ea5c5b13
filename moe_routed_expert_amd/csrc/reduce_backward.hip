// Backward of the routing-weighted reduce (moe_topk_reduce) and of the router's weights (moe_route_prep).
//
// out[t] = sum_j w[t,j] y[row(t,j)] gives dy[row(t,j)] = w[t,j] dout[t] and dw[t,j] = <dout[t], y[row(t,j)]>.
// w_j = softmax over the top-k logits gives dlogits[id_j] = w_j (dw_j - sum_i w_i dw_i), zero elsewhere.
//
// MI355X design: HBM-bound.  A workgroup takes one token and up to P of its routes: each thread holds 8
// columns of dout in registers, asks for the routes' y and then, route by route, adds to that route's dot product
// and writes dy, so y and dy move once and dout once per P routes (from L2 after the first).  P is 2: at 4096
// tokens, six routes and 4096 bf16 columns 2 took 91 us (4.8 TB/s, of a copy's 4.9), 1 94 us and 8, with a quarter
// of the workgroups, 98 us.  Below 1024 tokens P is 1, a workgroup per route, which fills more of the chip.  The dot
// products are summed in fp32: 8 columns at a time per thread, then lanes by
// shuffles, then waves through LDS, always in the same order.
#include <algorithm>

#include "cols8.h"
#include "host.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 23;           // a grid's threads fit 32 bits; workgroups take more items in turn

struct BackArgs {
    const uint16_t* dout;
    int64_t dout_stride;
    const void* y;
    int64_t y_stride;
    const int32_t* slots;
    const int32_t* route_rows;
    const float* weights;
    int64_t T, topk, H, y_rows;
    void* dy;
    int64_t dy_stride;
    float* dweights;
};

template <int DT, int P, bool VEC>
__global__ void __launch_bounds__(kThreads) topk_reduce_backward_kernel(const BackArgs a) {
    __shared__ float part[kThreads / kWave][P];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int64_t passes = ceil_div(a.topk, P);
    for (int64_t item = blockIdx.x; item < a.T * passes; item += gridDim.x) {
        const int64_t t = item / passes, j0 = item % passes * P;
        // per route: its row (-1: none to write), and its weight; an inactive route's weight and y are not read
        int64_t row[P];
        bool on[P];
        float w[P], dot[P];
#pragma unroll
        for (int u = 0; u < P; u++) {
            const int64_t rt = t * a.topk + j0 + u;
            const bool in = j0 + u < a.topk;
            on[u] = in && a.slots[in ? rt : 0] >= 0;
            row[u] = -1;
            if (a.route_rows) {
                if (on[u]) row[u] = a.route_rows[rt];
            } else if (in) {
                row[u] = rt;
            }
            if (row[u] >= a.y_rows) row[u] = -1;
            on[u] = on[u] && row[u] >= 0;
            w[u] = on[u] ? a.weights[rt] : 0.0f;
            dot[u] = 0.0f;
        }
        for (int64_t c = (int64_t)tid * kCols; c < a.H; c += kThreads * kCols) {
            const int valid = (int)(a.H - c < kCols ? a.H - c : kCols);
            float d[kCols];
            RawCols8<DT> raw[P];
            if constexpr (VEC) {                           // every route's y is on its way before the first is used
#pragma unroll
                for (int u = 0; u < P; u++)
                    if (on[u] && a.dweights) raw[u].load(a.y, row[u] * a.y_stride + c);
            }
            load_cols<kBF16, VEC>(a.dout, t * a.dout_stride + c, valid, d);
#pragma unroll
            for (int u = 0; u < P; u++) {
                if (on[u] && a.dweights) {
                    float y[kCols];
                    if constexpr (VEC) raw[u].get(y);
                    else load_cols<DT, false>(a.y, row[u] * a.y_stride + c, valid, y);
#pragma unroll
                    for (int i = 0; i < kCols; i++) dot[u] = __builtin_fmaf(d[i], y[i], dot[u]);
                }
                if (row[u] >= 0) {
                    float o[kCols];
#pragma unroll
                    for (int i = 0; i < kCols; i++) o[i] = on[u] ? w[u] * d[i] : 0.0f;
                    store_cols<DT, VEC>(a.dy, row[u] * a.dy_stride + c, valid, o);
                }
            }
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int u = 0; u < P; u++) {
#pragma unroll
            for (int m = 32; m > 0; m >>= 1) dot[u] += __shfl_xor(dot[u], m, kWave);
            if (lane == 0) part[wave][u] = dot[u];
        }
        __syncthreads();
        if (tid < P && j0 + tid < a.topk) {
            float sum = part[0][tid];
#pragma unroll
            for (int i = 1; i < kThreads / kWave; i++) sum += part[i][tid];
            a.dweights[t * a.topk + j0 + tid] = sum;
        }
        __syncthreads();                                   // part is read before the next item writes it
    }
}

template <int DT, int P>
void launch_back(hipStream_t st, bool vec, const BackArgs& a) {
    const int64_t items = a.T * ceil_div(a.topk, P);
    const dim3 grid((unsigned)(items < kMaxBlocks ? items : kMaxBlocks)), block(kThreads);
    if (vec) hipLaunchKernelGGL((topk_reduce_backward_kernel<DT, P, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((topk_reduce_backward_kernel<DT, P, false>), grid, block, 0, st, a);
}

template <int DT>
void launch_back_p(hipStream_t st, bool few, bool vec, const BackArgs& a) {
    if (few) launch_back<DT, 1>(st, vec, a);
    else launch_back<DT, 2>(st, vec, a);
}

// One wave per token: lane j holds route j's id and g_j = w_j (dw_j - sum_i w_i dw_i); every lane then writes
// its experts' entries, the routes' ids and values broadcast one by one.  An id named twice gets both.
__global__ void __launch_bounds__(256)
route_prep_backward_kernel(const int32_t* __restrict__ ids, const float* __restrict__ weights,
                           const float* __restrict__ dweights, int64_t T, int E, int topk, float* __restrict__ dlogits,
                           int64_t stride) {
    const int lane = threadIdx.x & (kWave - 1);
    for (int64_t t = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; t < T; t += (int64_t)gridDim.x * 4) {
        const bool in = lane < topk;
        const float w = in ? weights[t * topk + lane] : 0.0f, dw = in ? dweights[t * topk + lane] : 0.0f;
        const int id = in ? ids[t * topk + lane] : -1;
        float mean = in ? w * dw : 0.0f;
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) mean += __shfl_xor(mean, m, kWave);
        const float g = w * (dw - mean);
        for (int e = lane; e < E + kWave - 1 - (E + kWave - 1) % kWave; e += kWave) {
            float v = 0.0f;
            for (int j = 0; j < topk; j++) {
                const int idj = __builtin_amdgcn_readlane(id, j);
                const float gj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, g), j));
                if (idj == e) v += gj;
            }
            if (e < E) dlogits[t * stride + e] = v;
        }
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_topk_reduce_backward(const uint16_t* dout_bf16, int64_t dout_stride, const void* y, int y_dt,
                                        int64_t y_stride, int64_t y_rows, const int32_t* slot_ids,
                                        const int32_t* route_rows, const float* weights, int64_t T, int64_t topk,
                                        int64_t H, void* dy, int64_t dy_stride, float* dweights, void* stream) {
    if (!dtype_ok(y_dt)) return MOE_ERR_DTYPE;
    if (T < 0 || topk < 0 || topk > 1024 || H < 0 || y_rows < 0 || H > ((int64_t)1 << 30)) return MOE_ERR_SHAPE;
    if (T == 0 || topk == 0) return MOE_OK;
    if (T > 0x7FFFFFFF / topk) return MOE_ERR_SHAPE;
    if (!slot_ids || !weights || (H > 0 && (!dout_bf16 || (y_rows > 0 && (!dy || (dweights && !y)))))) return MOE_ERR_NULL;
    if (dout_stride < H || dy_stride < H || (dweights && y_stride < H)) return MOE_ERR_SHAPE;
    const uintptr_t es = y_dt == MOE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(dout_bf16) % 2 || reinterpret_cast<uintptr_t>(dy) % es || reinterpret_cast<uintptr_t>(y) % es)
        return MOE_ERR_ALIGN;
    const bool vec = H % 8 == 0 && dout_stride % 8 == 0 && dy_stride % 8 == 0 && aligned16(dout_bf16) && aligned16(dy) &&
                     (!dweights || (y_stride % 8 == 0 && aligned16(y)));
    const BackArgs a{dout_bf16, dout_stride, y, y_stride, slot_ids, route_rows, weights, T, topk, H, y_rows, dy, dy_stride, dweights};
    const bool few = T < 1024;
    auto st = as_stream(stream);
    if (y_dt == MOE_F32) launch_back_p<kF32>(st, few, vec, a);
    else if (y_dt == MOE_BF16) launch_back_p<kBF16>(st, few, vec, a);
    else launch_back_p<kF16>(st, few, vec, a);
    return launch_status();
}

extern "C" int moe_route_prep_backward(const int32_t* expert_ids, const float* weights, const float* dweights, int64_t T,
                                       int64_t E, int64_t topk, float* dlogits, int64_t dlogits_stride, void* stream) {
    if (T < 0 || T > 0x7FFFFFFF || E < 1 || E > 1024 || topk < 1 || topk > 64) return MOE_ERR_SHAPE;
    if (T == 0) return MOE_OK;
    if (!expert_ids || !weights || !dweights || !dlogits) return MOE_ERR_NULL;
    if (dlogits_stride < E) return MOE_ERR_SHAPE;
    hipLaunchKernelGGL(route_prep_backward_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(T, 4), kMaxBlocks)), dim3(256), 0, as_stream(stream),
                       expert_ids, weights, dweights, T, (int)E, (int)topk, dlogits, dlogits_stride);
    return launch_status();
}
