/*
 * moe_routed.h -- C ABI of the routed-expert hot path of a block-FP8
 * Mixture-of-Experts layer, for AMD Instinct MI355X (gfx950).
 *
 * Library: libmoe_routed.so (moe_routed_expert_amd/libmoe_routed.so).
 *
 * Number formats used by every entry point:
 *   - fp8 means the OCP e4m3fn byte (bias 7, max 448, 0x7F/0xFF NaN);
 *   - an activation row of K fp8 bytes carries ceil(K/128) fp32 scales, one
 *     per 1x128 group; a weight matrix [N][K] carries one fp32 scale per
 *     128x128 block, laid out [ceil(N/128)][ceil(K/128)];
 *   - the dequantized value is code * scale, and a scale is amax/448.
 *
 * Sources ("page" = one of the descriptions this library is built from):
 *   [inactive]  "perf(moe): skip inactive block-fp8 decode routes", opening
 *               section and Validation: a negative slot id marks an inactive
 *               route; its GEMM output tile is written as zero and nothing
 *               else of it is read; launch shapes stay fixed and the same
 *               captured graph must serve all-active, mixed and all-inactive
 *               steps with inputs changed in place.
 *   [gather]    "[MoE] Gather the cutlass MoE activation and its scales in
 *               one launch", Motivation / Modifications / Accuracy Tests:
 *               one pass over a dst2src map copies the fp8 row bytes and
 *               the row's k//128 fp32 scales; row bases in 64-bit; tails
 *               masked (k = 896 has 7 scale groups); an empty map is a no-op.
 *   [tile]      "perf(dsfp4): pick the grouped-prefill tile from route
 *               density on sm_89", The Hopper assumption / Measurements /
 *               What is not the mechanism / Testing: the prefill kernel's
 *               expert weights are FP4 and dequantizing them bounds it; the
 *               best M tile follows rows per expert (16, 32, 128 at about 6,
 *               24, 96 rows) and BLOCK_K is 128; the picker is a pure
 *               function of route and expert counts.
 *
 * Conventions for every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller.  The library
 *     allocates, frees and copies nothing, never synchronizes the stream and
 *     never reads device data on the host, so every call can be captured into
 *     a hipGraph.  `stream` is a hipStream_t (NULL = the null stream).
 *   - Sizes and strides are in ELEMENTS of the buffer they describe (bytes for
 *     fp8 buffers, floats for scale buffers), 64-bit.
 *   - Every output element named in a call is overwritten; outputs never need
 *     to be cleared by the caller (moe_topk_reduce_backward's dy may: rows of
 *     dropped routes are not named by its call).
 *   - Argument checks are host-side and look at scalars and pointers only.
 *     Device contents are not validated: a slot id >= the number of slots or
 *     offsets that disagree with m_rows are undefined behaviour (the gather's
 *     map entries are bounds-checked on the device, see below).
 *   - A call with no work (zero rows) returns MOE_OK without launching.
 *   - Results are deterministic: no floating-point atomics are used.
 */
#ifndef MOE_ROUTED_H
#define MOE_ROUTED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 1

typedef enum {
    MOE_OK = 0,
    MOE_ERR_NULL = -1,      /* a required pointer is NULL */
    MOE_ERR_SHAPE = -2,     /* a size, stride, mode or enum is out of range */
    MOE_ERR_DTYPE = -3,     /* unsupported element type for this argument */
    MOE_ERR_WORKSPACE = -4, /* workspace too small */
    MOE_ERR_ALIGN = -5,     /* a pointer or stride breaks the required alignment */
    MOE_ERR_HIP = -6,       /* the HIP runtime rejected the launch */
    MOE_ERR_SCRATCH = -7    /* moe_fused_decode_noalloc: the step needs more than its fixed scratch */
} moe_status;

/* MOE_E4M3 (codes with 1x128 scales) is taken by moe_b16_grouped_wgrad's saved operand only. */
typedef enum { MOE_BF16 = 0, MOE_F32 = 1, MOE_F16 = 2, MOE_E4M3 = 3 } moe_dtype;
/* Gated activations h = act(gate) * up: the five GLU variants (SwiGLU, GEGLU with the exact GELU,
 * ReGLU, GLU, bilinear); IDENTITY quantizes its input as is. */
typedef enum {
    MOE_ACT_IDENTITY = 0,
    MOE_ACT_SILU_MUL = 1,     /* (g / (1 + exp(-g))) * u */
    MOE_ACT_GELU_MUL = 2,     /* (g * (0.5 * (1 + erf(g / sqrt 2)))) * u */
    MOE_ACT_RELU_MUL = 3,     /* (g > 0 ? g : +0) * u */
    MOE_ACT_SIGMOID_MUL = 4,  /* (1 / (1 + exp(-g))) * u */
    MOE_ACT_MUL = 5           /* g * u */
} moe_act;
typedef enum { MOE_MODE_GROUPED = 0, MOE_MODE_SLOT = 1 } moe_gemm_mode;
/* Passed as the weight row stride (w_stride_n, w4_stride_n) of the grouped-mode GEMMs: the weights are
 * in the packed order that moe_pack_weights writes, and the expert stride keeps its meaning. */
#define MOE_W_PACKED (-1)

/* Version of this header the library was built from (MOE_ABI_VERSION). */
int moe_abi_version(void);

/* Human-readable text for a moe_status value (static storage). */
const char* moe_status_string(int status);

/* Text of the last HIP error seen by a launch on the calling host thread (thread-local storage). */
const char* moe_last_hip_error(void);

/*
 * moe_gather_rows_scales  [gather]
 *   for i in [0, n_dst):  src = dst2src[i]
 *     src >= 0: dst_q[i, 0:k] = src_q[src, 0:k]   (bytes, never decoded)
 *               dst_s[i, 0:g] = src_s[src, 0:g]   (raw 32-bit words)
 *     src <  0 or src >= n_src: dst_q[i, 0:k] = 0 and dst_s[i, 0:g] = +0.0
 *       (the page defines in-range entries only; an out-of-range entry is
 *       caught on the device and reads no source row)
 *   src_q  [n_src][src_q_stride] bytes;  src_s [n_src][src_s_stride] fp32
 *   dst_q  [n_dst][dst_q_stride] bytes;  dst_s [n_dst][dst_s_stride] fp32
 *   g is passed explicitly (normally ceil(k/128)); g == 0 reads and writes no
 *   scale word, so src_s and dst_s may then be NULL.  Strides >= widths.
 *   Alignment: none required; 16-byte aligned rows take the vector path.
 *   n_dst == 0 returns MOE_OK with no launch.
 */
int moe_gather_rows_scales(const void* src_q, int64_t src_q_stride,
                           const float* src_s, int64_t src_s_stride,
                           int64_t n_src, int64_t k, int64_t g,
                           const int32_t* dst2src, int64_t n_dst,
                           void* dst_q, int64_t dst_q_stride,
                           float* dst_s, int64_t dst_s_stride,
                           void* stream);

/*
 * moe_act_quant  -- per-row 1x128 fp8 quantization, optionally of a gated activation
 *   act = MOE_ACT_IDENTITY: v = in[r, c] for c in [0, n)
 *   gated acts (moe_act 1..5): in row is [gate(0:n) | up(n:2n)], v = act(gate) * up in fp32, with the
 *   expressions of moe_act ([inactive] Validation lists five activations; the five GLU variants are
 *   taken as them)
 *   per group of 128 columns of v (last group may be shorter):
 *     s = max|v| / 448 (fp32, correctly rounded);  q = (s == 0) ? 0x00 : e4m3_rne(v / s)
 *   in    [rows][in_stride] of in_dt (MOE_BF16, MOE_F16 or MOE_F32)
 *   out_q [rows][q_stride] bytes, out_s [rows][s_stride] fp32 (ceil(n/128) used)
 *   Inputs must be finite.  IDENTITY mode is bit-exact with a correctly
 *   rounded division and round-to-nearest-even e4m3 encoding, and so are
 *   RELU_MUL and MUL (exact fp32 products).  SILU and SIGMOID take the
 *   sigmoid as rcp(1 + exp2(-g * log2 e)) from the hardware exp2 and
 *   reciprocal (each within 1 ulp; 0 once 1 + e^-g exceeds 2^126, i.e. for
 *   g below about -87.3), GELU the device erff, so their values differ from
 *   the fp32 libm expressions of moe_act by a few ulp and a code may differ
 *   by one e4m3 step, rarely.  An all-zero group gives s = +0 and q = 0x00 (a zeroed
 *   inactive-route tile stays zero, [inactive] opening section).
 */
int moe_act_quant(const void* in, int in_dt, int64_t in_stride, int64_t rows, int64_t n, int act,
                  uint8_t* out_q, int64_t q_stride, float* out_s, int64_t s_stride, void* stream);

/*
 * moe_pick_block_m  [tile]
 *   The M tile of the grouped GEMM for `routes` routed rows over `experts`
 *   experts.  As on the page, the tile grows with rows per expert; the
 *   thresholds are MI355X's (a sweep of every tile at 6, 24, 48 and 96 rows
 *   per expert): with r = ceil(routes/experts), r <= 8 gives 16, r <= 64
 *   gives 64, larger r gives 128.  Pure function of its two arguments;
 *   returns 16 when either is <= 0.
 */
int moe_pick_block_m(int64_t routes, int64_t experts);

/*
 * moe_grouped_block_m  [tile]
 *   The M tile the grouped-mode GEMMs take when called with block_m = 0, for
 *   `routes` rows over `experts` experts, K, the weight format (mxfp4 = 0:
 *   block-FP8, 1: MXFP4), the bank layout (packed = 1: MOE_W_PACKED) and the
 *   form (fused = 1: the gate/up + requant entry points).  It refines
 *   moe_pick_block_m with an MI355X sweep of every tile at 48 to 24576 routes
 *   over 256 experts; with r = ceil(routes/experts):
 *     block-FP8 row-major: 128 (plain), moe_pick_block_m (fused);
 *     block-FP8 packed:    r <= 8: 16; r <= 64: 128 if K <= 2048, else 64; 128;
 *     MXFP4:               r <= 8: 16; r <= 64: 32 (packed) or 64; 128, or 64
 *                          for packed banks with K > 2048.
 *   Pure function; 16 when routes or experts is <= 0.
 */
int moe_grouped_block_m(int64_t routes, int64_t experts, int64_t K, int mxfp4, int packed, int fused);

/*
 * moe_bf8_grouped_gemm  -- block-FP8 GEMM for the gate/up and the down projections
 *   ("bf8" = block-FP8 with e4m3 operands.)
 *   out[r, n] = sum_kb ( sum_{k in kb} A[ar, k] * W[e, n, k] ) * a_s[ar, kb] * w_s[e, n/128, kb]
 *   with fp8 products exact; the 128 products of a K block are summed by the fp8 MFMA, which keeps
 *   about 13-14 significant bits of that sum (error below 2^-12 of the block's sum |products|), and
 *   the scaled block sums are accumulated in fp32.
 *   a_q  [*][a_stride] fp8,   a_s [*][a_s_stride] fp32 (K/128 used)
 *   w_q  [n_experts] x [N][K] fp8: element (e,n,k) at e*w_stride_e + n*w_stride_n + k
 *   w_s  fp32: block (e,nb,kb) at e*w_s_stride_e + nb*w_s_stride_n + kb
 *   out  [m_rows][out_stride] of out_dt (MOE_BF16, MOE_F16 or MOE_F32)
 *   mode MOE_MODE_GROUPED (prefill, [tile]): rows sorted by expert; rows
 *        [expert_offsets[e], expert_offsets[e+1]) use expert e and A row r;
 *        expert_offsets is a DEVICE int32 array of n_experts+1 entries with
 *        expert_offsets[0] = 0 and expert_offsets[n_experts] <= m_rows (rows
 *        beyond it are left untouched).  block_m = 0 picks the M tile with
 *        moe_grouped_block_m (moe_pick_block_m's density rule, refined per
 *        weight format and bank layout); 16, 32, 64 or 128 forces it.
 *        The kernel is persistent (one workgroup per resident slot); tiles
 *        come from the device offsets, clamped to [0, m_rows].
 *   mode MOE_MODE_SLOT (decode, [inactive]): row r uses slot slot_ids[r]
 *        (DEVICE int32 [m_rows]) and A row r / a_row_div; a negative slot
 *        writes a +0 output row and reads no A, W or scales of that row.
 *        Meant for decode-sized row counts (every row streams its expert).
 *   Requirements: K % 128 == 0, N % 16 == 0, m_rows <= 2^31 - 1 (every
 *   grouped entry point: MOE_ERR_SHAPE beyond); w_q, a_q and their strides
 *   16-byte aligned (MOE_ERR_ALIGN otherwise).  Grouped mode also needs
 *   N % 128 == 0, 1 <= n_experts <= 1024 and K <= 8192 (a tile keeps all its
 *   K-block scales in LDS); MOE_ERR_SHAPE otherwise.  n_experts == 0 with NULL
 *   w_q/w_s is allowed in slot mode (an empty bank: every slot must be < 0).
 *   Grouped mode also takes a packed bank (moe_pack_weights with step_bytes
 *   128): w_stride_n = MOE_W_PACKED, w_stride_e >= N*K when n_experts > 1.
 */
int moe_bf8_grouped_gemm(const uint8_t* a_q, int64_t a_stride, const float* a_s, int64_t a_s_stride,
                         const uint8_t* w_q, int64_t w_stride_e, int64_t w_stride_n,
                         const float* w_s, int64_t w_s_stride_e, int64_t w_s_stride_n,
                         int64_t n_experts, int64_t N, int64_t K,
                         int mode, const int32_t* expert_offsets, const int32_t* slot_ids,
                         int64_t m_rows, int64_t a_row_div, int32_t block_m,
                         void* out, int out_dt, int64_t out_stride, void* stream);

/*
 * moe_bf8_grouped_gemm_act_quant  -- the prefill gate/up GEMM with the gated
 *   activation and its requant in the epilogue  [tile] [inactive]
 *   The gate/up GEMM of grouped (prefill) mode followed by moe_act_quant with
 *   a gated act (moe_act 1..5), in one launch: with c1 the fp32 GEMM result of
 *   moe_bf8_grouped_gemm (N = 2I, W13 rows 0..I-1 gate, I..2I-1 up), never
 *   stored, h[r, c] = act(g) * u with g = c1[r, c], u = c1[r, I + c] (fp32,
 *   the moe_act expressions), then per 1x128 group s = amax/448 and
 *   q = e4m3(h/s) as in moe_act_quant (q = 0x00, s = +0 when amax = 0).
 *   a_q, a_s, w_q, w_s, expert_offsets, m_rows, block_m: as moe_bf8_grouped_gemm
 *   in MOE_MODE_GROUPED with N = 2I.
 *   out_q [m_rows][q_stride] fp8 (I used), out_s [m_rows][s_stride] fp32 (I/128
 *   used).  The results equal moe_bf8_grouped_gemm with MOE_F32 output followed
 *   by moe_act_quant with the same act on it, bit for bit.
 *   Requirements: I % 128 == 0, K % 128 == 0, K <= 8192, 1 <= n_experts <=
 *   1024, alignment as moe_bf8_grouped_gemm; m_rows == 0 launches nothing.
 *   w_stride_n = MOE_W_PACKED takes a packed bank as moe_bf8_grouped_gemm.
 */
int moe_bf8_grouped_gemm_act_quant(const uint8_t* a_q, int64_t a_stride, const float* a_s, int64_t a_s_stride,
                                   const uint8_t* w_q, int64_t w_stride_e, int64_t w_stride_n,
                                   const float* w_s, int64_t w_s_stride_e, int64_t w_s_stride_n,
                                   int64_t n_experts, int64_t I, int64_t K, const int32_t* expert_offsets,
                                   int64_t m_rows, int32_t block_m, int act, uint8_t* out_q, int64_t q_stride,
                                   float* out_s, int64_t s_stride, void* stream);

/*
 * moe_mxfp4_grouped_gemm  -- the grouped (prefill) GEMM with FP4 expert weights
 *   [tile]: the routed-expert prefill kernel of that page takes FP4 weights and
 *   is limited by dequantizing them.  The page does not fix the FP4 format;
 *   the one taken is OCP MXFP4: E2M1 elements (+-{0, 0.5, 1, 1.5, 2, 3, 4, 6}),
 *   two per byte with K element 2i in the low nibble, and one E8M0 scale byte
 *   (2^(e-127)) per 32 consecutive K elements.
 *   out[r, n] = sum_kb ( sum_{k in kb} A[r, k] * W[e, n, k] * 2^(w4_s[e, n, k/32] - 127) ) * a_s[r, kb]
 *   with products exact, each 128-wide K block (kb) summed by the MFMA as in moe_bf8_grouped_gemm
 *   and the scaled block sums accumulated in fp32.
 *   a_q, a_s: fp8 activations with 1x128 fp32 scales, as moe_bf8_grouped_gemm.
 *   w4   [n_experts] x [N][K/2] bytes: the byte of (e, n, k) is at
 *        e*w4_stride_e + n*w4_stride_n + k/2 (strides in BYTES).
 *   w4_s [n_experts] x [N][K/32] E8M0 bytes: block (e, n, k/32) at
 *        e*w4s_stride_e + n*w4s_stride_n + k/32 (strides in bytes).
 *   expert_offsets, m_rows, block_m, out, out_dt, out_stride: as
 *   moe_bf8_grouped_gemm in MOE_MODE_GROUPED.
 *   Requirements: N % 128 == 0, K % 128 == 0, K <= 8192, 1 <= n_experts <=
 *   1024 (MOE_ERR_SHAPE); a_q, w4 and their strides 16-byte aligned, w4_s and
 *   its strides 4-byte aligned (MOE_ERR_ALIGN).  A scale byte of 255 (NaN in
 *   the format) gives results this library does not define, and so do scaled
 *   products below the fp32 normal range.  m_rows == 0 launches nothing.
 *   w4_stride_n = MOE_W_PACKED takes a packed bank (moe_pack_weights with
 *   step_bytes 64), w4_stride_e >= N*K/2 when n_experts > 1; w4_s unchanged.
 */
int moe_mxfp4_grouped_gemm(const uint8_t* a_q, int64_t a_stride, const float* a_s, int64_t a_s_stride,
                           const uint8_t* w4, int64_t w4_stride_e, int64_t w4_stride_n,
                           const uint8_t* w4_s, int64_t w4s_stride_e, int64_t w4s_stride_n,
                           int64_t n_experts, int64_t N, int64_t K, const int32_t* expert_offsets,
                           int64_t m_rows, int32_t block_m, void* out, int out_dt, int64_t out_stride,
                           void* stream);

/*
 * moe_mxfp4_grouped_gemm_act_quant  -- moe_bf8_grouped_gemm_act_quant with
 *   MXFP4 gate/up weights  [tile] [inactive]
 *   c1 is the fp32 result of moe_mxfp4_grouped_gemm with N = 2I (W13 rows
 *   0..I-1 gate, I..2I-1 up), never stored; the gated activation and its
 *   1x128 requant into out_q / out_s are those of
 *   moe_bf8_grouped_gemm_act_quant.  The results equal moe_mxfp4_grouped_gemm
 *   with MOE_F32 output followed by moe_act_quant with the same act, bit for
 *   bit.  Requirements: I % 128 == 0 and the rest as moe_mxfp4_grouped_gemm.
 */
int moe_mxfp4_grouped_gemm_act_quant(const uint8_t* a_q, int64_t a_stride, const float* a_s, int64_t a_s_stride,
                                     const uint8_t* w4, int64_t w4_stride_e, int64_t w4_stride_n,
                                     const uint8_t* w4_s, int64_t w4s_stride_e, int64_t w4s_stride_n,
                                     int64_t n_experts, int64_t I, int64_t K, const int32_t* expert_offsets,
                                     int64_t m_rows, int32_t block_m, int act, uint8_t* out_q, int64_t q_stride,
                                     float* out_s, int64_t s_stride, void* stream);

/*
 * moe_pack_weights  -- an expert bank in the grouped GEMMs' operand order
 *   Not a step of the pages' method: a one-time copy of static weights into an
 *   order in which every 1 KiB load of the grouped GEMMs reads contiguous bytes
 *   (row-major weights are read as 64 bytes of each of 16 rows 4 KiB or more
 *   apart, which streams about 15 % slower on MI355X).
 *   w     [n_experts] x [N][row_bytes] bytes: byte (e, n, c) at e*w_stride_e + n*w_stride_n + c
 *         (block-FP8: row_bytes = K; MXFP4: row_bytes = K/2 nibble pairs).
 *   step_bytes: bytes of one 128-wide K block of a row: 128 (block-FP8) or 64 (MXFP4).
 *   out   packed bank, expert e at e*out_stride_e.  Within an expert, for each 16-row
 *         group g = n/16 and K step s = c/step_bytes, a block of 16*step_bytes bytes at
 *         (g*(row_bytes/step_bytes) + s)*16*step_bytes holds 16-byte pieces p = 0 ..
 *         step_bytes-1: piece p is row 16g + (p%16), bytes s*step_bytes + 64*(p/64) +
 *         16*((p%64)/16) .. +15.  The scale arrays keep their own layout.
 *   The grouped-mode GEMMs read such a bank when given w_stride_n = MOE_W_PACKED
 *   and the bank's expert stride; their results are those of the row-major bank,
 *   bit for bit.  Slot mode and the fused decode take row-major banks only.
 *   Requirements: N % 16 == 0, step_bytes 64 or 128, row_bytes % step_bytes == 0,
 *   w_stride_n >= row_bytes, w_stride_e >= N*w_stride_n and out_stride_e >=
 *   N*row_bytes when n_experts > 1 (MOE_ERR_SHAPE); w, out and every stride
 *   16-byte aligned (MOE_ERR_ALIGN).  w and out must not overlap.
 */
int moe_pack_weights(const uint8_t* w, int64_t w_stride_e, int64_t w_stride_n, int64_t n_experts, int64_t N,
                     int64_t row_bytes, int64_t step_bytes, uint8_t* out, int64_t out_stride_e, void* stream);

/*
 * moe_topk_reduce  -- routing-weighted sum over each token's top-k routes
 *   out[t, h] = bf16_rne( sum_{j = 0..topk-1, slot_ids[t,j] >= 0} weights[t,j] * y[row(t,j), h] )
 *   summed in fp32 in ascending j from +0; row(t,j) = route_rows[t*topk + j]
 *   (DEVICE int32) or t*topk + j when route_rows is NULL.  The weight of an
 *   inactive route is never read ([inactive] opening section).  A token with
 *   no active route gets +0.0.
 *   y [*][y_stride] of y_dt;  slot_ids, weights [T][topk];  out [T][out_stride] bf16.
 */
int moe_topk_reduce(const void* y, int y_dt, int64_t y_stride,
                    const int32_t* slot_ids, const int32_t* route_rows, const float* weights,
                    int64_t T, int64_t topk, int64_t H, uint16_t* out_bf16, int64_t out_stride,
                    void* stream);

/*
 * Fused decode workspace.  Layout (byte offsets written to offsets[0..6]):
 *   [0] c1   R x 2I           fp32 gate/up output (R = T*topk routes)
 *   [1] h    R x I            fp32 SiLU(gate)*up
 *   [2] aq   R x I            fp8 activation (1x128 requant of h)
 *   [3] as   R x ceil(I/128)  fp32 activation scales
 *   [4] c2   R x H            fp32 down output
 *   [5] ctl  control block: the error word and the hand-off state of the
 *            one-launch step (per-tile call counters, ready words and a
 *            tagged copy of h)
 *   [6] total size in bytes
 * Regions [0]..[4] may hold anything between calls: every call rewrites them
 * completely, and an inactive route's c1/h/aq/as/c2 rows become exact zeros
 * (h is only written when I <= 1024; wider I runs the step as four launches
 * that do not store h).  The control region must be cleared once with
 * moe_fused_decode_workspace_init before the first call and carries state
 * from call to call: a workspace serves one shape (T, H, I, topk), and calls
 * that share it must not overlap in time (e.g. on two streams without an
 * event between them).  Its first 32-bit word is the error word: nonzero
 * after a call means the step's output is not valid (its affected output
 * rows are NaN) and the workspace must be initialized again -- 1: a
 * hand-off wait gave up; 2: the workspace was
 * initialized for another (T, H, I, topk) (init writes the shape into word 1
 * of the control block, and the one-launch step checks it before it waits on
 * any hand-off word).  The library never reads the word on the host; callers
 * that need the check copy it back themselves.  Size 0 / MOE_ERR_SHAPE for
 * shapes moe_fused_decode rejects.
 */
size_t moe_fused_decode_workspace_size(int64_t T, int64_t H, int64_t I, int64_t topk);
int moe_fused_decode_workspace_layout(int64_t T, int64_t H, int64_t I, int64_t topk, int64_t offsets[7]);
int moe_fused_decode_workspace_init(void* workspace, size_t ws_bytes, int64_t T, int64_t H, int64_t I,
                                    int64_t topk, void* stream);

/*
 * moe_route_prep  -- routing prep of a prefill step  [gather] [tile]
 *   The step before the gather: the dst2src map that replicates each token's
 *   activation once per routed expert, and the expert-grouped row order of the
 *   grouped GEMM.
 *   logits   DEVICE fp32 [T][logits_stride] (E used), finite.  A NaN logit
 *   ranks as -inf so every selected id is a valid expert, but the weights of
 *   such a token are then unspecified.
 *   For each token: the topk experts with the largest logits in descending order
 *   (ties: lower expert index), and weights w_j = exp(l_j - l_max) /
 *   sum_{i in top-k} exp(l_i - l_max), i.e. the softmax over all E experts
 *   renormalized over the top-k.
 *   expert_ids [T][topk] int32, weights [T][topk] fp32.
 *   Route maps in (expert, token) order: dst2src [T*topk] int32 (token of each
 *   sorted row), route_rows [T*topk] int32 (row of route t*topk+j, the
 *   route_rows argument of moe_topk_reduce), expert_offsets [E+1] int32 (rows
 *   of expert e are [offsets[e], offsets[e+1]), the grouped GEMM's offsets).
 *   workspace: moe_route_prep_workspace_size(T, E) bytes of DEVICE memory,
 *   16-byte aligned; no initialization needed; scratch between the three
 *   launches of one call, so overlapping calls need their own workspaces.
 *   Deterministic (integer counting only).
 *   Requirements: 1 <= E <= 1024, 1 <= topk <= min(E, 64), T * topk < 2^31.
 *   T == 0 launches one small kernel that writes E + 1 zero offsets (the one
 *   exception to "no work, no launch").
 */
size_t moe_route_prep_workspace_size(int64_t T, int64_t E);
int moe_route_prep(const float* logits, int64_t logits_stride, int64_t T, int64_t E, int64_t topk,
                   int32_t* expert_ids, float* weights, int32_t* dst2src, int32_t* route_rows,
                   int32_t* expert_offsets, void* workspace, size_t ws_bytes, void* stream);

/*
 * moe_fused_decode  -- one decode step of the routed experts  [inactive]
 *   x (T x H bf16) -> 1x128 fp8 quant -> gate/up GEMM per route (slot mode,
 *   A row = token) -> act(gate)*up + 1x128 requant -> down GEMM per route
 *   -> routing-weighted top-k reduce -> out (T x H bf16).  act: a gated
 *   moe_act (1..5), as in moe_act_quant ([inactive] Validation: five
 *   activations).
 *   slot_ids, weights: DEVICE [T][topk]; slot < 0 = inactive route (zero
 *   c1/act/c2 tiles, no reads of its weights, scales or routing weight).
 *   w13_q [n_slots][2I][H] fp8 (gate rows 0..I-1, up rows I..2I-1), contiguous;
 *   w13_s [n_slots][ceil(2I/128)][ceil(H/128)] fp32;  w2_q [n_slots][H][I];
 *   w2_s [n_slots][ceil(H/128)][ceil(I/128)].
 *   Requirements: H % 128 == 0, I % 128 == 0, H and I <= 65536, 1 <= topk <= 64,
 *   T * topk <= 65535; 16-byte aligned weights and workspace, 4-byte aligned x.
 *   Launch shapes depend on (T, H, I, topk) and the device only, so one
 *   captured graph serves any slot/weight/x contents.  For small steps
 *   (H <= 2048, I <= 1024, I/8 even or a multiple of 3) whose workgroups all
 *   fit on the device at once, the step is a single launch in which gate/up
 *   tiles hand h to the down tiles through the workspace's control block;
 *   otherwise it is two launches (I <= 1024) or four (wider I).
 */
int moe_fused_decode(const uint16_t* x_bf16, int64_t T, int64_t H, int64_t I, int64_t topk, int act,
                     const int32_t* slot_ids, const float* weights, int64_t n_slots,
                     const uint8_t* w13_q, const float* w13_s,
                     const uint8_t* w2_q, const float* w2_s,
                     void* workspace, size_t ws_bytes, uint16_t* out_bf16, void* stream);

/*
 * moe_fused_decode_noalloc  -- moe_fused_decode without a caller workspace
 *   For callers that cannot allocate device memory at all: code under hipGraph
 *   capture, tight serving loops, harnesses that forbid allocation.  Arguments
 *   and results are those of moe_fused_decode minus the workspace; the step
 *   runs the same kernels on a fixed device array inside the library
 *   (4 MiB, 256-byte aligned; each GPU the library runs on holds its own copy
 *   until the process ends).  The call allocates and frees nothing.
 *   Limit: steps whose workspace (moe_fused_decode_workspace_size) exceeds
 *   4 MiB return MOE_ERR_SCRATCH without launching; e.g. up to 16 tokens at
 *   H = 4096, I = 1024, top-8.
 *   State: the array keeps the last call's contents.  The first call on a
 *   device, and every call whose (T, H, I, topk) differs from that device's
 *   previous call, first clears the control block with a fill kernel on
 *   `stream`; later calls of the same shape continue its call counters, as
 *   with an initialized workspace.  All calls on one GPU share the array, so
 *   calls that overlap in time on one GPU (two streams, two host threads
 *   without ordering) race and give undefined results.  The device is the
 *   current HIP device.
 *   Errors: as moe_fused_decode, plus MOE_ERR_SCRATCH; if a hand-off wait
 *   ever gives up, that step's affected output rows are NaN.
 */
int moe_fused_decode_noalloc(const uint16_t* x_bf16, int64_t T, int64_t H, int64_t I, int64_t topk, int act,
                             const int32_t* slot_ids, const float* weights, int64_t n_slots,
                             const uint8_t* w13_q, const float* w13_s,
                             const uint8_t* w2_q, const float* w2_s,
                             uint16_t* out_bf16, void* stream);

/*
 * 16-bit experts and the backward pass
 *   The entry points from here to moe_route_prep_backward are not steps of the pages' method: they serve
 *   expert banks that are not block-quantized, and training.  A step of the routed experts is, with W13
 *   [E][2I][H] and W2 [E][H][I] in bf16 or fp16:
 *     forward   c1 = moe_b16_grouped_gemm(x rows, W13);  h = moe_act_checkpoint(c1), which also saves c1 in
 *               8 bits;  y = moe_b16_grouped_gemm(h, W2);  out = moe_topk_reduce(y)
 *     backward  dy, dw = moe_topk_reduce_backward(dout, y);  dlogits = moe_route_prep_backward(dw);
 *               dh = moe_b16_grouped_gemm(dy, W2, w_trans);  dc1, h = moe_gated_act_backward(dh, saved c1);
 *               dW2 = moe_b16_grouped_wgrad(dy, h);  dW13 = moe_b16_grouped_wgrad(dc1, x rows, 16 bits or
 *               saved in 8);  dx rows = moe_b16_grouped_gemm(dc1, W13, w_trans), then moe_topk_reduce with
 *               unit weights sums each token's rows.
 *   Routes that are dropped after moe_route_prep (slots set negative) keep their rows in expert_offsets, and
 *   moe_topk_reduce_backward with route_rows does not write them: such a step clears dy before that call, in
 *   every step, or the gradients take up what the rows held before.
 */

/*
 * moe_b16_grouped_gemm  -- the expert GEMMs with 16-bit operands, and their data gradient
 *   out[r, n] = sum_k A[ar, k] * W(e, n, k), products and sums in fp32 (the MFMA's accumulator in grouped
 *   mode), one rounding to out_dt.
 *   a    [*][a_stride] of dt (MOE_BF16 or MOE_F16), K used
 *   w    of dt.  w_trans = 0: element (e, n, k) at e*w_stride_e + n*w_stride_r + k (rows of K: the forward).
 *        w_trans = 1: element (e, n, k) at e*w_stride_e + k*w_stride_r + n (rows of N): out = A W[e] of the
 *        bank [E][K][N], i.e. the gradient of the input of a layer whose forward used it as [E][N'=K][K'=N].
 *   out  [m_rows][out_stride] of out_dt (MOE_BF16, MOE_F16 or MOE_F32)
 *   mode, expert_offsets, slot_ids, m_rows, a_row_div: as moe_bf8_grouped_gemm.  Grouped: rows
 *        [expert_offsets[e], expert_offsets[e+1]) use expert e and A row r, offsets are clamped to [0, m_rows],
 *        rows beyond the last are left untouched, any number of rows per expert (none included); offsets that
 *        decrease somewhere leave all of out untouched.  Slot:
 *        w_trans = 0 only; a slot outside [0, n_experts) writes a +0 row and reads nothing of that row; and
 *        m_rows * ceil(N / 16) < 2^24 up to K = 1024, m_rows * ceil(N / 8) < 2^24 beyond (the workgroups of one
 *        launch; MOE_ERR_SHAPE).
 *   An infinity or NaN in a row of A or W reaches exactly the outputs whose sums hold it.
 *   Requirements: N % 8 == 0, K % 8 == 0, 8 <= N, K <= 2^20, m_rows <= 2^31 - 1, 1 <= n_experts <= 1024 in
 *   grouped mode (0 allowed in slot mode, with NULL a and w); a, w and their strides 16-byte aligned; out
 *   aligned to its type (16-byte aligned rows are stored faster).  m_rows == 0 launches nothing.
 */
int moe_b16_grouped_gemm(const void* a, int64_t a_stride, const void* w, int64_t w_stride_e, int64_t w_stride_r,
                         int64_t n_experts, int64_t N, int64_t K, int dt, int w_trans, int mode,
                         const int32_t* expert_offsets, const int32_t* slot_ids, int64_t m_rows, int64_t a_row_div,
                         void* out, int out_dt, int64_t out_stride, void* stream);

/*
 * moe_b16_grouped_tile
 *   The output tile (rows, columns) that moe_b16_grouped_gemm's grouped mode takes for m_rows rows over n_experts
 *   experts: the one of 32 x 64, 64 x 64, 64 x 256, 128 x 256 and 256 x 256 with the least estimated time.  (The
 *   largest leaves its experts' short last tiles to a second launch where with them it would take more rounds.)
 *   Pure function of its arguments; MOE_ERR_SHAPE for those the product rejects or has no work for.
 */
int moe_b16_grouped_tile(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K, int32_t tile[2]);

/*
 * moe_b16_grouped_wgrad  -- weight gradient of the grouped products
 *   dw[e, n, k] = (accumulate ? dw[e, n, k] : 0) + sum_{r in rows of e} dY[r, n] * A[r, k], in fp32, rounded
 *   once to dw_dt.  An expert without rows gets zeros (accumulate: keeps its gradient).
 *   dy   [m_rows][dy_stride] of dt (MOE_BF16 or MOE_F16), N used
 *   a    [m_rows][a_stride] of a_dt: dt, or MOE_E4M3 for rows saved in 8 bits: codes, and a_s
 *        [m_rows][a_s_stride] fp32 scales (ceil(K/128) used).  A saved operand is round_dt(code * scale);
 *        with moe_act_checkpoint's power-of-two scales that product is exact in bf16 for scales of 2^-124 and more
 *        (below, products under 2^-133, bf16's least value, round once more), and in fp16 within its range; with
 *        moe_act_quant's it is rounded once to dt.  In fp16 a product past its range is held at 65504,
 *        so finite rows saved by moe_act_checkpoint stay finite; a NaN code stays a NaN.  a_s is ignored otherwise.
 *   dw   element (e, n, k) at e*dw_stride_e + n*dw_stride_n + k, of dw_dt (MOE_BF16, MOE_F16 or MOE_F32)
 *   expert_offsets as moe_b16_grouped_gemm: rows beyond the last are not read, and offsets that decrease
 *   somewhere leave all of dw untouched.
 *   workspace: moe_b16_grouped_wgrad_workspace_size(m_rows, n_experts, N, K) bytes, 16-byte aligned, no
 *   initialization; 0 bytes (NULL allowed) unless the gradient has few tiles and long row ranges, which are
 *   then cut and their fp32 parts summed in order.  Scratch within one call: overlapping calls need their own.
 *   Requirements: 1 <= n_experts <= 1024, N % 8 == 0, K % 8 == 0 (MOE_E4M3: K % 16 == 0), 8 <= N, K <= 2^20;
 *   dy, a and their strides 16-byte aligned; dw aligned to its type.
 *   m_rows == 0 still writes the zeros (dy and a may be NULL).
 */
size_t moe_b16_grouped_wgrad_workspace_size(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K);
/* How moe_b16_grouped_wgrad takes such a problem: plan = {tile rows (N), tile columns (K), rows of a chunk or 0 where
 * the experts' rows stay whole}; tiles are 128 x 128, 256 x 128 and 256 x 256.  Pure function of its arguments. */
int moe_b16_grouped_wgrad_plan(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K, int32_t plan[3]);
int moe_b16_grouped_wgrad(const void* dy, int64_t dy_stride, int dt, const void* a, int64_t a_stride, int a_dt,
                          const float* a_s, int64_t a_s_stride, const int32_t* expert_offsets, int64_t n_experts,
                          int64_t N, int64_t K, int64_t m_rows, void* dw, int dw_dt, int64_t dw_stride_e,
                          int64_t dw_stride_n, int accumulate, void* workspace, size_t ws_bytes, void* stream);

/*
 * moe_act_checkpoint  -- activations saved in 8 bits for the backward pass
 *   Codes and scales laid out as moe_act_quant's, with power-of-two scales: per group of 128 columns
 *     s = the smallest power of two with max|v| / s <= 448, at least 2^-126 (0 for a group of zeros)
 *     q = e4m3_rne(v / s), the quotient exact; an infinity or NaN becomes the NaN code.
 *   act = MOE_ACT_IDENTITY: rows of n columns; h must be NULL.
 *   act = moe_act 1..5: in row is [gate(0:n) | up(n:2n)]; both halves are saved (codes at 0 and n, scales at
 *   0 and ceil(n/128)), and h[r, c] = act(gate) * up in fp32 of the unrounded inputs, rounded to dt, is
 *   written unless h is NULL.
 *   in    [rows][in_stride] of dt (MOE_BF16, MOE_F16 or MOE_F32);  h [rows][h_stride] of dt
 *   out_q [rows][q_stride] bytes, out_s [rows][s_stride] fp32
 *   A value v above 1.9375 * 2^127 rounds to 2^128, so code * s of it is an infinity; fp16's values from 63488 on
 *   round to 65536, which moe_b16_grouped_wgrad reads as 65504 in fp16.  A NaN gate gives a NaN in h,
 *   RELU's as well, and an infinity or NaN leaves its group a scale that may round the others to 0.
 *   Pointers aligned to their types; 16-byte aligned rows with n % 8 == 0 take the vector path.
 */
int moe_act_checkpoint(const void* in, int dt, int64_t in_stride, int64_t rows, int64_t n, int act, uint8_t* out_q,
                       int64_t q_stride, float* out_s, int64_t s_stride, void* h, int64_t h_stride, void* stream);

/*
 * moe_gated_act_backward  -- backward of h = act(gate) * up from the saved gate and up
 *   With g, u = code * scale of the two halves (moe_act_checkpoint's layout, any finite scales):
 *     dx[r, c] = dh * u * act'(g),  dx[r, n + c] = dh * act(g),  h[r, c] = act(g) * u (unless h is NULL)
 *   in fp32, rounded to dt.  ReLU's slope at 0 is 0; a NaN gate gives NaN in h, d up and (but for MUL's) d gate.
 *   dh [rows][dh_stride], dx [rows][dx_stride] (2n used), h [rows][h_stride], all of dt (MOE_BF16, MOE_F16 or
 *   MOE_F32); act: moe_act 1..5.  Alignment as moe_act_checkpoint.  An infinity or NaN in dh stays in its dx.
 */
int moe_gated_act_backward(const void* dh, int dt, int64_t dh_stride, const uint8_t* q, int64_t q_stride,
                           const float* s, int64_t s_stride, int64_t rows, int64_t n, int act, void* dx,
                           int64_t dx_stride, void* h, int64_t h_stride, void* stream);

/*
 * moe_topk_reduce_backward  -- backward of moe_topk_reduce
 *   For every route (t, j) with slot_ids[t, j] >= 0 and row(t, j) in [0, y_rows):
 *     dy[row, 0:H] = weights[t, j] * dout[t, 0:H] (fp32, rounded to y_dt)
 *     dweights[t, j] = sum_h dout[t, h] * y[row, h] (fp32, in a fixed order)
 *   Any other route gets dweights = +0 and reads neither its weight nor y; its dy row is +0 when route_rows is
 *   NULL (the row t*topk + j exists), and with route_rows it has no row (its entry is not read).  Rows that no
 *   active route names are then left as they were: clear dy first if a later product counts them.  Active routes
 *   name distinct rows.
 *   dout [T][dout_stride] bf16;  y [y_rows][y_stride] and dy [y_rows][dy_stride] of y_dt;  slot_ids, weights,
 *   dweights [T][topk];  route_rows as moe_topk_reduce (DEVICE int32 [T*topk] or NULL).
 *   dweights may be NULL (a router that is not trained); y is then not read and may be NULL.
 *   topk <= 1024, T * topk < 2^31; pointers aligned to their types, 16-byte aligned rows with H % 8 == 0 are
 *   faster.  T == 0 or topk == 0 launches nothing.
 */
int moe_topk_reduce_backward(const uint16_t* dout_bf16, int64_t dout_stride, const void* y, int y_dt, int64_t y_stride,
                             int64_t y_rows, const int32_t* slot_ids, const int32_t* route_rows, const float* weights,
                             int64_t T, int64_t topk, int64_t H, void* dy, int64_t dy_stride, float* dweights,
                             void* stream);

/*
 * moe_route_prep_backward  -- gradient of the router logits from the routing weights'
 *   dlogits[t, expert_ids[t, j]] = w_j * (dw_j - sum_i w_i dw_i), the softmax over the selected logits that
 *   moe_route_prep's weights are; every other entry +0.  An id outside [0, E) is skipped (its weight still
 *   counts in the sum); an id named twice gets the sum.
 *   expert_ids, weights, dweights [T][topk];  dlogits [T][dlogits_stride] fp32, E written.
 *   Requirements: 1 <= E <= 1024, 1 <= topk <= 64.  T == 0 launches nothing.
 */
int moe_route_prep_backward(const int32_t* expert_ids, const float* weights, const float* dweights, int64_t T,
                            int64_t E, int64_t topk, float* dlogits, int64_t dlogits_stride, void* stream);

/*
 * The router in its general form, and experts in MXFP4 on both sides
 *   The entry points from here on are not steps of the pages' method either.  moe_router is moe_route_prep with sigmoid or
 *   softmax scores, a balance bias, expert groups, masked experts and 16-bit logits, moe_router_backward its gradient.
 *   moe_mx4_* serve experts whose weights and activations are both MXFP4 (E2M1 codes, two a byte with the even element in
 *   the low nibble, one E8M0 scale byte per 32 elements: the format of moe_mxfp4_grouped_gemm's weights).  A prefill step is
 *     moe_router(logits);  xq = moe_mx4_quant(x);
 *     hq = moe_mx4_grouped_gemm_act_quant(xq, W13, a_rows = dst2src);  y = moe_mx4_grouped_gemm(hq, W2);
 *     out = moe_topk_reduce(y, slot_ids = expert_ids, route_rows)
 *   and a decode step the same in MOE_MODE_SLOT with slot_ids = expert_ids and a_row_div = topk instead of the maps.
 */

/* Scores of a router: s = softmax(logits) over the experts, or 1 / (1 + exp(-logit)) of each. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
/* Scale of an MXFP4 group: 2^(floor(log2 amax) - 2) (OCP MX; values above 6 scales saturate), or the least power of two
 * that holds amax without saturation (amax <= 6 scales). */
typedef enum { MOE_MX_FLOOR = 0, MOE_MX_CEIL = 1 } moe_mx_rule;

/*
 * moe_router  -- scores, choice, weights and route maps
 *   logits   DEVICE [T][logits_stride] of dt (MOE_BF16, MOE_F16 or MOE_F32), E used.  -inf and NaN mask their expert for that
 *            token (its score is 0); +inf counts as fp32's largest value, and fp32's lowest is a logit like any other.  (As a
 *            mask -inf is the quick one, in a bias too: fp32 logits ranked without a bias, and biased scores, leave the fast
 *            path where some lie beyond 1e30 or all that are not masked are equal: 6 to 8 us a token, one by one on a CU.)
 *   s        scores of the logits (moe_score).  The masked experts take no part in the softmax.
 *   c        choices s + bias (bias DEVICE fp32 [E]; a bias of -inf or NaN takes its expert from every choice), or, with bias
 *            NULL, the order of the logits themselves.
 *   groups   n_group groups of E / n_group consecutive experts; a group's value is its largest choice (group_top = 1) or
 *            the sum of its two largest (group_top = 2; a group with one choosable expert: that one's).  The topk_group
 *            groups of largest value stay.  (topk_group = n_group, as n_group = 1: all stay.)
 *   expert_ids [T][topk] int32: the topk largest choices in the groups that stay, descending; -1 where no choosable
 *            expert is left (an inactive route for every other entry point).
 *   weights  [T][topk] fp32: scale * s_j, or scale * s_j / sum_i s_i over the token's routes (renorm = 1; formed as
 *            ratios, so scores that underflow still divide); +0 where the id is -1.
 *   scores   [T][E] fp32: s, for an auxiliary loss; NULL: not wanted.  Formed in fp32 from the hardware's exponential: within
 *            (2.5 d + 48) 2^-24 of s, d the distance of the logit from the token's largest (sigmoid: from 0); one below 2^-126
 *            may be 0.  The weights are within 2^-18 of their value where that is 2^-126 or more.
 *   Ties go to the lower index, of experts and of groups.  Choices and sums of the two largest are formed in 64 bits and each
 *   rounded once to 43 significant bits for the comparison (those below 2^-1012 to fewer).
 *   dst2src, route_rows [T*topk], expert_offsets [E+1] int32: the route maps of moe_route_prep over the active routes;
 *   inactive routes have no row: their route_rows entry is -1, and the expert_offsets[E] rows are followed by dst2src
 *   entries of -1 (moe_gather_rows_scales and a_rows take these as rows of zeros).  All three NULL: not wanted.
 *   workspace: moe_router_workspace_size(T, E) bytes, 16-byte aligned, no initialization; 0 bytes (NULL allowed) up to
 *   64 tokens over up to 64 experts, up to 32 over more, and not used without maps.  Never less for more tokens or experts, so
 *   one sized for the largest batch serves the smaller ones.  Scratch within one call: overlapping calls need their own.
 *   Requirements: T <= 2^27, 1 <= E <= 1024, 1 <= topk <= min(E, 64), T * topk < 2^31; n_group <= 64 divides E,
 *   topk_group * (E / n_group) >= topk; scale positive and finite.  T == 0 with maps writes the zero offsets.
 */
size_t moe_router_workspace_size(int64_t T, int64_t E);
int moe_router(const void* logits, int dt, int64_t logits_stride, int64_t T, int64_t E, int64_t topk, int score,
               const float* bias, int64_t n_group, int64_t topk_group, int group_top, int renorm, float scale,
               int32_t* expert_ids, float* weights, float* scores, int32_t* dst2src, int32_t* route_rows,
               int32_t* expert_offsets, void* workspace, size_t ws_bytes, void* stream);

/*
 * moe_router_backward  -- gradient of the logits from the weights' and the scores'
 *   With n_j = w_j / scale and the sums over the token's routes (ids outside [0, E) are left out):
 *     renorm, softmax:  dl[e_j] += scale n_j (dw_j - sum_i n_i dw_i);   sigmoid: the same times (1 - s_j)
 *     not renorm:       u[e_j] += scale dw_j
 *   and u[e] += dscores[t, e] unless dscores is NULL; then dl[e] += s_e (u_e - sum_i s_i u_i) (softmax) or
 *   u_e s_e (1 - s_e) (sigmoid).  Masked experts' entries are +0.  bias and groups choose, they have no gradient.
 *   logits as moe_router's;  expert_ids, weights [T][topk] as it wrote them for these logits (an id named twice counts twice),
 *   dweights [T][topk];  dscores fp32 [T][dscores_stride], stride 0: one
 *   row for all tokens (an auxiliary loss on the batch's mean scores);  dlogits [T][dlogits_stride] of dt, E written.
 *   score, renorm, scale as in the forward call.  fp32 inside.  T == 0 launches nothing.
 */
int moe_router_backward(const void* logits, int dt, int64_t logits_stride, const int32_t* expert_ids, const float* weights,
                        const float* dweights, const float* dscores, int64_t dscores_stride, int64_t T, int64_t E,
                        int64_t topk, int score, int renorm, float scale, void* dlogits, int64_t dlogits_stride,
                        void* stream);

/*
 * moe_mx4_quant  -- rows, or a gated activation of them, to MXFP4
 *   act = MOE_ACT_IDENTITY: v = in[r, c];  moe_act 1..5: in row is [gate(0:n) | up(n:2n)], v = act(gate) * up in fp32.
 *   Per group of 32 columns (the last may be shorter): scale by `rule` (moe_mx_rule), at least 2^-127 (byte 0, also that
 *   of a group of zeros); codes e2m1_rne(v / scale), the quotient exact, saturating at 6.  Bit-exact for IDENTITY, RELU and
 *   MUL; v of the transcendental gates is, whatever dt, within (1.25 |gate| + 16) 2^-24 of its value (SiLU, sigmoid) or
 *   (1.25 gate^2 + 32) 2^-24 (GELU), and where act(gate) is below 2^-126 within 2^-150 |up| more.  A group that holds an
 *   infinity or NaN takes scale byte 255 (NaN) and codes 0: every value of it reads as NaN.
 *   in [rows][in_stride] of dt;  out_q [rows][q_stride] bytes, n/2 written;  out_s [rows][s_stride] bytes, ceil(n/32) written.
 *   Requirements: n even; in aligned to its type.  16-byte aligned rows with n % 8 == 0 and 4-byte aligned code rows take
 *   the vector path.  The products want scale rows at multiples of 4 bytes.
 */
int moe_mx4_quant(const void* in, int dt, int64_t in_stride, int64_t rows, int64_t n, int act, int rule,
                  uint8_t* out_q, int64_t q_stride, uint8_t* out_s, int64_t s_stride, void* stream);

/*
 * moe_mx4_dequant  -- MXFP4 rows back to values
 *   out[r, c] = code * scale, rounded once to out_dt: exact in fp32 (subnormals included) and bf16 (scales of 2^-126 and
 *   more); infinity past the type's largest value (fp16: 65504; fp32 and bf16: codes 4 and 6 under scales of 2^126 and 2^127,
 *   and 2 and 3 under 2^127).  NaN under scale byte 255.  Layouts as moe_mx4_quant.
 */
int moe_mx4_dequant(const uint8_t* q, int64_t q_stride, const uint8_t* s, int64_t s_stride, int64_t rows, int64_t n,
                    void* out, int out_dt, int64_t out_stride, void* stream);

/*
 * moe_mx4_grouped_gemm  -- the expert GEMM with MXFP4 on both sides
 *   out[r, n] = sum_k A[ar, k] 2^(a_s[ar, k/32] - 127) W[e, n, k] 2^(w_s[e, n, k/32] - 127), products exact, sums in fp32
 *   (the MFMA's, within 2^-23 of the sum of magnitudes per 128 products), one rounding to out_dt.
 *   a_q  [a_n][a_stride] codes (K/2 used), a_s [a_n][a_s_stride] scale bytes (K/32 used)
 *   w_q  codes of (e, n) at e*w_stride_e + n*w_stride_n, w_s scale bytes at e*w_s_stride_e + n*w_s_stride_n
 *   mode, expert_offsets, slot_ids, m_rows: as moe_b16_grouped_gemm (offsets that decrease somewhere leave all of out
 *        untouched; a slot outside [0, n_experts) writes a +0 row and reads nothing of it).
 *   ar   a_rows[r] (DEVICE int32 [m_rows]) if a_rows is given: an entry outside [0, a_n) is a row of zeros; else row r in
 *        grouped and r / a_row_div in slot mode, which have to lie below a_n.
 *   A scale byte of 255 makes exactly the outputs NaN whose sums hold it.
 *   Requirements: N % 8 == 0, K % 32 == 0, 8 <= N, 32 <= K, both <= 2^20; m_rows <= 2^31 - 1; 1 <= n_experts <= 1024 in
 *   grouped mode (0 allowed in slot mode); code rows 16-byte aligned; scale rows at multiples of 4 bytes and readable to the
 *   next one (strides >= 4 * ceil(K/128); what pads a row is not used); out aligned to its type.  Slot mode:
 *   m_rows * ceil(N / 16) < 2^24.  MOE_ERR_SHAPE, MOE_ERR_ALIGN otherwise.  m_rows == 0 launches nothing.
 */
int moe_mx4_grouped_gemm(const uint8_t* a_q, int64_t a_stride, const uint8_t* a_s, int64_t a_s_stride, int64_t a_n,
                         const int32_t* a_rows, const uint8_t* w_q, int64_t w_stride_e, int64_t w_stride_n,
                         const uint8_t* w_s, int64_t w_s_stride_e, int64_t w_s_stride_n, int64_t n_experts, int64_t N,
                         int64_t K, int mode, const int32_t* expert_offsets, const int32_t* slot_ids, int64_t m_rows,
                         int64_t a_row_div, void* out, int out_dt, int64_t out_stride, void* stream);

/* The output tile (rows, columns) that moe_mx4_grouped_gemm's grouped mode takes; pure function, as moe_b16_grouped_tile. */
int moe_mx4_grouped_tile(int64_t m_rows, int64_t n_experts, int64_t N, int64_t K, int32_t tile[2]);

/*
 * moe_mx4_grouped_gemm_act_quant  -- the gate/up GEMM with the gated activation and its MXFP4 requant in the epilogue
 *   c1 is the fp32 result of moe_mx4_grouped_gemm with N = 2I (W13 rows 0..I-1 gate, I..2I-1 up), never stored; out_q, out_s
 *   are moe_mx4_quant's of it with `act` (1..5) and `rule`.  The results equal moe_mx4_grouped_gemm with MOE_F32 output
 *   followed by moe_mx4_quant, bit for bit, in both modes.  Slot mode: an inactive route gets codes 0 and scale bytes 0.
 *   Grouped mode: rows from expert_offsets[n_experts] on, where moe_router leaves the inactive routes, stay as they were.
 *   Requirements: I % 32 == 0; out_q and q_stride even; slot mode: m_rows * I / 32 < 2^22; the rest as
 *   moe_mx4_grouped_gemm with N = 2I.
 */
int moe_mx4_grouped_gemm_act_quant(const uint8_t* a_q, int64_t a_stride, const uint8_t* a_s, int64_t a_s_stride, int64_t a_n,
                                   const int32_t* a_rows, const uint8_t* w_q, int64_t w_stride_e, int64_t w_stride_n,
                                   const uint8_t* w_s, int64_t w_s_stride_e, int64_t w_s_stride_n, int64_t n_experts,
                                   int64_t I, int64_t K, int mode, const int32_t* expert_offsets, const int32_t* slot_ids,
                                   int64_t m_rows, int64_t a_row_div, int act, int rule, uint8_t* out_q, int64_t q_stride,
                                   uint8_t* out_s, int64_t s_stride, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_ROUTED_H */
