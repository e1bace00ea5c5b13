"""Python binding of libmoe_routed (the MI355X routed-expert hot path).

Argument marshalling only: every function takes torch tensors that live on
the GPU, passes their device pointers, element strides and the current HIP
stream to the C entry point of the same name, and raises on a non-OK status.
No step of the path runs in Python or in torch, and there is no fallback: if
the shared library is missing, importing works but every call raises.

Dtypes: fp8 buffers are torch.uint8 (raw e4m3 codes), scales torch.float32,
slot ids / maps / offsets torch.int32, 16-bit outputs torch.bfloat16 or
torch.float16.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_routed.so")

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_WORKSPACE, MOE_ERR_ALIGN, MOE_ERR_HIP = 0, -1, -2, -3, -4, -5, -6
MOE_ERR_SCRATCH = -7
MOE_BF16, MOE_F32, MOE_F16, MOE_E4M3 = 0, 1, 2, 3
MOE_ACT_IDENTITY, MOE_ACT_SILU_MUL, MOE_ACT_GELU_MUL, MOE_ACT_RELU_MUL, MOE_ACT_SIGMOID_MUL, MOE_ACT_MUL = 0, 1, 2, 3, 4, 5
MOE_MODE_GROUPED, MOE_MODE_SLOT = 0, 1
MOE_W_PACKED = -1

EXPORTS = (
    "moe_abi_version", "moe_status_string", "moe_last_hip_error", "moe_gather_rows_scales", "moe_act_quant",
    "moe_pick_block_m", "moe_bf8_grouped_gemm", "moe_topk_reduce", "moe_fused_decode_workspace_size",
    "moe_fused_decode_workspace_layout", "moe_fused_decode_workspace_init", "moe_fused_decode",
    "moe_route_prep_workspace_size", "moe_route_prep", "moe_bf8_grouped_gemm_act_quant",
    "moe_mxfp4_grouped_gemm", "moe_mxfp4_grouped_gemm_act_quant", "moe_fused_decode_noalloc", "moe_pack_weights",
    "moe_grouped_block_m", "moe_b16_grouped_gemm", "moe_b16_grouped_tile", "moe_b16_grouped_wgrad", "moe_b16_grouped_wgrad_workspace_size",
    "moe_b16_grouped_wgrad_plan",
    "moe_act_checkpoint", "moe_gated_act_backward", "moe_topk_reduce_backward", "moe_route_prep_backward",
)

_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        L = lib()
        msg = L.moe_status_string(status).decode()
        if status == MOE_ERR_HIP:
            msg += ": " + L.moe_last_hip_error().decode()
        super().__init__("%s failed with status %d (%s)" % (fn, status, msg))
        self.status = status


def lib():
    """Load libmoe_routed.so (built in-tree by moe_routed_expert_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe_routed.so is not built (run moe_routed_expert_amd/build.py); "
                               "there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        sig = {
            "moe_abi_version": ([], I32),
            "moe_status_string": ([I32], ctypes.c_char_p),
            "moe_last_hip_error": ([], ctypes.c_char_p),
            "moe_gather_rows_scales": ([P, I64, P, I64, I64, I64, I64, P, I64, P, I64, P, I64, P], I32),
            "moe_act_quant": ([P, I32, I64, I64, I64, I32, P, I64, P, I64, P], I32),
            "moe_pick_block_m": ([I64, I64], I32),
            "moe_grouped_block_m": ([I64, I64, I64, I32, I32, I32], I32),
            "moe_bf8_grouped_gemm": ([P, I64, P, I64, P, I64, I64, P, I64, I64, I64, I64, I64, I32, P, P, I64, I64,
                                      ctypes.c_int32, P, I32, I64, P], I32),
            "moe_topk_reduce": ([P, I32, I64, P, P, P, I64, I64, I64, P, I64, P], I32),
            "moe_fused_decode_workspace_size": ([I64, I64, I64, I64], SZ),
            "moe_fused_decode_workspace_layout": ([I64, I64, I64, I64, P], I32),
            "moe_fused_decode_workspace_init": ([P, SZ, I64, I64, I64, I64, P], I32),
            "moe_fused_decode": ([P, I64, I64, I64, I64, I32, P, P, I64, P, P, P, P, P, SZ, P, P], I32),
            "moe_fused_decode_noalloc": ([P, I64, I64, I64, I64, I32, P, P, I64, P, P, P, P, P, P], I32),
            "moe_route_prep_workspace_size": ([I64, I64], SZ),
            "moe_route_prep": ([P, I64, I64, I64, I64, P, P, P, P, P, P, SZ, P], I32),
            "moe_bf8_grouped_gemm_act_quant": ([P, I64, P, I64, P, I64, I64, P, I64, I64, I64, I64, I64, P, I64,
                                                I32, I32, P, I64, P, I64, P], I32),
            "moe_mxfp4_grouped_gemm": ([P, I64, P, I64, P, I64, I64, P, I64, I64, I64, I64, I64, P, I64,
                                        I32, P, I32, I64, P], I32),
            "moe_mxfp4_grouped_gemm_act_quant": ([P, I64, P, I64, P, I64, I64, P, I64, I64, I64, I64, I64, P,
                                                  I64, I32, I32, P, I64, P, I64, P], I32),
            "moe_pack_weights": ([P, I64, I64, I64, I64, I64, I64, P, I64, P], I32),
            "moe_b16_grouped_gemm": ([P, I64, P, I64, I64, I64, I64, I64, I32, I32, I32, P, P, I64, I64, P, I32, I64,
                                      P], I32),
            "moe_b16_grouped_tile": ([I64, I64, I64, I64, P], I32),
            "moe_b16_grouped_wgrad_workspace_size": ([I64, I64, I64, I64], SZ),
            "moe_b16_grouped_wgrad_plan": ([I64, I64, I64, I64, P], I32),
            "moe_b16_grouped_wgrad": ([P, I64, I32, P, I64, I32, P, I64, P, I64, I64, I64, I64, P, I32, I64, I64, I32,
                                       P, SZ, P], I32),
            "moe_act_checkpoint": ([P, I32, I64, I64, I64, I32, P, I64, P, I64, P, I64, P], I32),
            "moe_gated_act_backward": ([P, I32, I64, P, I64, P, I64, I64, I64, I32, P, I64, P, I64, P], I32),
            "moe_topk_reduce_backward": ([P, I64, P, I32, I64, I64, P, P, P, I64, I64, I64, P, I64, P, P], I32),
            "moe_route_prep_backward": ([P, P, P, I64, I64, I64, P, I64, P], I32),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != MOE_OK:
        raise MoeError(fn, status)


def _ptr(t):
    if t is None:
        return None
    assert t.is_cuda, "device tensor expected"
    return t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


_DT = {torch.bfloat16: MOE_BF16, torch.float32: MOE_F32, torch.float16: MOE_F16}


def _dt(t: torch.Tensor) -> int:
    return _DT[t.dtype]


def _rowstride(t: torch.Tensor) -> int:
    assert t.dim() == 2 and t.stride(1) == 1, "row-major 2-D tensor with unit column stride expected"
    return t.stride(0)


# ---------------------------------------------------------------------------

def abi_version() -> int:
    return lib().moe_abi_version()


def pick_block_m(routes: int, experts: int) -> int:
    return lib().moe_pick_block_m(routes, experts)


def grouped_block_m(routes: int, experts: int, K: int, mxfp4: bool = False, packed: bool = False,
                    fused: bool = False) -> int:
    """The M tile the grouped GEMMs take for block_m = 0 (moe_grouped_block_m)."""
    return lib().moe_grouped_block_m(routes, experts, K, int(mxfp4), int(packed), int(fused))


def gather_rows_scales(src_q, src_s, dst2src, dst_q, dst_s, k=None, g=None, stream=None):
    """dst_q[i] = src_q[dst2src[i]] (bytes), dst_s[i] = src_s[dst2src[i]] (32-bit words)."""
    k = src_q.shape[1] if k is None else k
    g = src_s.shape[1] if g is None else g
    _check("moe_gather_rows_scales", lib().moe_gather_rows_scales(
        _ptr(src_q), _rowstride(src_q), _ptr(src_s), _rowstride(src_s), src_q.shape[0], k, g,
        _ptr(dst2src), dst2src.numel(), _ptr(dst_q), _rowstride(dst_q), _ptr(dst_s), _rowstride(dst_s),
        _stream(stream)))


def act_quant(x, out_q, out_s, act=MOE_ACT_IDENTITY, n=None, stream=None):
    """1x128 fp8 quantization of x rows (IDENTITY) or of SiLU(gate)*up (SILU_MUL, x = [gate | up])."""
    n = (x.shape[1] if act == MOE_ACT_IDENTITY else x.shape[1] // 2) if n is None else n
    _check("moe_act_quant", lib().moe_act_quant(
        _ptr(x), _dt(x), _rowstride(x), x.shape[0], n, act, _ptr(out_q), _rowstride(out_q), _ptr(out_s),
        _rowstride(out_s), _stream(stream)))


def pack_weights(w, step_bytes, out=None, stream=None):
    """The packed order of an expert bank (moe_pack_weights): w [E, N, row_bytes] bytes with unit last stride,
    step_bytes 128 for block-FP8 codes (row_bytes = K) or 64 for MXFP4 (row_bytes = K/2).  Returns out (a new
    contiguous [E, N, row_bytes] byte tensor when None), to be passed to the grouped GEMMs with w_packed=True."""
    E, N, RB = w.shape
    assert w.dtype == torch.uint8 and w.stride(2) == 1
    if out is None:
        out = torch.empty((E, N, RB), dtype=torch.uint8, device=w.device)
    assert out.dtype == torch.uint8 and tuple(out.shape) == (E, N, RB) and out.stride(2) == 1 and out.stride(1) == RB
    _check("moe_pack_weights", lib().moe_pack_weights(
        _ptr(w), w.stride(0), w.stride(1), E, N, RB, step_bytes, _ptr(out), out.stride(0), _stream(stream)))
    return out


def _w_strides(w, packed):
    """(expert stride, row stride) of a weight bank argument: MOE_W_PACKED as the row stride of a packed one."""
    if packed:
        assert w.stride(2) == 1 and w.stride(1) == w.shape[2], "a packed bank is contiguous per expert"
        return w.stride(0), MOE_W_PACKED
    return w.stride(0), w.stride(1)


def bf8_grouped_gemm(a_q, a_s, w_q, w_s, out, *, mode, expert_offsets=None, slot_ids=None, m_rows=None,
                     a_row_div=1, block_m=0, w_packed=False, stream=None):
    """Block-FP8 GEMM; w_q [E, N, K] (unit K stride; the packed order of pack_weights when w_packed),
    w_s [E, ceil(N/128), K/128]."""
    E, N, K = w_q.shape
    if m_rows is None:
        m_rows = out.shape[0]
    assert w_q.stride(2) == 1 and w_s.stride(2) == 1
    _check("moe_bf8_grouped_gemm", lib().moe_bf8_grouped_gemm(
        _ptr(a_q), _rowstride(a_q), _ptr(a_s), _rowstride(a_s),
        _ptr(w_q), *_w_strides(w_q, w_packed), _ptr(w_s), w_s.stride(0), w_s.stride(1),
        E, N, K, mode, _ptr(expert_offsets), _ptr(slot_ids), m_rows, a_row_div, block_m,
        _ptr(out), _dt(out), _rowstride(out), _stream(stream)))


def bf8_grouped_gemm_act_quant(a_q, a_s, w13_q, w13_s, expert_offsets, out_q, out_s, m_rows=None, block_m=0,
                               act=1, w_packed=False, stream=None):
    """Prefill gate/up GEMM with act(gate)*up (moe_act 1..5, default SwiGLU) and the 1x128 fp8 requant in
    its epilogue.
    w13_q [E, 2I, K] (gate rows, then up rows), w13_s [E, 2I/128, K/128]; out_q [rows, I] u8, out_s [rows, I/128]."""
    E, N, K = w13_q.shape
    if m_rows is None:
        m_rows = out_q.shape[0]
    assert w13_q.stride(2) == 1 and w13_s.stride(2) == 1
    _check("moe_bf8_grouped_gemm_act_quant", lib().moe_bf8_grouped_gemm_act_quant(
        _ptr(a_q), _rowstride(a_q), _ptr(a_s), _rowstride(a_s),
        _ptr(w13_q), *_w_strides(w13_q, w_packed), _ptr(w13_s), w13_s.stride(0), w13_s.stride(1),
        E, N // 2, K, _ptr(expert_offsets), m_rows, block_m, act, _ptr(out_q), _rowstride(out_q),
        _ptr(out_s), _rowstride(out_s), _stream(stream)))


def _mxfp4_weights(w4, w4_s):
    E, N, K2 = w4.shape
    assert w4.dtype == torch.uint8 and w4_s.dtype == torch.uint8, "MXFP4 weights are byte tensors"
    assert w4.stride(2) == 1 and w4_s.stride(2) == 1 and tuple(w4_s.shape) == (E, N, K2 // 16)
    return E, N, 2 * K2


def mxfp4_grouped_gemm(a_q, a_s, w4, w4_s, expert_offsets, out, m_rows=None, block_m=0, w_packed=False,
                       stream=None):
    """Grouped GEMM with MXFP4 weights: w4 [E, N, K/2] bytes (two E2M1 codes, even k in the low nibble),
    w4_s [E, N, K/32] E8M0 bytes; a_q/a_s/out as bf8_grouped_gemm in grouped mode."""
    E, N, K = _mxfp4_weights(w4, w4_s)
    if m_rows is None:
        m_rows = out.shape[0]
    _check("moe_mxfp4_grouped_gemm", lib().moe_mxfp4_grouped_gemm(
        _ptr(a_q), _rowstride(a_q), _ptr(a_s), _rowstride(a_s),
        _ptr(w4), *_w_strides(w4, w_packed), _ptr(w4_s), w4_s.stride(0), w4_s.stride(1),
        E, N, K, _ptr(expert_offsets), m_rows, block_m, _ptr(out), _dt(out), _rowstride(out), _stream(stream)))


def mxfp4_grouped_gemm_act_quant(a_q, a_s, w4, w4_s, expert_offsets, out_q, out_s, m_rows=None, block_m=0,
                                 act=1, w_packed=False, stream=None):
    """bf8_grouped_gemm_act_quant with MXFP4 gate/up weights w4 [E, 2I, K/2], w4_s [E, 2I, K/32]."""
    E, N, K = _mxfp4_weights(w4, w4_s)
    if m_rows is None:
        m_rows = out_q.shape[0]
    _check("moe_mxfp4_grouped_gemm_act_quant", lib().moe_mxfp4_grouped_gemm_act_quant(
        _ptr(a_q), _rowstride(a_q), _ptr(a_s), _rowstride(a_s),
        _ptr(w4), *_w_strides(w4, w_packed), _ptr(w4_s), w4_s.stride(0), w4_s.stride(1),
        E, N // 2, K, _ptr(expert_offsets), m_rows, block_m, act, _ptr(out_q), _rowstride(out_q),
        _ptr(out_s), _rowstride(out_s), _stream(stream)))


def topk_reduce(y, slot_ids, weights, out, route_rows=None, stream=None):
    """out[t] = bf16(sum over active j of weights[t,j] * y[row(t,j)])."""
    T, topk = slot_ids.shape
    H = out.shape[1]
    _check("moe_topk_reduce", lib().moe_topk_reduce(
        _ptr(y), _dt(y), _rowstride(y), _ptr(slot_ids), _ptr(route_rows), _ptr(weights), T, topk, H,
        _ptr(out), _rowstride(out), _stream(stream)))


def fused_decode_workspace_size(T, H, I, topk) -> int:
    return lib().moe_fused_decode_workspace_size(T, H, I, topk)


def fused_decode_workspace_layout(T, H, I, topk):
    offs = (ctypes.c_int64 * 7)()
    _check("moe_fused_decode_workspace_layout", lib().moe_fused_decode_workspace_layout(T, H, I, topk, offs))
    return dict(zip(("c1", "h", "aq", "as", "c2", "ctl", "total"), list(offs)))


def fused_decode_workspace(T, H, I, topk, device="cuda", stream=None) -> torch.Tensor:
    """Allocates (with torch) and initializes a workspace for moe_fused_decode."""
    size = fused_decode_workspace_size(T, H, I, topk)
    if size == 0:
        raise MoeError("moe_fused_decode_workspace_size", MOE_ERR_SHAPE)
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    _check("moe_fused_decode_workspace_init", lib().moe_fused_decode_workspace_init(
        _ptr(ws), size, T, H, I, topk, _stream(stream)))
    return ws


def fused_decode(x, slot_ids, weights, w13_q, w13_s, w2_q, w2_s, workspace, out, act=1, stream=None):
    """One routed-expert decode step: x [T, H] bf16 -> out [T, H] bf16."""
    T, H = x.shape
    topk = slot_ids.shape[1]
    S = w13_q.shape[0]
    I = w13_q.shape[1] // 2
    for t in (x, slot_ids, weights, w13_q, w13_s, w2_q, w2_s, out):
        assert t.is_contiguous()
    _check("moe_fused_decode", lib().moe_fused_decode(
        _ptr(x), T, H, I, topk, act, _ptr(slot_ids), _ptr(weights), S, _ptr(w13_q), _ptr(w13_s), _ptr(w2_q), _ptr(w2_s),
        _ptr(workspace), workspace.numel(), _ptr(out), _stream(stream)))


def fused_decode_noalloc(x, slot_ids, weights, w13_q, w13_s, w2_q, w2_s, out, act=1, stream=None):
    """fused_decode on the library's fixed device scratch (no workspace, nothing allocated)."""
    T, H = x.shape
    topk = slot_ids.shape[1]
    S = w13_q.shape[0]
    I = w13_q.shape[1] // 2
    for t in (x, slot_ids, weights, w13_q, w13_s, w2_q, w2_s, out):
        assert t.is_contiguous()
    _check("moe_fused_decode_noalloc", lib().moe_fused_decode_noalloc(
        _ptr(x), T, H, I, topk, act, _ptr(slot_ids), _ptr(weights), S, _ptr(w13_q), _ptr(w13_s), _ptr(w2_q),
        _ptr(w2_s), _ptr(out), _stream(stream)))


def route_prep(logits, topk, stream=None):
    """Top-k routing and the (expert, token)-ordered route maps of a prefill step.

    logits: [T, E] float32 on the GPU.  Returns (expert_ids [T,topk] i32, weights [T,topk] f32,
    dst2src [T*topk] i32, route_rows [T*topk] i32, expert_offsets [E+1] i32)."""
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
    w = torch.empty((T, topk), dtype=torch.float32, device=dev)
    d2s = torch.empty(T * topk, dtype=torch.int32, device=dev)
    rr = torch.empty(T * topk, dtype=torch.int32, device=dev)
    offs = torch.empty(E + 1, dtype=torch.int32, device=dev)
    size = lib().moe_route_prep_workspace_size(T, E)
    if size == 0:
        raise MoeError("moe_route_prep_workspace_size", MOE_ERR_SHAPE)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _check("moe_route_prep", lib().moe_route_prep(
        _ptr(logits), _rowstride(logits), T, E, topk, _ptr(ids) if T else None, _ptr(w) if T else None,
        _ptr(d2s) if T else None, _ptr(rr) if T else None, _ptr(offs), _ptr(ws), size, _stream(stream)))
    return ids, w, d2s, rr, offs


# ---------------------------------------------------------------------------
# 16-bit experts and the backward pass

# These wrappers are called once or more per layer, and a small operator's time is its call's: they read each tensor's
# properties once, in place.

_entry = {}          # C functions by name
_U8, _I32T, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_UNIT = "unit column stride expected"


def _call(fn, tensors, args, stream):
    """Calls C entry point fn(*args, stream) for tensors of one GPU, with that GPU current; stream None is its
    current stream, any other has to be one of that GPU's."""
    dev = tensors[0].get_device()
    assert dev >= 0, "tensors on a GPU expected"
    for t in tensors:
        assert t is None or t.get_device() == dev, "tensors of one GPU expected"
    assert stream is None or stream.device.index == dev, "a stream of the tensors' GPU expected"
    f = _entry.get(fn) or _entry.setdefault(fn, getattr(lib(), fn))
    if dev == _current_device():
        st = f(*args, _current_stream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, _current_stream(dev) if stream is None else stream.cuda_stream)
    if st != MOE_OK:
        raise MoeError(fn, st)


def _i32(t, n, what):
    assert t.dtype is _I32T and t.numel() == n and t.is_contiguous(), "%s: %d contiguous int32 expected" % (what, n)


def b16_grouped_gemm(a, w, out, *, mode, expert_offsets=None, slot_ids=None, m_rows=None, a_row_div=1,
                     w_trans=False, stream=None):
    """16-bit grouped GEMM: out[r] = a[r] @ w[e].T with w [E, N, K], or a[r] @ w[e] with w [E, K, N] when w_trans
    (the data gradient of a layer whose forward used the same bank).  a [rows, K] and w bf16 or fp16, out
    [rows, N] bf16, fp16 or fp32; rows by expert_offsets [E+1] (grouped) or slot_ids [m_rows] (slot mode)."""
    E, N, K = w.shape
    if w_trans:
        N, K = K, N
    w_e, w_r, w_1 = w.stride()
    a_rows, a_cols = a.shape
    a_r, a_1 = a.stride()
    o_rows, o_cols = out.shape
    o_r, o_1 = out.stride()
    dt = a.dtype
    rows = o_rows if m_rows is None else m_rows
    assert dt is w.dtype and a_cols == K and o_cols == N, "operands do not match"
    assert w_1 == 1 and a_1 == 1 and o_1 == 1, _UNIT
    assert 0 <= rows <= o_rows, "m_rows exceeds out"
    if mode == MOE_MODE_SLOT:
        _i32(slot_ids, rows, "slot_ids")
        assert a_rows * a_row_div >= rows, "a has too few rows"
        offs, slots = None if expert_offsets is None else expert_offsets.data_ptr(), slot_ids.data_ptr()
    else:
        _i32(expert_offsets, E + 1, "expert_offsets")
        assert a_rows >= rows, "a has too few rows"
        offs, slots = expert_offsets.data_ptr(), None if slot_ids is None else slot_ids.data_ptr()
    _call("moe_b16_grouped_gemm", (a, w, out, expert_offsets, slot_ids), (
        a.data_ptr(), a_r, w.data_ptr(), w_e, w_r, E, N, K, _DT[dt], 1 if w_trans else 0, mode, offs, slots, rows, a_row_div,
        out.data_ptr(), _DT[out.dtype], o_r), stream)


def b16_grouped_tile(m_rows, n_experts, N, K):
    """(rows, columns) of the output tile that b16_grouped_gemm's grouped mode takes."""
    t = (ctypes.c_int32 * 2)()
    _check("moe_b16_grouped_tile", lib().moe_b16_grouped_tile(m_rows, n_experts, N, K, t))
    return t[0], t[1]


def b16_grouped_wgrad_workspace_size(m_rows, n_experts, N, K) -> int:
    """Bytes of workspace b16_grouped_wgrad needs (0: none)."""
    return lib().moe_b16_grouped_wgrad_workspace_size(m_rows, n_experts, N, K)


def b16_grouped_wgrad_plan(m_rows, n_experts, N, K):
    """(tile rows, tile columns, rows of a chunk or 0) that b16_grouped_wgrad takes."""
    t = (ctypes.c_int32 * 3)()
    _check("moe_b16_grouped_wgrad_plan", lib().moe_b16_grouped_wgrad_plan(m_rows, n_experts, N, K, t))
    return tuple(t)


def b16_grouped_wgrad(dy, a, expert_offsets, dw, *, a_s=None, m_rows=None, accumulate=False, workspace=None,
                      stream=None):
    """Weight gradient dw[e] = dy[rows of e].T @ a[rows of e] (+ dw[e] when accumulate).  dy [rows, N] bf16 or
    fp16; a [rows, K] of dy's type, or uint8 e4m3 codes with scales a_s [rows, ceil(K/128)]; dw [E, N, K] bf16,
    fp16 or fp32.  workspace: uint8 tensor of b16_grouped_wgrad_workspace_size bytes, allocated here when None."""
    E, N, K = dw.shape
    rows = dy.shape[0] if m_rows is None else m_rows
    saved = a.dtype is _U8
    dy_rows, dy_cols = dy.shape
    a_rows, a_cols = a.shape
    dy_r, dy_1 = dy.stride()
    a_r, a_1 = a.stride()
    dw_e, dw_n, dw_1 = dw.stride()
    assert saved == (a_s is not None), "scales go with saved (uint8) rows"
    assert dy_cols == N and a_cols == K, "operands do not match"
    assert dy_1 == 1 and a_1 == 1 and dw_1 == 1, _UNIT
    assert 0 <= rows <= dy_rows and rows <= a_rows, "m_rows exceeds dy or a"
    s_r = 0
    if saved:
        assert a_s.dtype is _F32 and a_s.shape[0] >= rows and a_s.shape[1] >= (K + 127) // 128, "scales do not match"
        s_r, s_1 = a_s.stride()
        assert s_1 == 1, _UNIT
    _i32(expert_offsets, E + 1, "expert_offsets")
    size = b16_grouped_wgrad_workspace_size(rows, E, N, K)
    if size and workspace is None:
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(dy.device)):
            workspace = torch.empty(size, dtype=torch.uint8, device=dy.device)
    if workspace is not None:
        assert workspace.is_contiguous() and workspace.element_size() == 1, "workspace: contiguous bytes"
    _call("moe_b16_grouped_wgrad", (dy, a, a_s, expert_offsets, dw, workspace), (
        dy.data_ptr(), dy_r, _DT[dy.dtype], a.data_ptr(), a_r, MOE_E4M3 if saved else _DT[a.dtype],
        a_s.data_ptr() if saved else None, s_r, expert_offsets.data_ptr(), E, N, K, rows, dw.data_ptr(), _DT[dw.dtype],
        dw_e, dw_n, 1 if accumulate else 0, None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel()), stream)


def act_checkpoint(x, out_q, out_s, act=MOE_ACT_IDENTITY, h=None, stream=None):
    """Saves rows x in 8 bits (e4m3 codes out_q, power-of-two scales out_s per 1x128 group).  With a gated act, x =
    [gate | up]: both halves are saved and h = act(gate) * up (x's type) is written when given."""
    rows, width = x.shape
    n = width if act == MOE_ACT_IDENTITY else width // 2
    both = 1 if act == MOE_ACT_IDENTITY else 2
    dt = x.dtype
    x_r, x_1 = x.stride()
    q_r, q_1 = out_q.stride()
    s_r, s_1 = out_s.stride()
    assert width == both * n, "gate and up of one width expected"
    assert out_q.dtype is _U8 and out_s.dtype is _F32, "codes are uint8, scales float32"
    assert out_q.shape == (rows, width) and out_s.shape == (rows, both * ((n + 127) // 128)), "outputs do not match"
    assert x_1 == 1 and q_1 == 1 and s_1 == 1, _UNIT
    h_r, h_p = 0, None
    if h is not None:
        h_r, h_1 = h.stride()
        h_p = h.data_ptr()
        assert h.dtype is dt and h.shape == (rows, n) and h_1 == 1, "h does not match"
    _call("moe_act_checkpoint", (x, out_q, out_s, h), (
        x.data_ptr(), _DT[dt], x_r, rows, n, act, out_q.data_ptr(), q_r, out_s.data_ptr(), s_r, h_p, h_r), stream)


def gated_act_backward(dh, q, s, dx, act=MOE_ACT_SILU_MUL, h=None, stream=None):
    """Backward of h = act(gate) * up from saved codes q [rows, 2n] and scales s: dx [rows, 2n] = [d gate | d up],
    and h [rows, n] again when given.  dh, dx, h of one type."""
    rows, n = dh.shape
    dt = dh.dtype
    d_r, d_1 = dh.stride()
    q_r, q_1 = q.stride()
    s_r, s_1 = s.stride()
    x_r, x_1 = dx.stride()
    wide = (rows, 2 * n)
    assert q.dtype is _U8 and s.dtype is _F32, "codes are uint8, scales float32"
    assert q.shape == wide and s.shape == (rows, 2 * ((n + 127) // 128)), "saved rows do not match"
    assert dx.dtype is dt and dx.shape == wide, "dx does not match"
    assert d_1 == 1 and q_1 == 1 and s_1 == 1 and x_1 == 1, _UNIT
    h_r, h_p = 0, None
    if h is not None:
        h_r, h_1 = h.stride()
        h_p = h.data_ptr()
        assert h.dtype is dt and h.shape == (rows, n) and h_1 == 1, "h does not match"
    _call("moe_gated_act_backward", (dh, q, s, dx, h), (
        dh.data_ptr(), _DT[dt], d_r, q.data_ptr(), q_r, s.data_ptr(), s_r, rows, n, act, dx.data_ptr(), x_r, h_p, h_r),
        stream)


def topk_reduce_backward(dout, y, slot_ids, weights, dy, dweights=None, route_rows=None, stream=None):
    """Backward of topk_reduce: dy[row(t,j)] = weights[t,j] * dout[t], dweights[t,j] = <dout[t], y[row(t,j)]>.
    dout [T, H] bf16; y (None when dweights is None) and dy [rows, H] of one type.  With route_rows the rows of dropped
    routes (negative slots) are left as they were: call dy.zero_() first if expert offsets count them."""
    routes = slot_ids.shape
    T, topk = routes
    rows, H = dy.shape
    dt = dy.dtype
    d_r, d_1 = dout.stride()
    o_r, o_1 = dy.stride()
    _i32(slot_ids, T * topk, "slot_ids")
    assert dout.dtype is _BF16 and dout.shape == (T, H), "dout: [T, H] bfloat16"
    assert weights.dtype is _F32 and weights.is_contiguous() and weights.shape == routes, "weights do not match"
    assert d_1 == 1 and o_1 == 1, _UNIT
    y_r, y_p, dw_p, rr_p = 0, None, None, None
    if dweights is not None:
        assert dweights.dtype is _F32 and dweights.is_contiguous() and dweights.shape == routes, "dweights do not match"
        dw_p = dweights.data_ptr()
    if y is not None:
        y_r, y_1 = y.stride()
        y_p = y.data_ptr()
        assert y.dtype is dt and y.shape == (rows, H) and y_1 == 1, "y does not match dy"
    if route_rows is not None:
        _i32(route_rows, T * topk, "route_rows")
        rr_p = route_rows.data_ptr()
    else:
        assert rows >= T * topk, "a row for every route expected"
    _call("moe_topk_reduce_backward", (dout, y, slot_ids, route_rows, weights, dy, dweights), (
        dout.data_ptr(), d_r, y_p, _DT[dt], y_r, rows, slot_ids.data_ptr(), rr_p, weights.data_ptr(), T, topk, H,
        dy.data_ptr(), o_r, dw_p), stream)


def route_prep_backward(expert_ids, weights, dweights, dlogits, stream=None):
    """Router gradient: dlogits [T, E] from route_prep's expert_ids and weights and the weights' gradient."""
    routes = expert_ids.shape
    T, topk = routes
    rows, E = dlogits.shape
    l_r, l_1 = dlogits.stride()
    _i32(expert_ids, T * topk, "expert_ids")
    assert weights.dtype is _F32 and weights.is_contiguous() and weights.shape == routes, "weights do not match"
    assert dweights.dtype is _F32 and dweights.is_contiguous() and dweights.shape == routes, "dweights do not match"
    assert dlogits.dtype is _F32 and rows == T and l_1 == 1, "dlogits: [T, E] float32"
    _call("moe_route_prep_backward", (expert_ids, weights, dweights, dlogits), (
        expert_ids.data_ptr(), weights.data_ptr(), dweights.data_ptr(), T, E, topk, dlogits.data_ptr(), l_r), stream)
