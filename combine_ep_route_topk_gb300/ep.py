"""Thin Python binding of libep_gb300 (the C ABI declared in include/ep.h).

Argument marshalling only: every function checks that its tensors are CUDA
tensors of the expected dtype and shape, passes their device pointers and the
current CUDA stream to the C function of the same name, and raises EPError
on a non-zero status.  Output tensors may be passed in (for reuse or CUDA
graph capture) or are allocated with torch.empty.  There is no CPU path: if
the shared library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from collections import namedtuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libep_gb300.so")

EP_LAYOUT_CONTIG = 0
EP_LAYOUT_MASKED = 1
EP_DTYPE_BF16 = 0
EP_DTYPE_FP8_E4M3_B128 = 1
EP_DTYPE_F32 = 2
EP_SCORE_SOFTMAX = 0
EP_SCORE_SIGMOID = 1
EP_ACT_NONE = 0
EP_ACT_SWIGLU = 1

_FLOATS = {torch.bfloat16: EP_DTYPE_BF16, torch.float32: EP_DTYPE_F32}

_lib = None


class EPError(RuntimeError):
    pass


def lib():
    """The loaded libep_gb300 (loads it on first use; raises if it is absent)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise EPError(f"{LIB_PATH} is not built; run combine_ep_route_topk_gb300.build.build() "
                          "(nvcc, sm_103a). There is no fallback implementation.")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        L.ep_route_topk.argtypes = [P, i32, i32, i32, P, P, P, P]
        L.ep_expert_balance_map.argtypes = [P, i32, i32, P, P]
        L.ep_dispatch_layout_workspace_size.argtypes = [i32, i32, i32, i32]
        L.ep_dispatch_layout_workspace_size.restype = sz
        L.ep_dispatch_layout.argtypes = [P, P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P,
                                         sz, P]
        L.ep_route_layout_workspace_size.argtypes = [i32, i32, i32, i32]
        L.ep_route_layout_workspace_size.restype = sz
        L.ep_route_layout.argtypes = [P, P, i32, i32, i32, i32, P, i32, P, P, P, P, P, P, P, P, P,
                                      P, P, sz, P]
        L.ep_route_layout.restype = ctypes.c_int
        L.ep_dispatch.argtypes = [P, i32, i32, i32, i32, P, P, P, ctypes.c_int, i32, ctypes.c_int,
                                  P, P, P]
        L.ep_combine.argtypes = [P, i32, i32, i32, i32, P, P, P, P, ctypes.c_int, i32, P, P]
        L.ep_selftest_wait_timeout.argtypes = [P, P, sz, P]
        L.ep_route_dispatch_workspace_size.argtypes = [i32, i32, i32, i32]
        L.ep_route_dispatch_workspace_size.restype = sz
        L.ep_route_dispatch.argtypes = [P, P, P, i32, i32, i32, i32, i32, P, ctypes.c_int, i32,
                                        ctypes.c_int, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.ep_route_dispatch.restype = ctypes.c_int
        L.ep_host_pipeline_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32,
                                                      ctypes.c_int, i32]
        L.ep_host_pipeline_workspace_size.restype = sz
        L.ep_host_pipeline_create.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.c_int, i32, P,
                                              P, sz, ctypes.POINTER(P)]
        L.ep_host_pipeline_step.argtypes = [P, P, P, P, P, P, P]
        L.ep_host_pipeline_join.argtypes = [P, P]
        L.ep_host_pipeline_copy_ms.argtypes = [P, ctypes.POINTER(ctypes.c_float),
                                               ctypes.POINTER(ctypes.c_float)]
        L.ep_host_pipeline_copy_ms.restype = ctypes.c_int
        L.ep_host_pipeline_buffer.argtypes = [P, ctypes.c_int, ctypes.POINTER(P),
                                              ctypes.POINTER(sz)]
        L.ep_host_pipeline_destroy.argtypes = [P]
        L.ep_host_alloc.argtypes = [sz, ctypes.POINTER(P)]
        L.ep_host_alloc.restype = ctypes.c_int
        L.ep_host_free.argtypes = [P]
        L.ep_host_free.restype = ctypes.c_int
        for f in ("ep_route_topk", "ep_expert_balance_map", "ep_dispatch_layout", "ep_dispatch",
                  "ep_combine"):
            getattr(L, f).restype = ctypes.c_int
        f32, enum = ctypes.c_float, ctypes.c_int
        L.ep_gate_topk.argtypes = [P, enum, i32, i32, i32, enum, P, i32, i32, i32, i32, f32, P, P,
                                   P, P]
        L.ep_gate_topk_picks.argtypes = [P, enum, i32, i32, i32, enum, P, i32, i32, i32, i32, f32,
                                         P, P, P, P, P]
        L.ep_gate_topk_backward.argtypes = [P, P, enum, P, i32, i32, i32, enum, i32, f32, P, P, P]
        L.ep_quantize_rows.argtypes = [P, enum, enum, i32, i32, P, i32, enum, i32, P, P, P]
        L.ep_expert_matmul.argtypes = [P, P, i32, P, P, i32, i32, i32, P, enum, i32, i32, P, i32,
                                       enum, P, P, P]
        L.ep_quantize_blocks.argtypes = [P, enum, enum, i32, i32, P, i32, enum, i32, P, P, P, P, P]
        L.ep_dequantize_blocks.argtypes = [P, P, i32, i32, P, i32, enum, i32, enum, P, P]
        L.ep_swiglu_backward.argtypes = [P, enum, P, P, i32, i32, P, i32, enum, i32, P, P]
        L.ep_expert_matmul_fp8.argtypes = L.ep_expert_matmul.argtypes
        L.ep_rms_norm.argtypes = [P, enum, P, P, enum, i32, i32, f32, P, P, P, P, P, P]
        L.ep_rms_norm_backward_workspace_size.argtypes = [i32, i32]
        L.ep_rms_norm_backward_workspace_size.restype = sz
        L.ep_rms_norm_backward.argtypes = [P, enum, P, P, enum, P, P, i32, i32, P, P, P, sz, P]
        for f in ("ep_gate_topk", "ep_gate_topk_picks", "ep_gate_topk_backward",
                  "ep_quantize_rows", "ep_expert_matmul", "ep_quantize_blocks",
                  "ep_dequantize_blocks", "ep_swiglu_backward", "ep_expert_matmul_fp8",
                  "ep_rms_norm", "ep_rms_norm_backward"):
            getattr(L, f).restype = ctypes.c_int
        L.ep_status_string.argtypes = [ctypes.c_int]
        L.ep_status_string.restype = ctypes.c_char_p
        L.ep_last_cuda_error.argtypes = []
        L.ep_last_cuda_error.restype = ctypes.c_char_p
        L.ep_kernel_launch_count.argtypes = []
        L.ep_kernel_launch_count.restype = ctypes.c_uint64
        L.ep_abi_version.argtypes = []
        L.ep_abi_version.restype = ctypes.c_int32
        _lib = L
    return _lib


def _check(name, status):
    if status != 0:
        L = lib()
        raise EPError(f"{name}: {L.ep_status_string(status).decode()}"
                      f" {L.ep_last_cuda_error().decode()}".rstrip())


def _dev(t, dtype, name, shape=None):
    """Device pointer of a tensor after the checks (one expression on the usual
    path: a call's host time is a few microseconds, so every check counts)."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous() and \
            (shape is None or t.shape == shape):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise EPError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise EPError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise EPError(f"{name} must be contiguous")
    raise EPError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _opt(t, dtype, name, shape=None):
    return None if t is None else _dev(t, dtype, name, shape)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    """Handle of the given or the current stream (torch.cuda.current_stream()
    builds a Stream object, 3 us; the raw handle takes 0.2)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _raw_device is not None:
        return _raw_stream(_raw_device())
    return torch.cuda.current_stream().cuda_stream


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def ep_kernel_launch_count() -> int:
    return int(lib().ep_kernel_launch_count())


def ep_route_topk(logits, K, expert_map=None, topk_idx=None, topk_w=None, stream=None):
    """logits float32 [N, E] -> (topk_idx int32 [N, K], topk_w float32 [N, K])."""
    N, E = logits.shape
    if topk_idx is None:
        topk_idx = _empty((N, K), torch.int32, logits)
    if topk_w is None:
        topk_w = _empty((N, K), torch.float32, logits)
    _check("ep_route_topk", lib().ep_route_topk(
        _dev(logits, torch.float32, "logits"), N, E, K,
        _opt(expert_map, torch.int32, "expert_map", (E,)),
        _dev(topk_idx, torch.int32, "topk_idx", (N, K)),
        _dev(topk_w, torch.float32, "topk_w", (N, K)), _stream(stream)))
    return topk_idx, topk_w


def ep_expert_balance_map(counts, expert_map=None, stream=None):
    """counts int32 [R, E] -> expert_map int32 [E] (old id -> new id)."""
    R, E = counts.shape
    if expert_map is None:
        expert_map = _empty((E,), torch.int32, counts)
    _check("ep_expert_balance_map", lib().ep_expert_balance_map(
        _dev(counts, torch.int32, "counts"), R, E,
        _dev(expert_map, torch.int32, "expert_map", (E,)), _stream(stream)))
    return expert_map


def ep_dispatch_layout_workspace_size(N, E, K, R) -> int:
    return int(lib().ep_dispatch_layout_workspace_size(N, E, K, R))


Layout = namedtuple("Layout", "counts expert_offsets rank_expert_offsets pos row_src masked_m "
                              "overflow_count")


def alloc_layout(N, E, K, R, cap, device):
    def z(*s):
        return torch.empty(s, dtype=torch.int32, device=device)
    return Layout(z(R, E), z(E + 1), z(R, E), z(N, K), z(N * K),
                  z(E) if cap > 0 else None, z(1) if cap > 0 else None)


def ep_dispatch_layout(topk_idx, rank_offsets, E, cap=0, out: Layout | None = None,
                       workspace=None, stream=None) -> Layout:
    """Counts, offsets and the stable expert-major permutation of the picks."""
    N, K = topk_idx.shape
    R = rank_offsets.shape[0] - 1
    if out is None:
        out = alloc_layout(N, E, K, R, cap, topk_idx.device)
    need = ep_dispatch_layout_workspace_size(N, E, K, R)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=topk_idx.device)
    _check("ep_dispatch_layout", lib().ep_dispatch_layout(
        _dev(topk_idx, torch.int32, "topk_idx"), _dev(rank_offsets, torch.int32, "rank_offsets"),
        R, N, E, K, cap,
        _dev(out.counts, torch.int32, "counts", (R, E)),
        _dev(out.expert_offsets, torch.int32, "expert_offsets", (E + 1,)),
        _dev(out.rank_expert_offsets, torch.int32, "rank_expert_offsets", (R, E)),
        _dev(out.pos, torch.int32, "pos", (N, K)),
        _dev(out.row_src, torch.int32, "row_src", (N * K,)),
        _opt(out.masked_m, torch.int32, "masked_m", (E,)),
        _opt(out.overflow_count, torch.int32, "overflow_count", (1,)),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)))
    return out


def ep_route_layout_workspace_size(N, E, K, R) -> int:
    return int(lib().ep_route_layout_workspace_size(N, E, K, R))


def ep_route_layout(logits, rank_offsets, K, cap=0, expert_map=None, topk_idx=None,
                    topk_w=None, out: Layout | None = None, status=None, workspace=None,
                    stream=None):
    """ep_route_topk + ep_dispatch_layout in one cooperative kernel.
    Returns (topk_idx, topk_w, Layout)."""
    N, E = logits.shape
    R = rank_offsets.shape[0] - 1
    if topk_idx is None:
        topk_idx = _empty((N, K), torch.int32, logits)
    if topk_w is None:
        topk_w = _empty((N, K), torch.float32, logits)
    if out is None:
        out = alloc_layout(N, E, K, R, cap, logits.device)
    need = ep_route_layout_workspace_size(N, E, K, R)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=logits.device)
    _check("ep_route_layout", lib().ep_route_layout(
        _dev(logits, torch.float32, "logits"), _dev(rank_offsets, torch.int32, "rank_offsets"),
        R, N, E, K, _opt(expert_map, torch.int32, "expert_map", (E,)), cap,
        _dev(topk_idx, torch.int32, "topk_idx", (N, K)),
        _dev(topk_w, torch.float32, "topk_w", (N, K)),
        _dev(out.counts, torch.int32, "counts", (R, E)),
        _dev(out.expert_offsets, torch.int32, "expert_offsets", (E + 1,)),
        _dev(out.rank_expert_offsets, torch.int32, "rank_expert_offsets", (R, E)),
        _dev(out.pos, torch.int32, "pos", (N, K)),
        _dev(out.row_src, torch.int32, "row_src", (N * K,)),
        _opt(out.masked_m, torch.int32, "masked_m", (E,)),
        _opt(out.overflow_count, torch.int32, "overflow_count", (1,)),
        _opt(status, torch.int32, "status", (1,)),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)))
    return topk_idx, topk_w, out


def ep_route_dispatch_workspace_size(N, E, K, R) -> int:
    return int(lib().ep_route_dispatch_workspace_size(N, E, K, R))


def ep_route_dispatch(logits, rank_offsets, x, K, layout=EP_LAYOUT_CONTIG, cap=0,
                      dtype=EP_DTYPE_BF16, expert_map=None, topk_idx=None, topk_w=None,
                      lay: Layout | None = None, out=None, out_scales=None, workspace=None,
                      stream=None):
    """ep_route_topk + ep_dispatch_layout + ep_dispatch in one call (two
    launches up to 2048 tokens and 16384 picks).  Returns (topk_idx, topk_w,
    Layout, out, out_scales) as the three calls would."""
    N, E = logits.shape
    H = x.shape[1]
    R = rank_offsets.shape[0] - 1
    if topk_idx is None:
        topk_idx = _empty((N, K), torch.int32, logits)
    if topk_w is None:
        topk_w = _empty((N, K), torch.float32, logits)
    if lay is None:
        lay = alloc_layout(N, E, K, R, cap, logits.device)
    rows = dispatch_rows(N, K, E, layout, cap)
    if dtype == EP_DTYPE_BF16:
        if out is None:
            out = _empty((rows, H), torch.bfloat16, x)
        po = _dev(out, torch.bfloat16, "out")
    else:
        if out is None:
            out = _empty((rows, H), torch.uint8, x)
        if out_scales is None:
            out_scales = _empty((rows, H // 128), torch.float32, x)
        po = _dev(out, torch.uint8, "out")
    if out.numel() != rows * H:
        raise EPError(f"out must hold {rows} x {H} elements")
    if out_scales is not None and out_scales.numel() != rows * (H // 128):
        raise EPError(f"out_scales must hold {rows} x {H // 128} elements")
    if workspace is None:
        workspace = torch.empty(ep_route_dispatch_workspace_size(N, E, K, R), dtype=torch.uint8,
                                device=logits.device)
    _check("ep_route_dispatch", lib().ep_route_dispatch(
        _dev(logits, torch.float32, "logits"), _dev(rank_offsets, torch.int32, "rank_offsets"),
        _dev(x, torch.bfloat16, "x"), R, N, H, E, K,
        _opt(expert_map, torch.int32, "expert_map", (E,)), layout, cap, dtype,
        _dev(topk_idx, torch.int32, "topk_idx", (N, K)),
        _dev(topk_w, torch.float32, "topk_w", (N, K)),
        _dev(lay.counts, torch.int32, "counts", (R, E)),
        _dev(lay.expert_offsets, torch.int32, "expert_offsets", (E + 1,)),
        _dev(lay.rank_expert_offsets, torch.int32, "rank_expert_offsets", (R, E)),
        _dev(lay.pos, torch.int32, "pos", (N, K)),
        _dev(lay.row_src, torch.int32, "row_src", (N * K,)),
        _opt(lay.masked_m, torch.int32, "masked_m", (E,)),
        _opt(lay.overflow_count, torch.int32, "overflow_count", (1,)), po,
        _opt(out_scales, torch.float32, "out_scales"),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _stream(stream)))
    return topk_idx, topk_w, lay, out, out_scales


def dispatch_rows(N, K, E, layout, cap):
    return N * K if layout == EP_LAYOUT_CONTIG else E * cap


def ep_dispatch(x, topk_idx, pos, expert_offsets, E, layout=EP_LAYOUT_CONTIG, cap=0,
                dtype=EP_DTYPE_BF16, out=None, out_scales=None, stream=None):
    """Scatter x [N, H] bf16 into the expert-major buffer.  Returns
    (out, out_scales): out bf16 [rows, H] or uint8 FP8 codes [rows, H];
    out_scales float32 [rows, H/128] for FP8, else None."""
    N, H = x.shape
    K = topk_idx.shape[1]
    rows = dispatch_rows(N, K, E, layout, cap)
    if dtype == EP_DTYPE_BF16:
        if out is None:
            out = _empty((rows, H), torch.bfloat16, x)
        po = _dev(out, torch.bfloat16, "out")
    else:
        if out is None:
            out = _empty((rows, H), torch.uint8, x)
        if out_scales is None:
            out_scales = _empty((rows, H // 128), torch.float32, x)
        po = _dev(out, torch.uint8, "out")
    if out.numel() != rows * H:
        raise EPError(f"out must hold {rows} x {H} elements")
    if out_scales is not None and out_scales.numel() != rows * (H // 128):
        raise EPError(f"out_scales must hold {rows} x {H // 128} elements")
    _check("ep_dispatch", lib().ep_dispatch(
        _dev(x, torch.bfloat16, "x"), N, H, E, K, _dev(topk_idx, torch.int32, "topk_idx", (N, K)),
        _dev(pos, torch.int32, "pos", (N, K)),
        _opt(expert_offsets, torch.int32, "expert_offsets", (E + 1,)), layout, cap, dtype, po,
        _opt(out_scales, torch.float32, "out_scales"), _stream(stream)))
    return out, out_scales


def ep_combine(y, topk_idx, topk_w, pos, expert_offsets, E, layout=EP_LAYOUT_CONTIG, cap=0,
               out=None, stream=None):
    """K-way weighted sum of expert outputs y back to token order: [N, H] bf16."""
    N, K = topk_idx.shape
    H = y.shape[-1]
    rows = dispatch_rows(N, K, E, layout, cap)
    if y.numel() != rows * H:
        raise EPError(f"y must hold {rows} x {H} elements")
    if out is None:
        out = _empty((N, H), torch.bfloat16, y)
    _check("ep_combine", lib().ep_combine(
        _dev(y, torch.bfloat16, "y"), N, H, E, K, _dev(topk_idx, torch.int32, "topk_idx", (N, K)),
        _dev(topk_w, torch.float32, "topk_w", (N, K)), _dev(pos, torch.int32, "pos", (N, K)),
        _opt(expert_offsets, torch.int32, "expert_offsets", (E + 1,)), layout, cap,
        _dev(out, torch.bfloat16, "out", (N, H)), _stream(stream)))
    return out


def _float_type(t, name):
    d = _FLOATS.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if d is None:
        raise EPError(f"{name} must be a bfloat16 or float32 tensor")
    return d


def ep_gate_topk(logits, K, score=EP_SCORE_SOFTMAX, bias=None, groups=1, topk_groups=None,
                 group_top=2, renorm=True, scale=1.0, expert_map=None, topk_idx=None,
                 topk_w=None, stream=None, picks=None):
    """logits bf16 or float32 [N, E] -> (topk_idx int32 [N, K], topk_w float32
    [N, K]): softmax or sigmoid scores, optional balance bias [E] on the choice
    alone, the best topk_groups of `groups` groups, the K best experts, their
    scores (renormalised) times scale.  picks: int32 [N, K] that receives the
    ids before expert_map, for ep_gate_topk_backward."""
    N, E = logits.shape
    dt = _float_type(logits, "logits")
    if topk_idx is None:
        topk_idx = _empty((N, K), torch.int32, logits)
    if topk_w is None:
        topk_w = _empty((N, K), torch.float32, logits)
    _check("ep_gate_topk", lib().ep_gate_topk_picks(
        _dev(logits, logits.dtype, "logits"), dt, N, E, K, score,
        _opt(bias, torch.float32, "bias", (E,)), groups,
        groups if topk_groups is None else topk_groups, group_top, int(renorm), scale,
        _opt(expert_map, torch.int32, "expert_map", (E,)),
        _dev(topk_idx, torch.int32, "topk_idx", (N, K)),
        _dev(topk_w, torch.float32, "topk_w", (N, K)),
        _opt(picks, torch.int32, "picks", (N, K)), _stream(stream)))
    return topk_idx, topk_w


def ep_gate_topk_backward(d_topk_w, logits, topk_idx, score=EP_SCORE_SOFTMAX, renorm=True,
                          scale=1.0, expert_map=None, d_logits=None, stream=None):
    """Gradient of ep_gate_topk's weights: d_topk_w float32 [N, K] -> d_logits
    [N, E] of the logits' type.  topk_idx: the forward call's picks; or, with
    its expert_map, its topk_idx, where that map is a renumbering."""
    N, E = logits.shape
    K = topk_idx.shape[1]
    dt = _float_type(logits, "logits")
    if d_logits is None:
        d_logits = torch.empty_like(logits)
    _check("ep_gate_topk_backward", lib().ep_gate_topk_backward(
        _dev(d_topk_w, torch.float32, "d_topk_w", (N, K)), _dev(logits, logits.dtype, "logits"),
        dt, _dev(topk_idx, torch.int32, "topk_idx", (N, K)), N, E, K, score, int(renorm), scale,
        _opt(expert_map, torch.int32, "expert_map", (E,)),
        _dev(d_logits, logits.dtype, "d_logits", (N, E)), _stream(stream)))
    return d_logits


def ep_quantize_rows(x, act=EP_ACT_NONE, expert_offsets=None, layout=EP_LAYOUT_CONTIG, cap=0,
                     q=None, scales=None, stream=None):
    """x bf16 or float32 [rows, cols] (EP_ACT_SWIGLU: [rows, 2*cols]) -> (q int8
    [rows, cols], scales float32 [rows]).  With expert_offsets, rows that hold
    no token are skipped."""
    rows, wide = x.shape
    cols = wide // 2 if act == EP_ACT_SWIGLU else wide
    dt = _float_type(x, "x")
    if act == EP_ACT_SWIGLU and wide % 2:
        raise EPError("x must have an even number of columns for SwiGLU")
    if q is None:
        q = _empty((rows, cols), torch.int8, x)
    if scales is None:
        scales = _empty((rows,), torch.float32, x)
    _check("ep_quantize_rows", lib().ep_quantize_rows(
        _dev(x, x.dtype, "x"), dt, act, rows, cols,
        _opt(expert_offsets, torch.int32, "expert_offsets"),
        0 if expert_offsets is None else expert_offsets.numel() - 1, layout, cap,
        _dev(q, torch.int8, "q", (rows, cols)), _dev(scales, torch.float32, "scales", (rows,)),
        _stream(stream)))
    return q, scales


def _sources(row_src, expert_offsets):
    """(pointer, length) of row_src.  An empty tensor has no memory, and a null pointer would
    say that there is no row_src: it gets an address that is never read."""
    if row_src is None:
        return None, 0
    n = row_src.numel()
    return _dev(row_src, torch.int32, "row_src") or expert_offsets.data_ptr(), n


def ep_expert_matmul(x, x_scales, w, w_scales, expert_offsets, layout=EP_LAYOUT_CONTIG, cap=0,
                     row_src=None, out=None, out_dtype=torch.bfloat16, status=None, stream=None):
    """Every expert's rows times its weights: x int8 [x_rows, Kd], x_scales
    float32 [x_rows], w int8 [E, Nc, Kd], w_scales float32 [E, Nc] -> out bf16
    or float32 [rows, Nc] ([E*cap, Nc] for the masked layout).  With row_src
    (the layout's), x holds token rows.  Rows that hold no token are not
    written."""
    E, Nc, Kd = w.shape
    x_rows = x.shape[0]
    if layout == EP_LAYOUT_MASKED:
        rows = E * cap
    else:
        rows = x_rows if row_src is None else row_src.numel()
    if out is None:
        out = _empty((rows, Nc), out_dtype, x)
    elif out.numel() != rows * Nc:
        raise EPError(f"out must hold {rows} x {Nc} elements")
    dt = _float_type(out, "out")
    _check("ep_expert_matmul", lib().ep_expert_matmul(
        _dev(x, torch.int8, "x", (x_rows, Kd)),
        _dev(x_scales, torch.float32, "x_scales", (x_rows,)), x_rows, _dev(w, torch.int8, "w"),
        _dev(w_scales, torch.float32, "w_scales", (E, Nc)), E, Nc, Kd,
        _dev(expert_offsets, torch.int32, "expert_offsets", (E + 1,)), layout, cap, rows,
        *_sources(row_src, expert_offsets), dt,
        _dev(out, out.dtype, "out"), _opt(status, torch.int32, "status", (1,)), _stream(stream)))
    return out

SCALE_BLOCK = 128  # columns of a row that share a scale


def scale_blocks(cols) -> int:
    """Scales of a row of `cols` columns of E4M3 codes."""
    return -(-cols // SCALE_BLOCK)


def _rows(rows, cols, dtype, device):
    """torch.empty((rows, cols)) in half of its host time."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _codes(t, name, shape=None):
    """Device pointer of E4M3 codes: uint8, or torch's own type of them."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    return _dev(t, torch.uint8, name, shape)


def _tokens(expert_offsets):
    """(pointer, E) of the offsets that say which rows hold a token."""
    if expert_offsets is None:
        return None, 0
    return _dev(expert_offsets, torch.int32, "expert_offsets"), expert_offsets.numel() - 1


def _rows2d(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise EPError(f"{name} must be a tensor of rows (two dimensions)")
    return t.shape


def ep_quantize_blocks(x, act=EP_ACT_NONE, expert_offsets=None, layout=EP_LAYOUT_CONTIG, cap=0,
                       q=None, scales=None, x_q=None, x_scales=None, stream=None):
    """x bf16 or float32 [rows, cols] (EP_ACT_SWIGLU: [rows, 2*cols]) -> (q uint8
    E4M3 codes [rows, cols], scales float32 [rows, ceil(cols / 128)]).  With x_q
    [rows, 2*cols] and x_scales (SwiGLU), the codes of x itself are written too:
    the checkpoint that ep_swiglu_backward reads.  With expert_offsets, rows that
    hold no token are skipped."""
    rows, wide = _rows2d(x, "x")
    dt = _float_type(x, "x")
    if act == EP_ACT_SWIGLU and wide % 2:
        raise EPError("x must have an even number of columns for SwiGLU")
    cols = wide // 2 if act == EP_ACT_SWIGLU else wide
    if q is None:
        q = _rows(rows, cols, torch.uint8, x.device)
    if scales is None:
        scales = _rows(rows, scale_blocks(cols), torch.float32, x.device)
    offs, E = _tokens(expert_offsets)
    _check("ep_quantize_blocks", lib().ep_quantize_blocks(
        _dev(x, x.dtype, "x"), dt, act, rows, cols, offs, E, layout, cap,
        _codes(q, "q", (rows, cols)),
        _dev(scales, torch.float32, "scales", (rows, scale_blocks(cols))),
        None if x_q is None else _codes(x_q, "x_q", (rows, wide)),
        _opt(x_scales, torch.float32, "x_scales", (rows, scale_blocks(wide))), _stream(stream)))
    return q, scales


def ep_dequantize_blocks(q, scales, expert_offsets=None, layout=EP_LAYOUT_CONTIG, cap=0, out=None,
                         out_dtype=torch.bfloat16, stream=None):
    """E4M3 codes [rows, cols] and their scales [rows, ceil(cols / 128)] -> the
    values that they stand for, bf16 or float32 [rows, cols]."""
    rows, cols = _rows2d(q, "q")
    if out is None:
        out = _rows(rows, cols, out_dtype, q.device)
    dt = _float_type(out, "out")
    offs, E = _tokens(expert_offsets)
    _check("ep_dequantize_blocks", lib().ep_dequantize_blocks(
        _codes(q, "q"), _dev(scales, torch.float32, "scales", (rows, scale_blocks(cols))), rows,
        cols, offs, E, layout, cap, dt, _dev(out, out.dtype, "out", (rows, cols)),
        _stream(stream)))
    return out


def ep_swiglu_backward(d_out, x, x_scales=None, expert_offsets=None, layout=EP_LAYOUT_CONTIG,
                       cap=0, d_x=None, stream=None):
    """Gradient of silu(g) * u to x = (g, u): d_out bf16 or float32 [rows, cols]
    -> d_x [rows, 2*cols] of its type.  x: the rows [rows, 2*cols] of the same
    type, or their E4M3 codes with x_scales [rows, ceil(2*cols / 128)]."""
    rows, cols = _rows2d(d_out, "d_out")
    dt = _float_type(d_out, "d_out")
    if d_x is None:
        d_x = _rows(rows, 2 * cols, d_out.dtype, d_out.device)
    if x_scales is None:
        px = _dev(x, d_out.dtype, "x", (rows, 2 * cols))
    else:
        px = _codes(x, "x", (rows, 2 * cols))
    offs, E = _tokens(expert_offsets)
    _check("ep_swiglu_backward", lib().ep_swiglu_backward(
        _dev(d_out, d_out.dtype, "d_out"), dt, px,
        _opt(x_scales, torch.float32, "x_scales", (rows, scale_blocks(2 * cols))), rows, cols,
        offs, E, layout, cap, _dev(d_x, d_out.dtype, "d_x", (rows, 2 * cols)), _stream(stream)))
    return d_x


def ep_expert_matmul_fp8(x, x_scales, w, w_scales, expert_offsets, layout=EP_LAYOUT_CONTIG, cap=0,
                         row_src=None, out=None, out_dtype=torch.bfloat16, status=None,
                         stream=None):
    """Every expert's rows times its weights in E4M3 codes: x [x_rows, Kd] with
    x_scales float32 [x_rows, ceil(Kd / 128)], w [E, Nc, Kd] with w_scales float32
    [E, ceil(Nc / 128), ceil(Kd / 128)] -> out bf16 or float32 [rows, Nc] ([E*cap,
    Nc] for the masked layout).  With row_src (the layout's), x holds token rows.
    Rows that hold no token are not written."""
    x_rows = _rows2d(x, "x")[0]
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise EPError("w must be a tensor [E, Nc, Kd]")
    E, Nc, Kd = w.shape
    if layout == EP_LAYOUT_MASKED:
        rows = E * cap
    else:
        rows = x_rows if row_src is None else row_src.numel()
    if out is None:
        out = _rows(rows, Nc, out_dtype, x.device)
    elif out.numel() != rows * Nc:
        raise EPError(f"out must hold {rows} x {Nc} elements")
    dt = _float_type(out, "out")
    _check("ep_expert_matmul_fp8", lib().ep_expert_matmul_fp8(
        _codes(x, "x", (x_rows, Kd)),
        _dev(x_scales, torch.float32, "x_scales", (x_rows, scale_blocks(Kd))), x_rows,
        _codes(w, "w"),
        _dev(w_scales, torch.float32, "w_scales", (E, scale_blocks(Nc), scale_blocks(Kd))), E, Nc,
        Kd, _dev(expert_offsets, torch.int32, "expert_offsets", (E + 1,)), layout, cap, rows,
        *_sources(row_src, expert_offsets), dt,
        _dev(out, out.dtype, "out"), _opt(status, torch.int32, "status", (1,)), _stream(stream)))
    return out


Norm = namedtuple("Norm", "y residual q scales rstd")


def alloc_norm(rows, cols, dtype, device, y=True, residual=False, codes=False, rstd=False) -> Norm:
    """Outputs of ep_rms_norm, None for those that are not wanted."""
    return Norm(_rows(rows, cols, dtype, device) if y else None,
                _rows(rows, cols, dtype, device) if residual else None,
                _rows(rows, cols, torch.uint8, device) if codes else None,
                _rows(rows, scale_blocks(cols), torch.float32, device) if codes else None,
                torch.empty_strided((rows,), (1,), dtype=torch.float32, device=device)
                if rstd else None)


def ep_rms_norm(x, weight, residual=None, eps=1e-6, out: Norm | None = None, stream=None) -> Norm:
    """Root-mean-square norm of x (+ residual), rows bf16 or float32 [rows, cols],
    weight bf16 or float32 [cols].  Writes the outputs that `out` holds
    (alloc_norm): y, residual (the sum, in the rows' type), q and scales (the E4M3
    codes of y), rstd float32 [rows].  Without `out`: y, rstd and, with a residual,
    the sum."""
    rows, cols = _rows2d(x, "x")
    dt, wt = _float_type(x, "x"), _float_type(weight, "weight")
    if out is None:
        out = alloc_norm(rows, cols, x.dtype, x.device, residual=residual is not None, rstd=True)
    shape = (rows, cols)
    _check("ep_rms_norm", lib().ep_rms_norm(
        _dev(x, x.dtype, "x"), dt, _opt(residual, x.dtype, "residual", shape),
        _dev(weight, weight.dtype, "weight", (cols,)), wt, rows, cols, eps,
        _opt(out.residual, x.dtype, "out.residual", shape), _opt(out.y, x.dtype, "out.y", shape),
        None if out.q is None else _codes(out.q, "out.q", shape),
        _opt(out.scales, torch.float32, "out.scales", (rows, scale_blocks(cols))),
        _opt(out.rstd, torch.float32, "out.rstd", (rows,)), _stream(stream)))
    return out


def ep_rms_norm_backward_workspace_size(rows, cols) -> int:
    return int(lib().ep_rms_norm_backward_workspace_size(rows, cols))


def ep_rms_norm_backward(d_y, z, weight, rstd, d_residual=None, d_x=None, d_weight=None,
                         weight_grad=True, workspace=None, stream=None):
    """Gradients of ep_rms_norm's y: z (its residual output, or x where it had no
    residual) and rstd are what the forward call kept.  Returns (d_x of the rows'
    type: the gradient of x and of the residual, with d_residual added; d_weight
    float32 [cols], None with weight_grad=False)."""
    rows, cols = _rows2d(z, "z")
    dt, wt = _float_type(z, "z"), _float_type(weight, "weight")
    shape = (rows, cols)
    if d_x is None:
        d_x = torch.empty_like(z)
    if not weight_grad:
        d_weight = workspace = None
    else:
        if d_weight is None:
            d_weight = _empty((cols,), torch.float32, z)
        if workspace is None:
            workspace = _empty((ep_rms_norm_backward_workspace_size(rows, cols),), torch.uint8, z)
            if stream is not None and workspace.is_cuda:
                workspace.record_stream(stream)
    _check("ep_rms_norm_backward", lib().ep_rms_norm_backward(
        _dev(d_y, z.dtype, "d_y", shape), dt, _dev(z, z.dtype, "z"),
        _dev(weight, weight.dtype, "weight", (cols,)), wt,
        _dev(rstd, torch.float32, "rstd", (rows,)), _opt(d_residual, z.dtype, "d_residual", shape),
        rows, cols, _dev(d_x, z.dtype, "d_x", shape),
        _opt(d_weight, torch.float32, "d_weight", (cols,)),
        _opt(workspace, torch.uint8, "workspace"),
        0 if workspace is None else workspace.numel(), _stream(stream)))
    return d_x, d_weight



def ep_selftest_wait_timeout(stream=None):
    """Runs the bounded-wait self-test (a grid barrier that can never complete
    gives up, sets the status word to 1 and returns).  Returns the device
    status tensor (int32 [1]); read it after synchronising."""
    dev = torch.device("cuda", torch.cuda.current_device())
    status = torch.full((1,), -1, dtype=torch.int32, device=dev)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    _check("ep_selftest_wait_timeout", lib().ep_selftest_wait_timeout(
        ctypes.c_void_p(status.data_ptr()), ctypes.c_void_p(ws.data_ptr()), ws.numel(),
        _stream(stream)))
    # keep the workspace alive until the kernel has run
    ws.record_stream(torch.cuda.current_stream(dev) if stream is None else stream)
    return status
