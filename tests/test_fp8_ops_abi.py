"""Refusals of the FP8 layer's calls: host-side checks that launch nothing (no GPU
needed), and the binding's own."""
import ctypes

import pytest
import torch

from combine_ep_route_topk_gb300 import build as ep_build
from combine_ep_route_topk_gb300 import ep

OK, INVALID, WORKSPACE, CUDA, UNSUPPORTED = 0, 1, 2, 3, 4
P = ctypes.c_void_p
BF16, FP8, F32 = ep.EP_DTYPE_BF16, ep.EP_DTYPE_FP8_E4M3_B128, ep.EP_DTYPE_F32


@pytest.fixture(scope="module")
def L():
    ep_build.build()
    return ep.lib()


@pytest.fixture(autouse=True)
def nothing_launched(L):
    before = L.ep_kernel_launch_count()
    yield
    assert L.ep_kernel_launch_count() == before


def p(v=4096):
    return P(v)


def quant(L, x=p(), dt=BF16, act=1, rows=10, cols=64, offs=None, E=0, layout=0, cap=0, q=p(),
          s=p(), xq=None, xs=None):
    return L.ep_quantize_blocks(x, dt, act, rows, cols, offs, E, layout, cap, q, s, xq, xs, None)


def restore(L, q=p(), s=p(), rows=10, cols=64, offs=None, E=0, layout=0, cap=0, dt=BF16, out=p()):
    return L.ep_dequantize_blocks(q, s, rows, cols, offs, E, layout, cap, dt, out, None)


def swiglu(L, d=p(), dt=BF16, x=p(), xs=None, rows=10, cols=64, offs=None, E=0, layout=0, cap=0,
           dx=p()):
    return L.ep_swiglu_backward(d, dt, x, xs, rows, cols, offs, E, layout, cap, dx, None)


@pytest.mark.parametrize("f", [quant, restore, swiglu])
def test_rows_and_tokens(L, f):
    assert f(L, rows=0) == OK
    assert f(L, rows=-1) == INVALID and f(L, cols=0) == INVALID and f(L, cols=24) == INVALID
    assert f(L, dt=FP8) == INVALID and f(L, dt=9) == INVALID
    assert f(L, layout=2) == INVALID and f(L, layout=-1) == INVALID
    assert f(L, offs=p(), E=0) == INVALID and f(L, offs=p(), E=1025) == UNSUPPORTED
    assert f(L, offs=p(), E=5, layout=1, cap=0) == INVALID
    assert f(L, offs=p(), E=5, layout=1, cap=3) == INVALID  # 15 rows, not 10
    assert f(L, offs=p(4098), E=2) == INVALID
    assert f(L, cols=(1 << 31) - 16) == UNSUPPORTED
    assert f(L, rows=(1 << 31) - 1, cols=272) == UNSUPPORTED


def test_quantize_blocks_refusals(L):
    assert quant(L, act=2) == INVALID and quant(L, act=-1) == INVALID
    for name in ("x", "q", "s"):
        assert quant(L, **{name: None}) == INVALID
    assert quant(L, x=p(4104)) == INVALID and quant(L, q=p(4104)) == INVALID
    assert quant(L, s=p(4098)) == INVALID
    # the checkpoint: codes and scales, of SwiGLU's rows
    assert quant(L, xq=p()) == INVALID and quant(L, xs=p()) == INVALID
    assert quant(L, act=0, xq=p(), xs=p()) == INVALID
    assert quant(L, xq=p(4104), xs=p()) == INVALID and quant(L, xq=p(), xs=p(4098)) == INVALID
    assert quant(L, rows=0, xq=p(), xs=p()) == OK


def test_dequantize_blocks_refusals(L):
    for name in ("q", "s", "out"):
        assert restore(L, **{name: None}) == INVALID
    assert restore(L, q=p(4104)) == INVALID and restore(L, out=p(4104)) == INVALID
    assert restore(L, s=p(4098)) == INVALID


def test_swiglu_backward_refusals(L):
    for name in ("d", "x", "dx"):
        assert swiglu(L, **{name: None}) == INVALID
        assert swiglu(L, **{name: p(4104)}) == INVALID
    assert swiglu(L, xs=p(4098)) == INVALID


def mm(L, x=p(), xs=p(), x_rows=10, w=p(), ws=p(), E=4, Nc=64, Kd=128, offs=p(), layout=0, cap=0,
       rows=10, src=None, n_src=0, dt=BF16, out=p(), status=None):
    return L.ep_expert_matmul_fp8(x, xs, x_rows, w, ws, E, Nc, Kd, offs, layout, cap, rows, src,
                                  n_src, dt, out, status, None)


def test_matmul_refusals(L):
    assert mm(L, rows=0, x_rows=0) == OK
    assert mm(L, E=0) == INVALID and mm(L, Nc=0) == INVALID and mm(L, rows=-1) == INVALID
    assert mm(L, Kd=0) == INVALID and mm(L, Kd=120) == INVALID
    assert mm(L, E=1025) == UNSUPPORTED and mm(L, Kd=65552) == UNSUPPORTED
    assert mm(L, E=1024, Nc=1 << 21) == UNSUPPORTED
    assert mm(L, layout=2) == INVALID and mm(L, dt=FP8) == INVALID
    assert mm(L, layout=1, cap=0) == INVALID and mm(L, layout=1, cap=3) == INVALID
    assert mm(L, x_rows=9) == INVALID  # without row_src, x rows are the output's
    assert mm(L, src=p(), n_src=-1) == INVALID
    for name in ("x", "xs", "w", "ws", "offs", "out"):
        assert mm(L, **{name: None}) == INVALID
    for name in ("x", "w", "out"):
        assert mm(L, **{name: p(4104)}) == INVALID
    for name in ("xs", "ws", "offs", "src", "status"):
        assert mm(L, **{name: p(4098)}) == INVALID


def norm(L, x=p(), dt=BF16, res=None, w=p(), wdt=F32, rows=10, cols=64, eps=1e-6, ro=None, y=p(),
         q=None, s=None, r=None):
    return L.ep_rms_norm(x, dt, res, w, wdt, rows, cols, eps, ro, y, q, s, r, None)


def norm_grad(L, dy=p(), dt=BF16, z=p(), w=p(), wdt=F32, r=p(), dres=None, rows=10, cols=64,
              dx=p(), dw=p(), ws=p(), n=1 << 30):
    return L.ep_rms_norm_backward(dy, dt, z, w, wdt, r, dres, rows, cols, dx, dw, ws, n, None)


@pytest.mark.parametrize("f", [norm, norm_grad])
def test_norm_sizes(L, f):
    assert f(L, rows=-1) == INVALID and f(L, cols=0) == INVALID and f(L, cols=40) == INVALID
    assert f(L, cols=16400) == UNSUPPORTED
    assert f(L, dt=FP8) == INVALID and f(L, wdt=FP8) == INVALID and f(L, wdt=-1) == INVALID
    assert f(L, w=None) == INVALID and f(L, w=p(4104)) == INVALID


def test_norm_refusals(L):
    assert norm(L, rows=0) == OK
    for eps in (0.0, -1e-6, float("inf"), float("nan")):
        assert norm(L, eps=eps) == INVALID
    assert norm(L, x=None) == INVALID
    assert norm(L, y=None) == INVALID  # nothing to write
    assert norm(L, q=p()) == INVALID and norm(L, s=p()) == INVALID
    for name in ("x", "res", "ro", "y"):
        assert norm(L, **{name: p(4104)}) == INVALID
    assert norm(L, q=p(4104), s=p()) == INVALID and norm(L, q=p(), s=p(4098)) == INVALID
    assert norm(L, r=p(4098)) == INVALID


def test_norm_gradient_refusals(L):
    for name in ("dy", "z", "r", "dx"):
        assert norm_grad(L, **{name: None}) == INVALID
    for name in ("dy", "z", "dres", "dx", "ws"):
        assert norm_grad(L, **{name: p(4104)}) == INVALID
    assert norm_grad(L, r=p(4098)) == INVALID and norm_grad(L, dw=p(4098)) == INVALID
    need = L.ep_rms_norm_backward_workspace_size(10, 64)
    assert need % 256 == 0 and need >= 64 * 4
    assert norm_grad(L, ws=None, n=0) == WORKSPACE and norm_grad(L, n=need - 1) == WORKSPACE
    assert norm_grad(L, rows=0, dw=None, ws=None, n=0) == OK


def test_binding_refuses_cpu_and_mistyped_tensors(L):
    z, zf = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1)
    offs = torch.zeros(3, dtype=torch.int32)
    calls = [
        lambda: ep.ep_quantize_blocks(torch.zeros(4, 32)),
        lambda: ep.ep_quantize_blocks(torch.zeros(4, 32, dtype=torch.float16)),
        lambda: ep.ep_quantize_blocks(torch.zeros(2, 4, 32)),
        lambda: ep.ep_quantize_blocks(torch.zeros(4, 33), act=ep.EP_ACT_SWIGLU),
        lambda: ep.ep_dequantize_blocks(z, zf),
        lambda: ep.ep_dequantize_blocks(z, zf, out_dtype=torch.float16),
        lambda: ep.ep_swiglu_backward(torch.zeros(4, 16), torch.zeros(4, 32)),
        lambda: ep.ep_expert_matmul_fp8(z, zf, torch.zeros(2, 8, 32, dtype=torch.uint8),
                                        torch.zeros(2, 1, 1), offs),
        lambda: ep.ep_expert_matmul_fp8(z, zf, z, zf, offs),
        lambda: ep.ep_rms_norm(torch.zeros(4, 32), torch.zeros(32)),
        lambda: ep.ep_rms_norm(torch.zeros(4, 32), torch.zeros(32, dtype=torch.float16)),
        lambda: ep.ep_rms_norm_backward(torch.zeros(4, 32), torch.zeros(4, 32), torch.zeros(32),
                                        torch.zeros(4)),
    ]
    for call in calls:
        with pytest.raises(ep.EPError):
            call()
