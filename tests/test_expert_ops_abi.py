"""Refusals of the gate, quantisation and expert product calls: host-side
checks that launch nothing (no GPU needed), and the binding's own."""
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


def gate(L, logits=p(), dt=F32, N=10, E=64, K=4, score=0, bias=None, groups=8, tg=4, gt=2,
         renorm=1, emap=None, idx=p(), w=p()):
    return L.ep_gate_topk(logits, dt, N, E, K, score, bias, groups, tg, gt, renorm, 1.0, emap, idx,
                          w, None)


def test_gate_refusals(L):
    assert gate(L, N=0) == OK
    assert gate(L, K=65) == INVALID and gate(L, K=0) == INVALID and gate(L, N=-1) == INVALID
    assert gate(L, E=1032, groups=1, tg=1) == UNSUPPORTED
    assert gate(L, E=64, K=33, groups=1, tg=1) == UNSUPPORTED
    assert gate(L, N=1 << 30, K=4) == UNSUPPORTED
    assert gate(L, dt=FP8) == INVALID and gate(L, dt=7) == INVALID
    assert gate(L, score=2) == INVALID and gate(L, score=-1) == INVALID
    assert gate(L, groups=0) == INVALID and gate(L, groups=7) == INVALID
    assert gate(L, groups=64, tg=8) == UNSUPPORTED
    assert gate(L, tg=0) == INVALID and gate(L, tg=9) == INVALID
    assert gate(L, tg=1, K=9) == INVALID  # one group holds 8 experts
    assert gate(L, gt=0) == INVALID and gate(L, gt=3) == INVALID
    assert gate(L, logits=None) == INVALID and gate(L, idx=None) == INVALID
    assert gate(L, w=None) == INVALID
    assert gate(L, logits=p(4098)) == INVALID and gate(L, logits=p(4097), dt=BF16) == INVALID
    assert gate(L, bias=p(4098)) == INVALID and gate(L, emap=p(4097)) == INVALID
    assert gate(L, idx=p(4098)) == INVALID and gate(L, w=p(4098)) == INVALID


def grad(L, g=p(), logits=p(), dt=F32, idx=p(), N=10, E=64, K=4, score=0, emap=None, d=p()):
    return L.ep_gate_topk_backward(g, logits, dt, idx, N, E, K, score, 1, 1.0, emap, d, None)


def test_gate_gradient_refusals(L):
    assert grad(L, N=0) == OK
    assert grad(L, K=65) == INVALID and grad(L, N=-2) == INVALID
    assert grad(L, E=1025) == UNSUPPORTED
    assert grad(L, dt=FP8) == INVALID and grad(L, score=5) == INVALID
    for name in ("g", "logits", "idx", "d"):
        assert grad(L, **{name: None}) == INVALID
        assert grad(L, **{name: p(4098)}) == INVALID
    assert grad(L, emap=p(4098)) == INVALID


def quant(L, x=p(), dt=BF16, act=0, rows=10, cols=64, offs=None, E=0, layout=0, cap=0, q=p(), s=p()):
    return L.ep_quantize_rows(x, dt, act, rows, cols, offs, E, layout, cap, q, s, None)


def test_quantize_refusals(L):
    assert quant(L, rows=0) == OK
    assert quant(L, rows=-1) == INVALID
    assert quant(L, cols=0) == INVALID and quant(L, cols=24) == INVALID
    assert quant(L, dt=FP8) == INVALID and quant(L, act=2) == INVALID
    assert quant(L, layout=3) == INVALID
    assert quant(L, offs=p(), E=0) == INVALID and quant(L, offs=p(), E=2000) == UNSUPPORTED
    assert quant(L, offs=p(), E=5, layout=1, cap=0) == INVALID
    assert quant(L, offs=p(), E=5, layout=1, cap=3) == INVALID  # 15 rows, not 10
    for name in ("x", "q", "s"):
        assert quant(L, **{name: None}) == INVALID
    assert quant(L, x=p(4104)) == INVALID and quant(L, q=p(4104)) == INVALID
    assert quant(L, s=p(4098)) == INVALID and quant(L, offs=p(4098), E=2) == INVALID
    assert quant(L, cols=1 << 30, act=1) == UNSUPPORTED


def mm(L, x=p(), xs=p(), x_rows=10, w=p(), ws=p(), E=4, Nc=64, Kd=128, offs=p(), layout=0, cap=0,
       rows=10, src=None, n_src=0, dt=BF16, out=p(), status=None):
    return L.ep_expert_matmul(x, xs, x_rows, w, ws, E, Nc, Kd, offs, layout, cap, rows, src, n_src,
                              dt, out, status, None)


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


def test_binding_refuses_cpu_and_mistyped_tensors(L):
    with pytest.raises(ep.EPError):
        ep.ep_gate_topk(torch.zeros(4, 16), 2)
    with pytest.raises(ep.EPError):
        ep.ep_gate_topk(torch.zeros(4, 16, dtype=torch.float16), 2)
    with pytest.raises(ep.EPError):
        ep.ep_gate_topk_backward(torch.zeros(4, 2), torch.zeros(4, 16),
                                 torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ep.EPError):
        ep.ep_quantize_rows(torch.zeros(4, 32))
    with pytest.raises(ep.EPError):
        ep.ep_quantize_rows(torch.zeros(4, 33), act=ep.EP_ACT_SWIGLU)
    z8, zf = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4)
    offs = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ep.EPError):
        ep.ep_expert_matmul(z8, zf, torch.zeros(2, 8, 32, dtype=torch.int8), torch.zeros(2, 8), offs)
    with pytest.raises(ep.EPError):
        ep.ep_expert_matmul(z8, zf, torch.zeros(2, 8, 32, dtype=torch.int8), torch.zeros(2, 8), offs,
                            out=torch.zeros(3, 8))
