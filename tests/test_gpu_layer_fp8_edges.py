"""The FP8 layer's calls at the edges of their sizes, on the GPU: no rows, no tokens."""
import pytest
import torch

import combine_ep_route_topk_gb300 as ep
from combine_ep_route_topk_gb300 import pipeline as pl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def weights(E, H, inner, seed=1):
    g = torch.Generator().manual_seed(seed)
    up = (torch.randn((E, 2 * inner, H), generator=g) * H ** -0.5).to(BF).cuda()
    down = (torch.randn((E, H, inner), generator=g) * inner ** -0.5).to(BF).cuda()
    return pl.quantize_expert_weights_fp8(up, down, gradients=True)


def test_experts_that_got_no_rows():
    """A rank that received no tokens runs its step all the same."""
    E, H, inner = 3, 272, 80
    w = weights(E, H, inner)
    buf = pl.make_mlp_buffers_fp8(0, H, inner, keep=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    q, s = ep.ep_quantize_blocks(torch.zeros((0, H), dtype=BF, device="cuda"))
    assert pl.expert_mlp_fp8(q, s, offsets, w, buf).shape == (0, H)
    d = torch.zeros((0, H), dtype=BF, device="cuda")
    assert pl.expert_mlp_fp8_backward(d, offsets, w, buf).shape == (0, H)
    buf.check()


@pytest.mark.parametrize("cap", [0, 4])
@pytest.mark.parametrize("coded", [False, True])
def test_layer_without_tokens(cap, coded):
    E, K, H, inner = 4, 2, 256, 128
    w = weights(E, H, inner)
    buf = pl.make_layer_buffers_fp8(0, E, K, H, inner, 1, cap, keep=True)
    x = torch.zeros((0, H), dtype=BF, device="cuda")
    if coded:
        x = ep.ep_quantize_blocks(x)
    ro = torch.zeros(2, dtype=torch.int32, device="cuda")
    logits = torch.zeros((0, E), device="cuda")
    assert pl.expert_layer_fp8(x, logits, ro, w, buf).shape == (0, H)
    d = torch.zeros_like(buf.mlp.down)
    pl.expert_mlp_fp8_backward(d, buf.lay.expert_offsets, w, buf.mlp)
    buf.check()


@pytest.mark.parametrize("product", ["fp8", "int8"])
def test_an_empty_row_src_reads_nothing(product):
    """Not even where x has as many rows as the output."""
    E, cap, Nc, Kd = 2, 3, 48, 64
    g = torch.Generator().manual_seed(2)
    x = torch.randint(1, 9, (E * cap, Kd), generator=g)
    w = torch.randint(1, 9, (E, Nc, Kd), generator=g)
    offs = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    src = torch.empty((0,), dtype=torch.int32, device="cuda")
    kw = dict(layout=ep.EP_LAYOUT_MASKED, cap=cap, row_src=src)
    out = torch.full((E * cap, Nc), -7.0, device="cuda")
    if product == "fp8":
        x, w = (t.float().to(torch.float8_e4m3fn).cuda() for t in (x, w))
        ep.ep_expert_matmul_fp8(x, torch.ones((E * cap, 1), device="cuda"), w,
                                torch.ones((E, 1, 1), device="cuda"), offs, out=out, **kw)
    else:
        x, w = (t.to(torch.int8).cuda() for t in (x, w))
        ep.ep_expert_matmul(x, torch.ones(E * cap, device="cuda"), w,
                            torch.ones((E, Nc), device="cuda"), offs, out=out, **kw)
    held = torch.tensor([True, True, False] * E)
    assert (out.cpu()[held] == 0).all() and (out.cpu()[~held] == -7.0).all()


@pytest.mark.parametrize("cap", [0, 4])
def test_integer_layer_without_tokens(cap):
    E, K, H, inner = 4, 2, 256, 128
    up = torch.ones((E, 2 * inner, H), dtype=BF, device="cuda")
    w = pl.quantize_expert_weights(up, torch.ones((E, H, inner), dtype=BF, device="cuda"))
    buf = pl.make_layer_buffers(0, E, K, H, inner, 1, cap)
    ro = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros((0, H), dtype=BF, device="cuda")
    assert pl.expert_layer(x, torch.zeros((0, E), device="cuda"), ro, w, buf).shape == (0, H)
    buf.check()
