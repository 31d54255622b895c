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
