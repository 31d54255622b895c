"""Sizes that the FP8 layer's calls meet at their edges, on the host: a rank whose experts
got no rows, and codes that do not hold the call's tokens.  The kernels' calls are fakes
that record what they are given."""
import pytest
import torch

import combine_ep_route_topk_gb300 as ep
from combine_ep_route_topk_gb300 import pipeline as pl

E, K, H, INNER = 4, 2, 256, 160


@pytest.fixture
def calls(monkeypatch):
    """Fakes of the kernels' calls: each records its name and its outputs."""
    seen = []

    def product(x, x_scales, w, w_scales, offsets, out=None, **kw):
        seen.append(("product", tuple(x.shape), tuple(x_scales.shape), tuple(out.shape)))
        return out

    def quantize(x, q=None, scales=None, **kw):
        assert q.shape == x.shape or q.shape[1] * 2 == x.shape[1]
        assert scales.shape == (q.shape[0], ep.scale_blocks(q.shape[1]))
        seen.append(("codes", tuple(q.shape), tuple(scales.shape)))
        return q, scales

    def gradient(d, x, x_scales, d_x=None, **kw):
        seen.append(("gradient", tuple(d.shape), tuple(x.shape), tuple(d_x.shape)))
        return d_x

    monkeypatch.setattr(pl._ep, "ep_expert_matmul_fp8", product)
    monkeypatch.setattr(pl._ep, "ep_quantize_blocks", quantize)
    monkeypatch.setattr(pl._ep, "ep_swiglu_backward", gradient)
    for name in ("ep_gate_topk", "ep_dispatch_layout", "ep_dispatch"):
        monkeypatch.setattr(pl._ep, name, lambda *a, _n=name, **k: seen.append((_n,)))
    monkeypatch.setattr(pl._ep, "ep_combine", lambda *a, out=None, **k: out)
    monkeypatch.setattr(pl._ep, "ep_dispatch_layout_workspace_size", lambda *a: 256)
    return seen


WEIGHTS = pl.ExpertWeightsFP8(*(torch.zeros(1) for _ in range(8)))


@pytest.mark.parametrize("rows", [0, 3])
def test_experts_forward_and_backward_of_any_number_of_rows(calls, rows):
    buf = pl.make_mlp_buffers_fp8(rows, H, INNER, keep=True, device="cpu")
    offsets = torch.full((E + 1,), rows, dtype=torch.int32)
    offsets[0] = 0
    x, xs = torch.zeros((rows, H), dtype=torch.uint8), torch.zeros((rows, 2))
    assert pl.expert_mlp_fp8(x, xs, offsets, WEIGHTS, buf) is buf.down
    assert pl.expert_mlp_fp8_backward(torch.zeros((rows, H)), offsets, WEIGHTS, buf) is buf.d_rows
    assert calls[3:] == [
        ("codes", (rows, H), (rows, 2)), ("product", (rows, H), (rows, 2), (rows, INNER)),
        ("gradient", (rows, INNER), (rows, 2 * INNER), (rows, 2 * INNER)),
        ("codes", (rows, 2 * INNER), (rows, 3)),
        ("product", (rows, 2 * INNER), (rows, 3), (rows, H))]


@pytest.mark.parametrize("cap", [0, 8])
def test_layer_refuses_codes_of_fewer_rows_than_tokens(calls, cap):
    """A token without its row would count as zeros; rows behind the last token are none's."""
    N = 5
    buf = pl.make_layer_buffers_fp8(N, E, K, H, INNER, 1, cap, device="cpu")
    logits, ro = torch.zeros((N, E)), torch.tensor([0, N])

    def layer(rows):
        x = torch.zeros((rows, H), dtype=torch.uint8), torch.zeros((rows, 2))
        return pl.expert_layer_fp8(x, logits, ro, WEIGHTS, buf)
    for rows in (0, N - 1):
        with pytest.raises(ep.EPError, match=f"{rows} rows of codes for {N} tokens"):
            layer(rows)
    assert calls == []  # refused before anything is launched
    for rows in (N, N + 3):
        assert layer(rows) is buf.comb
