"""The FP8 layer passes on whether its products completed: each product writes its own
status word in the buffers, and check() raises where one gave up.  The give-up is a
fake's, on the host."""
import pytest
import torch

import combine_ep_route_topk_gb300 as ep
from combine_ep_route_topk_gb300 import pipeline as pl

N, E, K, H, INNER = 12, 4, 2, 128, 32


@pytest.mark.parametrize("gave_up", [None, 0, 1])
@pytest.mark.parametrize("cap", [0, 8])
def test_a_product_that_gave_up_is_seen(monkeypatch, gave_up, cap):
    calls = []

    def product(*args, status=None, **kw):
        assert status is not None and status.dtype == torch.int32 and status.shape == (1,)
        status[0] = int(len(calls) == gave_up)
        calls.append(status)

    monkeypatch.setattr(pl._ep, "ep_expert_matmul_fp8", product)
    for name in ("ep_gate_topk", "ep_dispatch_layout", "ep_dispatch"):
        monkeypatch.setattr(pl._ep, name, lambda *a, **k: None)
    monkeypatch.setattr(pl._ep, "ep_quantize_blocks", lambda *a, q=None, scales=None, **k: (q, scales))
    monkeypatch.setattr(pl._ep, "ep_combine", lambda *a, out=None, **k: out)
    monkeypatch.setattr(pl._ep, "ep_dispatch_layout_workspace_size", lambda *a: 256)
    buf = pl.make_layer_buffers_fp8(N, E, K, H, INNER, 1, cap, device="cpu")
    w = pl.ExpertWeightsFP8(*(torch.zeros(1) for _ in range(4)))
    out = pl.expert_layer_fp8(torch.zeros(N, H), torch.zeros(N, E), torch.tensor([0, N]), w, buf)
    assert out is buf.comb and len(calls) == 2
    assert calls[0].data_ptr() != calls[1].data_ptr()
    if gave_up is None:
        buf.check()
    else:
        with pytest.raises(ep.EPError, match=("first", "second")[gave_up]):
            buf.check()


@pytest.mark.parametrize("gave_up", [0, 1])
def test_a_gradient_that_gave_up_is_seen(monkeypatch, gave_up):
    calls = []

    def product(*args, status=None, **kw):
        status[0] = int(len(calls) == gave_up)
        calls.append(status)

    monkeypatch.setattr(pl._ep, "ep_expert_matmul_fp8", product)
    monkeypatch.setattr(pl._ep, "ep_quantize_blocks", lambda *a, q=None, scales=None, **k: (q, scales))
    monkeypatch.setattr(pl._ep, "ep_swiglu_backward", lambda *a, **k: None)
    buf = pl.make_mlp_buffers_fp8(5, H, INNER, keep=True, device="cpu")
    w = pl.ExpertWeightsFP8(*(torch.zeros(1) for _ in range(8)))
    pl.expert_mlp_fp8_backward(torch.zeros(5, H), torch.tensor([0, 5]), w, buf)
    assert len(calls) == 2
    with pytest.raises(ep.EPError, match=("second's", "first's")[gave_up] + " gradient"):
        buf.check()
