"""pipeline.expert_layer passes on whether its products completed: each product
writes its own status word in the buffers, and LayerBuffers.check() raises where
one gave up.  The give-up is a fake's, on the host."""
import pytest
import torch

import combine_ep_route_topk_gb300 as ep
from combine_ep_route_topk_gb300 import pipeline as pl

N, E, K, H, INNER = 12, 4, 2, 64, 32


@pytest.mark.parametrize("gave_up", [None, 0, 1])
@pytest.mark.parametrize("cap", [0, 8])
def test_a_product_that_gave_up_is_seen(monkeypatch, gave_up, cap):
    calls = []

    def product(*args, status=None, **kw):
        assert status is not None and status.dtype == torch.int32 and status.shape == (1,)
        status[0] = int(len(calls) == gave_up)
        calls.append(status)

    monkeypatch.setattr(pl._ep, "ep_expert_matmul", product)
    for name in ("ep_gate_topk", "ep_dispatch_layout", "ep_quantize_rows"):
        monkeypatch.setattr(pl._ep, name, lambda *a, **k: None)
    monkeypatch.setattr(pl._ep, "ep_combine", lambda *a, out=None, **k: out)
    monkeypatch.setattr(pl._ep, "ep_dispatch_layout_workspace_size", lambda *a: 256)
    buf = pl.make_layer_buffers(N, E, K, H, INNER, 1, cap, device="cpu")
    w = pl.ExpertWeights(*(torch.zeros(1) for _ in range(4)))
    out = pl.expert_layer(torch.zeros(N, H), torch.zeros(N, E), torch.tensor([0, N]), w, buf)
    assert out is buf.comb and len(calls) == 2
    assert calls[0].data_ptr() != calls[1].data_ptr()  # the second call does not clear the first's
    if gave_up is None:
        buf.check()
    else:
        with pytest.raises(ep.EPError, match=("first", "second")[gave_up]):
            buf.check()


@pytest.mark.gpu
def test_products_that_complete_clear_the_status():
    g = torch.Generator().manual_seed(1)
    w = pl.quantize_expert_weights(torch.randn((E, 2 * INNER, H), generator=g).cuda(),
                                   torch.randn((E, H, INNER), generator=g).cuda())
    buf = pl.make_layer_buffers(N, E, K, H, INNER, 1)
    buf.up_status.fill_(7)
    buf.down_status.fill_(7)
    pl.expert_layer(torch.randn((N, H), generator=g).to(torch.bfloat16).cuda(),
                    torch.randn((N, E), generator=g).cuda(),
                    torch.tensor([0, N], dtype=torch.int32, device="cuda"), w, buf)
    buf.check()
    assert int(buf.up_status) == 0 and int(buf.down_status) == 0
