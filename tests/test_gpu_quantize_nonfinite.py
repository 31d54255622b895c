"""A NaN or an infinity in a row that is quantised stays visible: the row's scale
is not finite (so neither is any product of the row), its codes are 0, and no
other row changes."""
import pytest
import torch

import combine_ep_route_topk_gb300 as ep
from combine_ep_route_topk_gb300 import pipeline as pl

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_SWIGLU])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(40, 16), (40, 256), (40, 512), (4100, 1024), (4100, 1536), (40, 1040),
                                       (40, 2048), (4100, 4096), (40, 4096), (40, 8192), (40, 16384), (40, 20000)])
def test_nonfinite_rows(rows, cols, dtype, act):
    wide = 2 * cols if act == ep.EP_ACT_SWIGLU else cols
    x = torch.randn((rows, wide), generator=torch.Generator().manual_seed(cols)).to(dtype)
    bad = {3: (0, NAN), 7: (wide - 1, NAN), 9: (wide // 2, -NAN), 11: (cols - 1, INF), 20: (5, -INF), 39: (8, INF)}
    y = x.clone()
    for r, (c, v) in bad.items():
        y[r, c] = v
    y[30], x[30] = NAN, 0.0
    q0, s0 = (t.cpu() for t in ep.ep_quantize_rows(x.cuda(), act=act))
    q, s = (t.cpu() for t in ep.ep_quantize_rows(y.cuda(), act=act))
    hit = torch.zeros(rows, dtype=torch.bool)
    hit[list(bad) + [30]] = True
    if act == ep.EP_ACT_SWIGLU:
        hit[20] = hit[20] and not torch.isfinite(torch.nn.functional.silu(y[20, 5].double()) * y[20, 5 + cols].double())
    assert not torch.isfinite(s[hit]).any(), s[hit]
    assert s[30].isnan() and s[3].isnan() and s[7].isnan() and s[9].isnan()
    assert (q[hit] == 0).all()
    assert torch.equal(q[~hit], q0[~hit]) and torch.equal(s[~hit], s0[~hit])


@pytest.mark.parametrize("cap", [0, 64])
@pytest.mark.parametrize("N", [3, 50])
def test_a_layer_passes_nan_on(N, cap):
    E, K, H, inner = 4, 2, 128, 64
    g = torch.Generator().manual_seed(N)
    x = torch.randn((N, H), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((N, E), generator=g).cuda()
    up = torch.randn((E, 2 * inner, H), generator=g).cuda()
    down = torch.randn((E, H, inner), generator=g).cuda()
    w = pl.quantize_expert_weights(up, down)
    buf = pl.make_layer_buffers(N, E, K, H, inner, 1, cap)
    ro = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    want = pl.expert_layer(x, logits, ro, w, buf).clone()
    assert torch.isfinite(want).all()
    x[1, 17] = NAN
    got = pl.expert_layer(x, logits, ro, w, buf)
    assert got[1].isnan().all()
    rest = torch.arange(N, device="cuda") != 1
    assert torch.equal(got[rest], want[rest])
