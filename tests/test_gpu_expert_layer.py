"""pipeline.expert_layer: gate, layout, quantised tokens, the experts' two 8-bit
products, SwiGLU and combine together, against the layer in 64 bits.

Quantisation is part of the layer, so the 64-bit layer uses the same codes: the
tokens' and the inner rows' as the GPU wrote them (their own tests check them),
and the rows of the first product as bf16, as the layer stores them.  Bounds:
each product within its float32 scaling and sum (the sums' terms are at most
Kd / 16 + 4 roundings of 2^-23 on the magnitudes) and half a bf16 unit; the
combine within K FMAs and half a unit."""
import numpy as np
import pytest
import torch

import _expert_ref as ref
import combine_ep_route_topk_gb300 as ep
from combine_ep_route_topk_gb300 import pipeline as pl

pytestmark = pytest.mark.gpu


def make(N, E, K, H, inner, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, H), generator=g).to(torch.bfloat16)
    logits = torch.randn((N, E), generator=g)
    up = (torch.randn((E, 2 * inner, H), generator=g) * H ** -0.5).to(torch.bfloat16)
    down = (torch.randn((E, H, inner), generator=g) * inner ** -0.5).to(torch.bfloat16)
    return x.cuda(), logits.cuda(), up.cuda(), down.cuda()


def check(x, logits, w, buf, K):
    E, two, H = w.up.shape
    inner = two // 2
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    offs = buf.lay.expert_offsets.cpu().numpy()
    src = buf.lay.row_src.cpu().numpy()
    masked = buf.layout == ep.EP_LAYOUT_MASKED
    rows = buf.up.shape[0]
    i8 = lambda t: t.cpu().numpy()  # noqa: E731
    want, mag, written = ref.matmul(i8(buf.xq), n(buf.xs), i8(w.up), n(w.up_scales), offs,
                                    int(masked), buf.cap, src, rows)
    got = n(buf.up)
    tol = (H / 16 + 4) * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= tol)[written].all()
    v = ref.swiglu(got[written])
    q, scale = ref.quantize(v)
    assert np.abs(n(buf.hq)[written] - q).max() <= 0.5 + 2e-4
    np.testing.assert_allclose(n(buf.hs)[written], scale, rtol=1e-6)
    want, mag, _ = ref.matmul(i8(buf.hq), n(buf.hs), i8(w.down), n(w.down_scales), offs,
                              int(masked), buf.cap, None, rows)
    got = n(buf.down)
    tol = (inner / 16 + 4) * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= tol)[written].all()
    # combine of the stored rows
    idx, wt, pos = buf.idx.cpu().numpy(), n(buf.wt), buf.lay.pos.cpu().numpy()
    out = n(buf.comb)
    for t in range(x.shape[0]):
        acc, m = np.zeros(H), np.zeros(H)
        for k in range(K):
            e, p = idx[t, k], pos[t, k]
            if e < 0:
                continue
            r = p
            if masked:
                if p - offs[e] >= buf.cap:
                    continue
                r = e * buf.cap + p - offs[e]
            acc += wt[t, k] * got[r]
            m += np.abs(wt[t, k] * got[r])
        assert (np.abs(out[t] - acc) <= 2 * K * 2.0 ** -24 * m + 2.0 ** -8 * np.abs(acc) + 1e-30).all()


@pytest.mark.parametrize("N,E,K,H,inner,cap,groups", [
    (1, 16, 2, 128, 64, 0, 1),        # one token
    (24, 16, 2, 128, 64, 8, 4),       # masked, some experts past their capacity
    (70, 8, 3, 272, 80, 0, 2),        # ragged, odd multiples of 16
    (300, 4, 2, 256, 144, 200, 1),    # many rows an expert
])
def test_layer_against_64_bits(N, E, K, H, inner, cap, groups):
    x, logits, up, down = make(N, E, K, H, inner, N)
    w = pl.quantize_expert_weights(up, down)
    R = 2
    ro = torch.tensor([0, N // 3, N], dtype=torch.int32, device="cuda")
    buf = pl.make_layer_buffers(N, E, K, H, inner, R, cap)
    bias = torch.linspace(-0.1, 0.1, E, device="cuda")
    pl.expert_layer(x, logits, ro, w, buf, bias=bias, groups=groups,
                    topk_groups=max(1, groups // 2), scale=2.5)
    check(x, logits, w, buf, K)


def test_layer_is_near_the_unquantised_one():
    """8-bit codes against bf16 weights and rows in float64: a code is off by up
    to 1/254 of its row's largest value, 1 / sqrt(12) / 127 of it on average, so
    four roundings of rows whose largest value is about 4 sigma leave a relative
    error near 2 * 4 / sqrt(12) / 127 = 0.018; 0.05 is allowed."""
    N, E, K, H, inner = 64, 8, 2, 512, 256
    x, logits, up, down = make(N, E, K, H, inner, 3)
    buf = pl.make_layer_buffers(N, E, K, H, inner, 1)
    ro = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    out = pl.expert_layer(x, logits, ro, pl.quantize_expert_weights(up, down), buf).double()
    want = torch.zeros_like(out)
    for t in range(N):
        for k in range(K):
            e = int(buf.idx[t, k])
            h = up[e].double() @ x[t].double()
            h = torch.nn.functional.silu(h[:inner]) * h[inner:]
            want[t] += float(buf.wt[t, k]) * (down[e].double() @ h)
    assert float((out - want).norm() / want.norm()) < 0.05


def test_layer_masked_experts_maps_and_no_picks():
    """A failed rank's experts (-inf), rows with no expert left, renumbering."""
    N, E, K, H, inner = 40, 8, 2, 128, 64
    x, logits, up, down = make(N, E, K, H, inner, 5)
    logits[:, 2:4] = -float("inf")
    logits[7] = -float("inf")
    emap = torch.randperm(E, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    w = pl.quantize_expert_weights(up, down)
    buf = pl.make_layer_buffers(N, E, K, H, inner, 1)
    ro = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    pl.expert_layer(x, logits, ro, w, buf, expert_map=emap)
    assert (buf.comb[7] == 0).all()
    off = buf.lay.expert_offsets.cpu()
    for e in (2, 3):
        m = int(emap[e])
        assert off[m] == off[m + 1]
    check(x, logits, w, buf, K)


def test_layer_in_a_graph():
    N, E, K, H, inner, cap = 32, 16, 4, 256, 128, 16
    x, logits, up, down = make(N, E, K, H, inner, 11)
    w = pl.quantize_expert_weights(up, down)
    buf = pl.make_layer_buffers(N, E, K, H, inner, 4, cap)
    ro = torch.tensor([0, 8, 16, 24, N], dtype=torch.int32, device="cuda")
    pl.expert_layer(x, logits, ro, w, buf)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pl.expert_layer(x, logits, ro, w, buf)
    x2, logits2, _, _ = make(N, E, K, H, inner, 12)
    x.copy_(x2)
    logits.copy_(logits2)
    g.replay()
    torch.cuda.synchronize()
    got = buf.comb.clone()
    pl.expert_layer(x, logits, ro, w, buf)
    assert torch.equal(got, buf.comb)
    check(x, logits, w, buf, K)


def test_weight_quantisation_refuses_mismatched_shapes():
    with pytest.raises(ValueError):
        pl.quantize_expert_weights(torch.zeros((2, 64, 32), device="cuda"),
                                   torch.zeros((2, 32, 16), device="cuda"))
