"""Gradient of the gate's weights where expert_map drops experts or sends several
to one id: the weights are taken over the picks before the map, so the gradient
needs those (ep_gate_topk's `picks`).  Tolerance: the gradient's roundings,
counted in test_gpu_gate.py (3e-5 of scale * max|g|)."""
import ctypes

import numpy as np
import pytest
import torch

import _expert_ref as ref
import combine_ep_route_topk_gb300 as ep
from combine_ep_route_topk_gb300 import build as ep_build

SIG, SOFT = ep.EP_SCORE_SIGMOID, ep.EP_SCORE_SOFTMAX
GRAD_TOL = 3e-5


def maps(E):
    """Name -> map: experts dropped, several at one id, both."""
    keep = torch.arange(E, dtype=torch.int32)
    dropped, joined = keep.clone(), keep // 2
    dropped[::3] = -1
    dropped[1] = E + 5
    both = joined.clone()
    both[1::4] = -7
    return {"dropped": dropped, "joined": joined, "both": both}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["dropped", "joined", "both"])
@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("N,E,K", [(60, 40, 5), (4099, 16, 8), (33, 96, 12)])
def test_gradient_through_a_map_that_is_not_one_to_one(N, E, K, renorm, score, kind):
    scale, h = 2.5, 1e-5
    g = torch.Generator().manual_seed(N + E)
    logits = torch.randn((N, E), generator=g) * 1.5
    logits[torch.rand((N, E), generator=g) < 0.1] = -float("inf")
    d_w = torch.randn((N, K), generator=g)
    emap = maps(E)[kind]
    plain, w0 = ep.ep_gate_topk(logits.cuda(), K, score, renorm=renorm, scale=scale)
    picks = torch.full((N, K), -9, dtype=torch.int32, device="cuda")
    idx, w = ep.ep_gate_topk(logits.cuda(), K, score, renorm=renorm, scale=scale,
                             expert_map=emap.cuda(), picks=picks)
    assert torch.equal(picks, plain) and torch.equal(w, w0)
    mapped = torch.where(plain.cpu() >= 0, emap[plain.cpu().clamp(min=0).long()], -1)
    assert torch.equal(idx.cpu(), torch.where((mapped >= 0) & (mapped < E), mapped, -1))
    got = ep.ep_gate_topk_backward(d_w.cuda(), logits.cuda(), picks, score, renorm=renorm,
                                   scale=scale).double().cpu().numpy()
    ids, G, L = picks.cpu().numpy(), d_w.double().numpy(), logits.double().numpy()
    for t in range(N):
        tol = GRAD_TOL * scale * np.abs(G[t]).max()
        want = ref.gate_grad_row(L[t], ids[t], G[t], score == SOFT, renorm, scale)
        assert np.abs(got[t] - want).max() <= tol, t
        if t < 4:  # and the forward's own weights, by central differences in 64 bits
            for e in range(E):
                if not np.isfinite(L[t, e]):
                    continue
                up, dn = L[t].copy(), L[t].copy()
                up[e] += h
                dn[e] -= h
                diff = sum(G[t] * (ref.weights_of(up, ids[t], score == SOFT, renorm, scale) -
                                   ref.weights_of(dn, ids[t], score == SOFT, renorm, scale))) / (2 * h)
                assert abs(got[t, e] - diff) <= tol + 1e-8


@pytest.mark.gpu
def test_a_dropped_pick_by_hand():
    """Two picks of equal logits, the second dropped by the map: w_0 = 1 / (1 +
    exp(l_1 - l_0)) has the gradient (1/4, -1/4)."""
    logits = torch.tensor([[1.0, 1.0, -3.0, -3.0]], device="cuda")
    emap = torch.tensor([0, -1, 2, 3], dtype=torch.int32, device="cuda")
    picks = torch.empty((1, 2), dtype=torch.int32, device="cuda")
    idx, w = ep.ep_gate_topk(logits, 2, SOFT, expert_map=emap, picks=picks)
    assert idx.tolist() == [[0, -1]] and w.tolist() == [[0.5, 0.5]] and picks.tolist() == [[0, 1]]
    d = ep.ep_gate_topk_backward(torch.tensor([[1.0, 0.0]], device="cuda"), logits, picks, SOFT)
    assert d.tolist() == [[0.25, -0.25, 0.0, 0.0]]


def test_refusals_of_the_picks_output():
    ep_build.build()
    L = ep.ep.lib()
    p = ctypes.c_void_p(4096)
    before = L.ep_kernel_launch_count()

    def call(N=10, K=4, idx=p, picks=p):
        return L.ep_gate_topk_picks(p, ep.EP_DTYPE_F32, N, 64, K, 0, None, 1, 1, 1, 1, 1.0, None, idx, p,
                                    picks, None)
    assert call(picks=ctypes.c_void_p(4098)) == 1
    assert call(idx=None) == 1 and call(K=65) == 1
    assert call(N=0) == 0 and call(N=0, picks=None) == 0
    assert L.ep_kernel_launch_count() == before
    with pytest.raises(ep.EPError):
        ep.ep_gate_topk(torch.zeros(4, 16), 2, picks=torch.zeros((4, 2), dtype=torch.int32))


@pytest.mark.gpu
def test_a_layer_keeps_its_picks():
    """pipeline.expert_layer under a map that drops experts: buf.picks gives the
    gradient that buf.idx cannot."""
    from combine_ep_route_topk_gb300 import pipeline as pl
    N, E, K, H, inner = 40, 8, 3, 64, 32
    g = torch.Generator().manual_seed(2)
    x = torch.randn((N, H), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((N, E), generator=g).cuda()
    w = pl.quantize_expert_weights(torch.randn((E, 2 * inner, H), generator=g).cuda(),
                                   torch.randn((E, H, inner), generator=g).cuda())
    emap = torch.arange(E, dtype=torch.int32)
    emap[2:4] = -1
    buf = pl.make_layer_buffers(N, E, K, H, inner, 1)
    ro = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    pl.expert_layer(x, logits, ro, w, buf, expert_map=emap.cuda())
    ids, _ = ep.ep_gate_topk(logits, K, SIG)
    assert torch.equal(buf.picks, ids) and not torch.equal(buf.idx, ids)
    d_w = torch.randn((N, K), generator=g)
    got = ep.ep_gate_topk_backward(d_w.cuda(), logits, buf.picks, SIG).double().cpu().numpy()
    for t in range(N):
        want = ref.gate_grad_row(logits[t].double().cpu().numpy(), ids[t].cpu().numpy(), d_w[t].double().numpy(),
                                 False, True, 1.0)
        assert np.abs(got[t] - want).max() <= GRAD_TOL * float(d_w[t].abs().max())
