"""ep_gate_topk and ep_gate_topk_backward against the plain 64-bit form.

Tolerances.  A score carries expf's 2 ulp, one addition and one division; the
softmax adds |l - m| 2^-24 from the rounded difference (|d| <= 40 here), a sum
of at most 1024 terms in lanes (37 roundings) and K <= 32 more for the
renormalisation: together below (40 + 4 + 37 + 32 + 4) 2^-23 < 1.5e-5 relative.
Keys therefore agree with the 64-bit ones within KEY_TOL of the row's largest
score, and ids must be the same wherever neighbours in the order are further
apart than that or exactly equal (ties go to the lower id)."""
import numpy as np
import pytest
import torch

import _expert_ref as ref
import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu
RTOL = 1.5e-5
KEY_TOL = 1e-6
SIG, SOFT = ep.EP_SCORE_SIGMOID, ep.EP_SCORE_SOFTMAX


def make(N, E, dtype, seed, masked=0.0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((N, E), generator=g) * spread).to(dtype)
    if masked:
        x[torch.rand((N, E), generator=g) < masked] = -float("inf")
        x[:: 7] = -float("inf")
    return x


def check(logits, K, score, bias, groups, topk_groups, group_top, renorm, scale, idx, w):
    L = logits.double().numpy()
    b = None if bias is None else bias.double().numpy()
    idx, w = idx.cpu().numpy(), w.double().cpu().numpy()
    same = 0
    for t in range(L.shape[0]):
        rid, rw, key = ref.gate_row(L[t], K, score == SOFT, b, groups, topk_groups, group_top,
                                    renorm, scale)
        got = idx[t]
        assert ((got == -1) == (rid == -1)).all(), (t, got, rid)
        n = int((rid >= 0).sum())
        assert len(set(got[:n])) == n
        if not np.array_equal(got, rid):
            # only experts (or groups) that the 64-bit form holds for as good
            tol = KEY_TOL * max(1.0, np.abs(key[rid[:n]]).max())
            assert np.abs(key[got[:n]] - key[rid[:n]]).max() <= tol, (t, got, rid)
            for k in range(n - 1):
                assert key[got[k]] != key[got[k + 1]] or got[k] < got[k + 1]
        else:
            same += 1
        np.testing.assert_allclose(w[t], ref.weights_of(L[t], got, score == SOFT, renorm, scale), rtol=RTOL,
                                   atol=1e-37)
    assert same >= 0.99 * L.shape[0]


CASES = [
    # N, E, K, score, bias, groups, topk_groups, group_top, renorm, scale, dtype, masked
    (1, 256, 8, SIG, True, 8, 4, 2, True, 2.5, torch.float32, 0.0),
    (67, 256, 8, SIG, True, 8, 4, 2, True, 2.5, torch.bfloat16, 0.0),
    (130, 256, 8, SOFT, False, 1, 1, 2, True, 1.0, torch.float32, 0.0),
    (65, 61, 6, SOFT, False, 1, 1, 1, False, 1.0, torch.float32, 0.1),
    (33, 1, 1, SIG, False, 1, 1, 1, False, 1.0, torch.float32, 0.0),
    (40, 1, 1, SOFT, True, 1, 1, 1, True, 3.0, torch.bfloat16, 0.0),
    (50, 160, 6, SOFT, False, 8, 3, 1, False, 16.0, torch.float32, 0.0),
    (50, 160, 6, SOFT, True, 8, 3, 2, True, 1.0, torch.bfloat16, 0.05),
    (31, 32, 32, SIG, True, 1, 1, 1, True, 1.0, torch.float32, 0.0),
    (31, 1024, 32, SOFT, True, 32, 5, 2, True, 1.0, torch.float32, 0.1),
    (31, 1000, 17, SIG, False, 25, 7, 2, False, 1.0, torch.bfloat16, 0.1),
    (29, 510, 3, SIG, True, 30, 1, 1, True, 1.0, torch.float32, 0.0),
    (29, 129, 5, SOFT, True, 3, 2, 2, False, 0.5, torch.float32, 0.3),
    (64, 16, 2, SIG, False, 4, 2, 2, True, 1.0, torch.float32, 0.5),
    (64, 12, 4, SIG, True, 12, 5, 2, True, 1.0, torch.float32, 0.2),
    (2050, 128, 4, SIG, True, 4, 2, 1, True, 1.0, torch.bfloat16, 0.0),
    (70, 100, 8, SIG, True, 5, 3, 2, True, 1.0, torch.float32, 0.1),
    (70, 128, 6, SOFT, True, 8, 4, 2, False, 1.0, torch.float32, 0.0),
    (70, 200, 4, SOFT, False, 1, 1, 1, True, 1.0, torch.bfloat16, 0.9),
    (70, 256, 5, SIG, False, 32, 9, 2, True, 1.0, torch.float32, 0.6),
    (4099, 256, 8, SOFT, False, 4, 2, 2, True, 1.0, torch.float32, 0.0),
]


@pytest.mark.parametrize("N,E,K,score,bias,groups,tg,gt,renorm,scale,dtype,masked", CASES)
def test_gate_against_plain(N, E, K, score, bias, groups, tg, gt, renorm, scale, dtype, masked):
    logits = make(N, E, dtype, seed=N + E, masked=masked)
    b = torch.randn(E, generator=torch.Generator().manual_seed(5)) * 0.1 if bias else None
    idx, w = ep.ep_gate_topk(logits.cuda(), K, score, bias=None if b is None else b.cuda(),
                             groups=groups, topk_groups=tg, group_top=gt, renorm=renorm,
                             scale=scale)
    check(logits, K, score, b, groups, tg, gt, renorm, scale, idx, w)


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,groups", [(256, 8), (96, 4), (40, 1)])
def test_gate_ties_go_to_the_lower_id(score, bias, E, groups):
    g = torch.Generator().manual_seed(3)
    logits = torch.randint(-2, 3, (64, E), generator=g).float()
    logits[logits == 0] *= torch.where(torch.rand((logits == 0).sum(), generator=g) < 0.5, -1.0, 1.0)
    b = torch.zeros(E) if bias else None
    tg = max(1, groups // 2)
    idx, w = ep.ep_gate_topk(logits.cuda(), 8, score, bias=None if b is None else b.cuda(),
                             groups=groups, topk_groups=tg, group_top=2)
    for t in range(64):
        rid, _, _ = ref.gate_row(logits[t].double().numpy(), 8, score == SOFT,
                                 None if b is None else b.double().numpy(), groups, tg, 2, True, 1.0)
        assert np.array_equal(idx[t].cpu().numpy(), rid), t


WIDE = [(160, 6, 8), (160, 16, 8), (144, 6, 8), (129, 4, 3), (150, 8, 1), (257, 1, 1), (300, 5, 1), (384, 8, 8),
        (384, 8, 1), (384, 12, 6), (385, 8, 5), (512, 7, 16), (512, 9, 1), (640, 8, 4), (1000, 8, 1), (1024, 3, 4)]


@pytest.mark.parametrize("E,K,groups", WIDE)
@pytest.mark.parametrize("score,bias,dtype", [(SIG, True, torch.float32), (SOFT, False, torch.bfloat16)])
def test_gate_of_many_experts(E, K, groups, score, bias, dtype):
    logits = make(41, E, dtype, seed=E + K, masked=0.02)
    b = torch.randn(E, generator=torch.Generator().manual_seed(6)) * 0.1 if bias else None
    tg = max(1, groups // 2)
    idx, w = ep.ep_gate_topk(logits.cuda(), K, score, bias=None if b is None else b.cuda(), groups=groups,
                             topk_groups=tg, group_top=2)
    check(logits, K, score, b, groups, tg, 2, True, 1.0, idx, w)


@pytest.mark.parametrize("E,K,groups", WIDE)
def test_gate_of_many_experts_ties(E, K, groups):
    """Equal keys within a lane and across lanes, in numbers beyond K; rows with fewer than K experts."""
    g = torch.Generator().manual_seed(E)
    logits = torch.randint(0, 3, (24, E), generator=g).float()
    logits[8:16] = 1.0
    logits[16:][torch.rand(8, E, generator=g) < 0.99] = float("-inf")
    tg = max(1, groups // 2)
    idx, w = ep.ep_gate_topk(logits.cuda(), K, SIG, groups=groups, topk_groups=tg, group_top=2)
    for t in range(24):
        rid, _, _ = ref.gate_row(logits[t].double().numpy(), K, False, None, groups, tg, 2, True, 1.0)
        assert np.array_equal(idx[t].cpu().numpy(), rid), t


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("groups", [1, 4])
def test_gate_special_values(score, renorm, groups):
    """-inf, NaN, +inf, the type's lowest value and rows that hold nothing else."""
    inf, nan, low = float("inf"), float("nan"), float(np.finfo(np.float32).min)
    E, K = 16, 4
    rows = [[0.5] * E, [-inf] * E, [nan] * E, [low] * E, [inf] * E, [-inf] * 13 + [1.0, 2.0, nan],
            [inf, -inf] * 8, [low] * 15 + [0.0], [nan, 3.0] + [-inf] * 14,
            [-200.0] * 8 + [-300.0] * 8, [88.0, 90.0] + [-90.0] * 14, [0.0, -0.0] * 8]
    logits = torch.tensor(rows)
    for b in (None, torch.linspace(-0.5, 0.5, E), torch.tensor([-inf, nan] + [0.0] * 14)):
        idx, w = ep.ep_gate_topk(logits.cuda(), K, score, bias=None if b is None else b.cuda(),
                                 groups=groups, topk_groups=max(1, groups // 2), group_top=2,
                                 renorm=renorm)
        assert not torch.isnan(w).any()
        bb = None if b is None else b.double().numpy()
        for t, r in enumerate(rows):
            rid, rw, _ = ref.gate_row(np.array(r), K, score == SOFT, bb, groups,
                                      max(1, groups // 2), 2, renorm, 1.0)
            assert np.array_equal(idx[t].cpu().numpy(), rid), (t, b, idx[t], rid)
            np.testing.assert_allclose(w[t].double().cpu().numpy(), rw, rtol=RTOL, atol=1e-37)


def test_gate_maps_ids_and_feeds_the_layout():
    N, E, K = 300, 64, 6
    logits = make(N, E, torch.float32, 9, masked=0.4)
    emap = torch.randperm(E, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    emap[3] = -1  # an expert that is renumbered to nothing
    plain, w0 = ep.ep_gate_topk(logits.cuda(), K, SIG, scale=2.0)
    idx, w = ep.ep_gate_topk(logits.cuda(), K, SIG, scale=2.0, expert_map=emap.cuda())
    p = plain.cpu()
    want = torch.where(p >= 0, emap[p.clamp(min=0).long()], -1)
    assert torch.equal(idx.cpu(), want) and torch.equal(w, w0)
    lay = ep.ep_dispatch_layout(idx, torch.tensor([0, N], dtype=torch.int32, device="cuda"), E)
    assert int(lay.expert_offsets[-1]) == int((want >= 0).sum())


def test_gate_unaligned_rows():
    """Rows that start off the vector boundary: a view one element into a buffer."""
    for dtype in (torch.float32, torch.bfloat16):
        logits = make(37, 256, dtype, 21)
        buf = torch.empty(37 * 256 + 1, dtype=dtype, device="cuda")
        view = buf[1:].view(37, 256)
        view.copy_(logits)
        a = ep.ep_gate_topk(view, 8, SIG, groups=8, topk_groups=4)
        b = ep.ep_gate_topk(logits.cuda(), 8, SIG, groups=8, topk_groups=4)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        g = torch.randn(37, 8, device="cuda")
        da = ep.ep_gate_topk_backward(g, view, a[0], SIG)
        db = ep.ep_gate_topk_backward(g, logits.cuda(), a[0], SIG)
        assert torch.equal(da, db)


def test_gate_empty_batch_streams_and_graph():
    idx, w = ep.ep_gate_topk(torch.empty((0, 64), device="cuda"), 4, SIG)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    d = ep.ep_gate_topk_backward(w, torch.empty((0, 64), device="cuda"), idx, SIG)
    assert d.shape == (0, 64)
    logits = make(200, 256, torch.float32, 2).cuda()
    out = (torch.empty((200, 8), dtype=torch.int32, device="cuda"),
           torch.empty((200, 8), device="cuda"))
    want = ep.ep_gate_topk(logits, 8, SIG)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ep.ep_gate_topk(logits, 8, SIG, topk_idx=out[0], topk_w=out[1])
    logits.copy_(make(200, 256, torch.float32, 3))
    g.replay()
    want = ep.ep_gate_topk(logits, 8, SIG)
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


# ---- gradient ---------------------------------------------------------------------------------
# The gradient of a token is a few products of scores: its error is relative to the largest term,
# |scale| max|g| (|dl| <= |scale| (|g| + |sum q g|) / 4 for the sigmoid, / 1 for the softmax), with
# the same count of roundings as the weights, twice: GRAD_TOL.
GRAD_TOL = 3e-5

GRAD = [
    # N, E, K, score, renorm, scale, dtype, masked
    (1, 256, 8, SIG, True, 2.5, torch.float32, 0.0),
    (70, 256, 8, SIG, True, 2.5, torch.bfloat16, 0.0),
    (70, 256, 8, SIG, False, 1.0, torch.float32, 0.0),
    (70, 256, 8, SOFT, True, 1.0, torch.float32, 0.0),
    (70, 128, 4, SOFT, False, 2.0, torch.float32, 0.1),
    (41, 61, 6, SOFT, False, 1.0, torch.bfloat16, 0.3),
    (41, 61, 6, SIG, True, 1.0, torch.float32, 0.3),
    (20, 1024, 32, SOFT, False, 1.0, torch.float32, 0.0),
    (20, 1023, 32, SIG, True, 1.0, torch.float32, 0.1),
    (20, 1, 1, SIG, False, 1.0, torch.float32, 0.0),
    (20, 3, 1, SOFT, True, 1.0, torch.float32, 0.0),
    (4103, 61, 8, SIG, True, 1.5, torch.float32, 0.2),
    (4097, 256, 8, SOFT, True, 1.0, torch.bfloat16, 0.0),
    (4098, 96, 5, SIG, False, 1.0, torch.float32, 0.9),
]


@pytest.mark.parametrize("N,E,K,score,renorm,scale,dtype,masked", GRAD)
def test_gate_gradient_against_formula(N, E, K, score, renorm, scale, dtype, masked):
    logits = make(N, E, dtype, seed=N * E, masked=masked)
    g = torch.randn((N, K), generator=torch.Generator().manual_seed(8))
    idx, _ = ep.ep_gate_topk(logits.cuda(), K, score, renorm=renorm, scale=scale)
    d = torch.full((N, E), 7.0, dtype=dtype, device="cuda")
    ep.ep_gate_topk_backward(g.cuda(), logits.cuda(), idx, score, renorm=renorm, scale=scale,
                             d_logits=d)
    got, L, ids = d.double().cpu().numpy(), logits.double().numpy(), idx.cpu().numpy()
    for t in range(N):
        want = ref.gate_grad_row(L[t], ids[t], g[t].double().numpy(), score == SOFT, renorm, scale)
        tol = GRAD_TOL * scale * float(g[t].abs().max())
        if dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(want)
        assert (np.abs(got[t] - want) <= tol).all(), (t, np.abs(got[t] - want).max())
        other = np.ones(E, dtype=bool)
        other[ids[t][ids[t] >= 0]] = False
        if score == SIG or renorm:
            assert (got[t][other] == 0).all()


@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_against_differences(score, renorm):
    """Central differences of the 64-bit weights (picks held): with h = 1e-5
    the truncation is below h^2 and the cancellation below 1e-16 / h."""
    N, E, K, scale, h = 6, 40, 5, 2.5, 1e-5
    logits = make(N, E, torch.float32, 77)
    g = torch.randn((N, K), generator=torch.Generator().manual_seed(8))
    idx, _ = ep.ep_gate_topk(logits.cuda(), K, score, renorm=renorm, scale=scale)
    got = ep.ep_gate_topk_backward(g.cuda(), logits.cuda(), idx, score, renorm=renorm,
                                   scale=scale).double().cpu().numpy()
    ids, G = idx.cpu().numpy(), g.double().numpy()
    for t in range(N):
        L = logits[t].double().numpy()

        def loss(x):
            w = ref.weights_of(x, ids[t], score == SOFT, renorm, scale)
            return float((w * G[t]).sum())
        for e in range(E):
            up, dn = L.copy(), L.copy()
            up[e] += h
            dn[e] -= h
            diff = (loss(up) - loss(dn)) / (2 * h)
            assert abs(got[t, e] - diff) <= GRAD_TOL * scale * np.abs(G[t]).max() + 1e-8


def test_gate_gradient_maps_ids_back_and_skips_no_picks():
    N, E, K = 50, 96, 6
    logits = make(N, E, torch.float32, 4)
    emap = torch.randperm(E, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    g = torch.randn((N, K), device="cuda")
    plain, _ = ep.ep_gate_topk(logits.cuda(), K, SIG)
    mapped, _ = ep.ep_gate_topk(logits.cuda(), K, SIG, expert_map=emap)
    a = ep.ep_gate_topk_backward(g, logits.cuda(), plain, SIG)
    b = ep.ep_gate_topk_backward(g, logits.cuda(), mapped, SIG, expert_map=emap)
    assert torch.equal(a, b)
    bad = plain.clone()
    bad[:, 2] = -1
    bad[:, 4] = E + 7
    d = ep.ep_gate_topk_backward(g, logits.cuda(), bad, SIG).double().cpu().numpy()
    for t in range(N):
        want = ref.gate_grad_row(logits[t].double().numpy(), bad[t].cpu().numpy(),
                                 g[t].double().cpu().numpy(), False, True, 1.0)
        assert np.abs(d[t] - want).max() <= GRAD_TOL * float(g[t].abs().max())


def test_gate_gradient_of_masked_and_saturated_logits_is_finite():
    inf, low = float("inf"), float(np.finfo(np.float32).min)
    logits = torch.tensor([[-inf] * 8, [low] * 8, [inf] * 8, [-200.0] * 8, [200.0] * 8,
                           [inf, low, -inf, 0.0, 1.0, 2.0, 3.0, 4.0]])
    g = torch.ones((6, 3), device="cuda")
    for score in (SIG, SOFT):
        for renorm in (True, False):
            idx, _ = ep.ep_gate_topk(logits.cuda(), 3, score, renorm=renorm)
            d = ep.ep_gate_topk_backward(g, logits.cuda(), idx, score, renorm=renorm)
            assert torch.isfinite(d).all(), (score, renorm, d)
            assert (d[0] == 0).all()
