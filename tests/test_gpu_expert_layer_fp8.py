"""pipeline.expert_layer_fp8 and the experts' part with its backward pass, against the
same computation in 64 bits.

Quantisation is part of the layer, so the 64-bit form takes the codes that the GPU
wrote (their own tests check them) and rows as bf16, as the layer stores them.  Bounds:
each product _fp8_ref.matmul_tol; SwiGLU and its gradient as in test_gpu_blocks; the
combine within K FMAs and half a bf16 unit.

Against unquantised bf16 weights and rows: a code is off by 2^-3 / sqrt(12) of its
binade's base, 0.026 of the value on average over a binade; rows, first weights (through
SwiGLU, whose slope relative to its value is about 1.2 in each half), inner rows and
second weights give 0.026 * sqrt(2 * 2 * 1.2^2 + 2) = 0.073; twice that is allowed.  The
gradient rounds as often again: 0.1, twice allowed."""
import numpy as np
import pytest
import torch

import _fp8_ref as ref
import combine_ep_route_topk_gb300 as ep
from combine_ep_route_topk_gb300 import pipeline as pl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def n64(t):
    return t.double().cpu().numpy()


def u8(t):
    return t.cpu().numpy()


def make(N, E, K, H, inner, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, H), generator=g).to(BF)
    logits = torch.randn((N, E), generator=g)
    up = (torch.randn((E, 2 * inner, H), generator=g) * H ** -0.5).to(BF)
    down = (torch.randn((E, H, inner), generator=g) * inner ** -0.5).to(BF)
    return x.cuda(), logits.cuda(), up.cuda(), down.cuda()


def near_product(got, x, xs, w, ws, offs, layout, cap, src, rows):
    want, mag, written = ref.matmul(u8(x), n64(xs), u8(w), n64(ws), offs, layout, cap, src, rows)
    rel_mag, rel = ref.matmul_tol(w.shape[2], True)
    assert (np.abs(n64(got) - want) <= rel_mag * mag + rel * np.abs(want))[written].all()
    return written


def near_codes(q, s, v):
    scale = ref.block_scales(v)
    t = v / ref.widen(scale, v.shape[1])
    off = np.abs(ref.values(u8(q), n64(s)) / ref.widen(scale, v.shape[1]) - t)
    assert (off <= ref.half_step(np.abs(t) * (1 + 2.0 ** -15)) + 2.0 ** -14 * np.abs(t)).all()


def check(w, buf, K, xq, xs, in_place):
    mlp = buf.mlp
    offs, src = buf.lay.expert_offsets.cpu().numpy(), buf.lay.row_src.cpu().numpy()
    masked, rows = mlp.layout == ep.EP_LAYOUT_MASKED, mlp.up.shape[0]
    buf.check()
    written = near_product(mlp.up, xq, xs, w.up, w.up_scales, offs, int(masked), mlp.cap,
                           src if in_place else None, rows)
    near_codes(mlp.hq[torch.from_numpy(written).cuda()], mlp.hs[torch.from_numpy(written).cuda()],
               ref.swiglu(n64(mlp.up)[written]))
    near_product(mlp.down, mlp.hq, mlp.hs, w.down, w.down_scales, offs, int(masked), mlp.cap, None, rows)
    got, idx, wt, pos, out = n64(mlp.down), buf.idx.cpu().numpy(), n64(buf.wt), buf.lay.pos.cpu().numpy(), n64(buf.comb)
    for t in range(idx.shape[0]):
        acc, m = np.zeros(out.shape[1]), np.zeros(out.shape[1])
        for k in range(K):
            e, p = idx[t, k], pos[t, k]
            if e < 0 or (masked and p - offs[e] >= mlp.cap):
                continue
            r = e * mlp.cap + p - offs[e] if masked else p
            acc += wt[t, k] * got[r]
            m += np.abs(wt[t, k] * got[r])
        assert (np.abs(out[t] - acc) <= 2 * K * 2.0 ** -24 * m + 2.0 ** -8 * np.abs(acc) + 1e-30).all()


@pytest.mark.parametrize("N,E,K,H,inner,cap,groups", [
    (1, 16, 2, 128, 64, 0, 1),        # one token, dispatched
    (24, 16, 2, 128, 64, 8, 4),       # masked, some experts past their capacity
    (70, 8, 3, 272, 80, 0, 2),        # ragged, odd multiples of 16: read in place
    (300, 4, 2, 256, 144, 200, 1),    # many rows an expert
    (260, 4, 2, 384, 208, 0, 1),
])
def test_layer_against_64_bits(N, E, K, H, inner, cap, groups):
    x, logits, up, down = make(N, E, K, H, inner, N)
    w = pl.quantize_expert_weights_fp8(up, down)
    ro = torch.tensor([0, N // 3, N], dtype=torch.int32, device="cuda")
    buf = pl.make_layer_buffers_fp8(N, E, K, H, inner, 2, cap)
    bias = torch.linspace(-0.1, 0.1, E, device="cuda")
    kw = dict(bias=bias, groups=groups, topk_groups=max(1, groups // 2), scale=2.5)
    pl.expert_layer_fp8(x, logits, ro, w, buf, **kw)
    check(w, buf, K, buf.xq, buf.xs, buf.xq.shape[0] == N and not (cap == 0 and H % 128 == 0))
    # the same from codes that are there already
    q, s = ep.ep_quantize_blocks(x)
    before = buf.comb.clone()
    pl.expert_layer_fp8((q, s), logits, ro, w, buf, **kw)
    check(w, buf, K, q, s, True)
    assert (buf.comb.float() - before.float()).abs().max() <= 2.0 ** -6 * before.float().abs().max()


def test_norm_feeds_the_layer():
    """Residual addition, norm, gate logits and the layer from the norm's codes."""
    N, E, K, H, inner = 33, 8, 2, 256, 128
    x, _, up, down = make(N, E, K, H, inner, 1)
    r = make(N, E, K, H, inner, 2)[0]
    weight = torch.ones(H, device="cuda")
    router = torch.randn((E, H), generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    out = ep.ep_rms_norm(x, weight, r, out=ep.alloc_norm(N, H, BF, "cuda", residual=True, codes=True))
    logits = out.y @ router.T
    ro = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    w = pl.quantize_expert_weights_fp8(up, down)
    buf = pl.make_layer_buffers_fp8(N, E, K, H, inner, 1, 16)
    pl.expert_layer_fp8((out.q, out.scales), logits, ro, w, buf)
    check(w, buf, K, out.q, out.scales, True)


def dense(x, idx, wt, up, down):
    """The layer on unquantised values in 64 bits, with its experts' rows."""
    inner = up.shape[1] // 2
    out = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for k in range(idx.shape[1]):
            e = int(idx[t, k])
            h = up[e] @ x[t]
            out[t] += wt[t, k] * (down[e] @ (torch.nn.functional.silu(h[:inner]) * h[inner:]))
    return out


def test_layer_is_near_the_unquantised_one():
    N, E, K, H, inner = 64, 8, 2, 512, 256
    x, logits, up, down = make(N, E, K, H, inner, 3)
    buf = pl.make_layer_buffers_fp8(N, E, K, H, inner, 1)
    ro = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    out = pl.expert_layer_fp8(x, logits, ro, pl.quantize_expert_weights_fp8(up, down), buf).double()
    want = dense(x.double(), buf.idx, buf.wt.double(), up.double(), down.double())
    assert float((out - want).norm() / want.norm()) < 2 * 0.073


def test_layer_maps_and_tokens_without_picks():
    N, E, K, H, inner = 40, 8, 2, 128, 64
    x, logits, up, down = make(N, E, K, H, inner, 5)
    logits[:, 2:4] = -float("inf")
    logits[7] = -float("inf")
    emap = torch.randperm(E, generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    w = pl.quantize_expert_weights_fp8(up, down)
    for cap in (0, 40):
        buf = pl.make_layer_buffers_fp8(N, E, K, H, inner, 1, cap)
        ro = torch.tensor([0, N], dtype=torch.int32, device="cuda")
        pl.expert_layer_fp8(x, logits, ro, w, buf, expert_map=emap)
        assert (buf.comb[7] == 0).all()
        check(w, buf, K, buf.xq, buf.xs, cap > 0)


def test_layer_in_a_graph():
    N, E, K, H, inner = 32, 16, 4, 256, 128
    x, logits, up, down = make(N, E, K, H, inner, 11)
    w = pl.quantize_expert_weights_fp8(up, down)
    ro = torch.tensor([0, 8, 16, 24, N], dtype=torch.int32, device="cuda")
    for cap in (16, 0):
        buf = pl.make_layer_buffers_fp8(N, E, K, H, inner, 4, cap)
        pl.expert_layer_fp8(x, logits, ro, w, buf)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pl.expert_layer_fp8(x, logits, ro, w, buf)
        x2, logits2, _, _ = make(N, E, K, H, inner, 12 + cap)
        x.copy_(x2)
        logits.copy_(logits2)
        g.replay()
        torch.cuda.synchronize()
        got = buf.comb.clone()
        pl.expert_layer_fp8(x, logits, ro, w, buf)
        assert torch.equal(got, buf.comb)


def test_weights_by_blocks():
    """Each 128 x 128 block by its largest; transposing moves codes and scales only."""
    _, _, up, down = make(1, 3, 1, 272, 144, 7)
    up[1, :128, :128] = 0.0
    w = pl.quantize_expert_weights_fp8(up, down, gradients=True)
    for full, codes, scales in ((up, w.up, w.up_scales), (down, w.down, w.down_scales)):
        for e in range(3):
            v, s = n64(full[e]), n64(scales[e])
            n, k = v.shape
            for i in range(s.shape[0]):
                for j in range(s.shape[1]):
                    b = v[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
                    top = np.abs(b).max()
                    assert abs(s[i, j] - (top / 448 if top else 1.0)) <= 2.0 ** -24 * s[i, j]
                    t = b / s[i, j]
                    got = ref.e4m3(u8(codes[e, i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]))
                    assert (np.abs(got - t) <= ref.half_step(t) + 2.0 ** -22 * np.abs(t)).all()
    assert torch.equal(w.up_t, w.up.transpose(1, 2)) and torch.equal(w.down_t_scales, w.down_scales.transpose(1, 2))
    with pytest.raises(ValueError):
        pl.quantize_expert_weights_fp8(up, up)


def problem(counts, H, inner, cap, seed):
    E = len(counts)
    g = torch.Generator().manual_seed(seed)
    offs = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    rows = E * cap if cap else int(offs[-1]) + 3  # three rows that hold no token
    x = torch.randn((rows, H), generator=g).to(BF).cuda()
    d = (torch.randn((rows, H), generator=g) * 1e-2).to(BF).cuda()
    _, _, up, down = make(1, E, 1, H, inner, seed)
    layout = ep.EP_LAYOUT_MASKED if cap else ep.EP_LAYOUT_CONTIG
    if cap:
        valid = [e * cap + i for e in range(E) for i in range(min(cap, counts[e]))]
    else:
        valid = list(range(int(offs[-1])))
    return offs, rows, x, d, up, down, layout, torch.tensor(valid, device="cuda")


@pytest.mark.parametrize("counts,H,inner,cap", [([3, 0, 40], 128, 64, 0), ([5, 2, 30], 272, 144, 16),
                                                ([200, 1, 60], 256, 128, 0)])
def test_backward_of_the_experts_against_64_bits(counts, H, inner, cap):
    offs, rows, x, d, up, down, layout, valid = problem(counts, H, inner, cap, H)
    w = pl.quantize_expert_weights_fp8(up, down, gradients=True)
    buf = pl.make_mlp_buffers_fp8(rows, H, inner, layout, cap, keep=True)
    xq, xs = ep.ep_quantize_blocks(x)
    o = offs.cuda()
    buf.d_rows.fill_(-3.0)
    pl.expert_mlp_fp8(xq, xs, o, w, buf)
    v = valid.cpu().numpy()
    want_q, want_s = ref.quantize32(buf.up[valid].cpu())
    assert torch.equal(buf.upq[valid].cpu(), want_q) and torch.equal(buf.ups[valid].cpu(), want_s)
    pl.expert_mlp_fp8_backward(d, o, w, buf)
    buf.check()
    args = (offs.numpy(), int(cap > 0), cap, None, rows)
    dq, ds = ep.ep_quantize_blocks(d)
    near_product(buf.d_h, dq, ds, w.down_t, w.down_t_scales, *args)
    up_values = ref.values(u8(buf.upq)[v], n64(buf.ups)[v])
    want, mag = ref.swiglu_grad(up_values, n64(buf.d_h)[v])
    got = n64(buf.d_up)[v]
    assert (np.abs(got - want) <= 2.0 ** -16 * mag + 2.0 ** -8 * np.abs(want) + 1e-37).all()
    gq, gs = ep.ep_quantize_blocks(buf.d_up)
    near_product(buf.d_rows, gq, gs, w.up_t, w.up_t_scales, *args)
    rest = np.setdiff1d(np.arange(rows), v)
    assert (buf.d_rows[torch.from_numpy(rest).cuda()] == -3.0).all()


def test_backward_is_near_the_unquantised_gradient():
    counts, H, inner = [20, 44], 512, 256
    offs, rows, x, d, up, down, layout, valid = problem(counts, H, inner, 0, 21)
    w = pl.quantize_expert_weights_fp8(up, down, gradients=True)
    buf = pl.make_mlp_buffers_fp8(rows, H, inner, keep=True)
    pl.expert_mlp_fp8(*ep.ep_quantize_blocks(x), offs.cuda(), w, buf)
    got = pl.expert_mlp_fp8_backward(d, offs.cuda(), w, buf)[valid].double()
    xd = x.double().requires_grad_()
    out = []
    for e in range(2):
        h = xd[int(offs[e]):int(offs[e + 1])] @ up[e].double().T
        out.append((torch.nn.functional.silu(h[:, :inner]) * h[:, inner:]) @ down[e].double().T)
    (torch.cat(out) * d[valid].double()).sum().backward()
    want = xd.grad[valid]
    assert float((got - want).norm() / want.norm()) < 2 * 0.1


def test_forward_and_backward_in_a_graph():
    counts, H, inner = [30, 0, 9], 256, 128
    offs, rows, x, d, up, down, layout, valid = problem(counts, H, inner, 0, 31)
    w = pl.quantize_expert_weights_fp8(up, down, gradients=True)
    buf = pl.make_mlp_buffers_fp8(rows, H, inner, keep=True)
    xq, xs = ep.ep_quantize_blocks(x)
    o = offs.cuda()

    def step():
        ep.ep_quantize_blocks(x, q=xq, scales=xs)
        pl.expert_mlp_fp8(xq, xs, o, w, buf)
        pl.expert_mlp_fp8_backward(d, o, w, buf)
    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    x.copy_(x.flip(0))
    d.copy_(d.flip(0))
    g.replay()
    torch.cuda.synchronize()
    got = buf.down[valid].clone(), buf.d_rows[valid].clone()
    step()
    assert torch.equal(got[0], buf.down[valid]) and torch.equal(got[1], buf.d_rows[valid])


def test_backward_needs_what_the_forward_kept():
    _, _, up, down = make(1, 2, 1, 128, 64, 1)
    d = torch.zeros((4, 128), dtype=BF, device="cuda")
    o = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for w, keep in ((pl.quantize_expert_weights_fp8(up, down, True), False),
                    (pl.quantize_expert_weights_fp8(up, down), True)):
        with pytest.raises(ValueError):
            pl.expert_mlp_fp8_backward(d, o, w, pl.make_mlp_buffers_fp8(4, 128, 64, keep=keep))
