"""Calls of the FP8 layer's operators that their arguments allow and sizes alone do not
reach: tensors that start on 16 bytes but not on 32, torch's own type of the codes, the
least and the most columns and experts, weights that are not finite, calls at once on
two streams, replays of a graph on other inputs.  Most of them compare two ways of the
same call bit for bit; the rest has the bounds that test_gpu_norm derives."""
import numpy as np
import pytest
import torch

import _fp8_ref as ref
import combine_ep_route_topk_gb300 as ep
from test_gpu_norm import EPS, SUM, U, half, n64, rows_of, weight_of

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MASKED = ep.EP_LAYOUT_MASKED
PAD = 16  # bytes


def off16(t):
    """A copy that starts 16 bytes past a boundary of 32."""
    t = t.cuda().contiguous()
    n = t.numel() * t.element_size()
    raw = torch.empty(n + 64, dtype=torch.uint8, device="cuda")
    start = -raw.data_ptr() % 32 + PAD
    out = raw[start:start + n].view(t.dtype).view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


def on32(t):
    t = t.cuda().contiguous()
    assert t.data_ptr() % 32 == 0
    return t


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(3, 16), (7, 1040), (40, 528), (5, 8208)])
def test_rows_on_16_bytes(rows, cols, dtype):
    x, r, dy, w = (rows_of(rows, cols, dtype, cols), rows_of(rows, cols, dtype, 1),
                   rows_of(rows, cols, dtype, 2), weight_of(cols, dtype))
    wide = torch.cat([x, r], 1)

    def every(at):
        out = ep.alloc_norm(rows, cols, dtype, "cuda", residual=True, codes=True, rstd=True)
        out = ep.Norm(at(out.y), at(out.residual), at(out.q), out.scales, out.rstd)
        ep.ep_rms_norm(at(x), at(w), at(r), EPS, out)
        dx, dw = ep.ep_rms_norm_backward(at(dy), out.residual, at(w), out.rstd, at(r), d_x=at(dy))
        q, s = ep.ep_quantize_blocks(at(x), q=at(torch.zeros((rows, cols), dtype=torch.uint8)))
        xq = at(torch.zeros((rows, 2 * cols), dtype=torch.uint8))
        xs = torch.empty((rows, ep.scale_blocks(2 * cols)), device="cuda")
        h, hs = ep.ep_quantize_blocks(at(wide), act=ep.EP_ACT_SWIGLU, x_q=xq, x_scales=xs)
        v = ep.ep_dequantize_blocks(at(q), s, out=at(dy))
        g1 = ep.ep_swiglu_backward(at(dy), xq, xs, d_x=at(wide))
        g2 = ep.ep_swiglu_backward(at(dy), at(wide), d_x=at(wide))
        return [*out, dx, dw, q, s, xq, xs, h, hs, v, g1, g2]
    for a, b in zip(every(on32), every(off16)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("rows", [30, 700])
def test_product_on_16_bytes_and_typed_codes(rows, out_dtype):
    """Both shapes of the kernel; codes as uint8 and as torch.float8_e4m3fn."""
    E, Nc, Kd = 8, 4992, 272
    g = torch.Generator().manual_seed(rows)
    n = E * rows
    x = torch.randn((n, Kd), generator=g).to(torch.float8_e4m3fn).cuda()
    w = torch.randn((E, Nc, Kd), generator=g).to(torch.float8_e4m3fn).cuda()
    xs = torch.rand((n, 3), generator=g).cuda()
    ws = torch.rand((E, 39, 3), generator=g).cuda()
    offs = torch.arange(0, n + 1, rows, dtype=torch.int32, device="cuda")
    a = ep.ep_expert_matmul_fp8(x, xs, w, ws, offs, out_dtype=out_dtype)
    b = ep.ep_expert_matmul_fp8(off16(x.view(torch.uint8)), xs, off16(w.view(torch.uint8)), ws,
                                offs, out=off16(torch.zeros((n, Nc), dtype=out_dtype)))
    assert torch.equal(a, b)


def test_typed_codes_of_rows():
    x = rows_of(6, 272, BF, 4).cuda()
    q, s = ep.ep_quantize_blocks(x)
    typed = torch.empty((6, 272), dtype=torch.float8_e4m3fn, device="cuda")
    ep.ep_quantize_blocks(x, q=typed)
    assert torch.equal(typed.view(torch.uint8), q)
    assert torch.equal(ep.ep_dequantize_blocks(typed, s), ep.ep_dequantize_blocks(q, s))
    wide = torch.cat([typed, typed], 1)
    ws = torch.rand((6, 5), device="cuda")
    d = rows_of(6, 272, BF, 5).cuda()
    assert torch.equal(ep.ep_swiglu_backward(d, wide, ws),
                       ep.ep_swiglu_backward(d, wide.view(torch.uint8), ws))


@pytest.mark.parametrize("rows,cols", [(100003, 16), (70001, 32), (1, 16384), (400, 16384)])
def test_norm_of_the_least_and_most_columns(rows, cols):
    x, w, dy = rows_of(rows, cols, BF, 6), weight_of(cols, F32), rows_of(rows, cols, BF, 7)
    out = ep.ep_rms_norm(x.cuda(), w.cuda())
    y, rstd = ref.norm(n64(x), n64(w), EPS)
    assert (np.abs(n64(out.y) - y) <= (SUM / 2 + 8 * U + half(BF)) * np.abs(y)).all()
    dx, dw = ep.ep_rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), out.rstd)
    want, mag, wdw, mdw = ref.norm_grad(n64(dy), n64(x), n64(w), n64(out.rstd), None)
    assert (np.abs(n64(dx) - want) <= (2 * SUM + 8 * U) * mag + half(BF) * np.abs(want)).all()
    assert (np.abs(n64(dw) - wdw) <= (rows + 40) * U * mdw).all()


def test_infinite_weight_in_the_last_columns():
    """mean(g n) is infinite, so every other column is; threads past the row's end, which
    have no columns, add nothing to it."""
    rows, cols = 3, 1040
    x, dy, w = torch.ones((rows, cols)), torch.ones((rows, cols)), torch.ones(cols)
    w[-1] = float("inf")
    rstd = torch.ones(rows)
    dx, dw = ep.ep_rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), rstd.cuda())
    assert (dx[:, :-1] == -float("inf")).all() and dx[:, -1].isnan().all()
    assert (dw == rows).all()


def test_many_experts_of_one_row():
    E, Nc, Kd, cap = 1024, 40, 144, 2
    g = torch.Generator().manual_seed(9)
    counts = torch.randint(0, 3, (E,), generator=g)
    offs = torch.cat([torch.zeros(1), counts.cumsum(0)]).int().cuda()
    n = int(counts.sum())
    x = torch.randint(-8, 9, (n, Kd), generator=g).float().to(torch.float8_e4m3fn).cuda()
    w = torch.randint(-8, 9, (E, Nc, Kd), generator=g).float().to(torch.float8_e4m3fn).cuda()
    xs, ws = torch.ones((n, 2), device="cuda"), torch.ones((E, 1, 2), device="cuda")
    owner = torch.repeat_interleave(torch.arange(E), counts).cuda()
    want = torch.einsum("rk,rnk->rn", x.double(), w.double()[owner])  # exact in float32 too
    got = ep.ep_expert_matmul_fp8(x, xs, w, ws, offs, out_dtype=F32)
    assert torch.equal(got.double(), want)
    out = torch.full((E * cap, Nc), -3.0, device="cuda")
    src = torch.arange(n, dtype=torch.int32, device="cuda")
    ep.ep_expert_matmul_fp8(x, xs, w, ws, offs, layout=MASKED, cap=cap, row_src=src, out=out)
    place = owner * cap + src - offs.long()[owner]
    assert torch.equal(out[place].double(), want)
    rest = torch.ones(E * cap, dtype=torch.bool, device="cuda")
    rest[place] = False
    assert (out[rest] == -3.0).all()


def test_one_source_for_every_row():
    """row_src may hold the same row many times."""
    g = torch.Generator().manual_seed(10)
    x = torch.randint(-8, 9, (3, 272), generator=g).float().to(torch.float8_e4m3fn).cuda()
    w = torch.randint(-8, 9, (2, 136, 272), generator=g).float().to(torch.float8_e4m3fn).cuda()
    xs, ws = torch.ones((3, 3), device="cuda"), torch.ones((2, 2, 3), device="cuda")
    offs = torch.tensor([0, 150, 290], dtype=torch.int32, device="cuda")
    src = torch.ones(290, dtype=torch.int32, device="cuda")
    got = ep.ep_expert_matmul_fp8(x, xs, w, ws, offs, row_src=src, out_dtype=F32).double()
    want = torch.einsum("k,enk->en", x[1].double(), w.double())
    assert (got[:150] == want[0]).all() and (got[150:] == want[1]).all()


def test_norm_gradients_at_once_on_two_streams():
    rows, cols = 3000, 2880
    w = weight_of(cols, F32).cuda()
    x, dy = [rows_of(rows, cols, BF, s).cuda() for s in (1, 2)], rows_of(rows, cols, BF, 3).cuda()
    outs = [ep.ep_rms_norm(t, w) for t in x]
    want = [ep.ep_rms_norm_backward(dy, t, w, o.rstd) for t, o in zip(x, outs)]
    size = ep.ep_rms_norm_backward_workspace_size(rows, cols)
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in x]
    got = [(torch.empty_like(t), torch.empty(cols, device="cuda")) for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(20):
        for t, o, ws, (dx, dw), s in zip(x, outs, spaces, got, streams):
            ep.ep_rms_norm_backward(dy, t, w, o.rstd, d_x=dx, d_weight=dw, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, d)


def test_block_codes_in_a_graph_with_other_rows():
    """The replay sees the inputs, and the rows that hold a token, of its own time."""
    rows, cols, E = 96, 272, 4
    x = torch.zeros((rows, 2 * cols), dtype=BF, device="cuda")
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    d = rows_of(rows, cols, BF, 8).cuda()
    q = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    s = torch.empty((rows, 3), device="cuda")
    xq = torch.empty((rows, 2 * cols), dtype=torch.uint8, device="cuda")
    xs = torch.empty((rows, 5), device="cuda")
    dx, v = torch.empty_like(x), torch.empty((rows, cols), device="cuda")
    kw = dict(expert_offsets=offs, layout=MASKED, cap=rows // E)

    def calls():
        ep.ep_quantize_blocks(x, act=ep.EP_ACT_SWIGLU, q=q, scales=s, x_q=xq, x_scales=xs, **kw)
        ep.ep_dequantize_blocks(q, s, out=v, **kw)
        ep.ep_swiglu_backward(d, xq, xs, d_x=dx, **kw)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed, counts in ((1, [24, 0, 5, 1]), (2, [0, 24, 3, 40])):
        x.copy_(rows_of(rows, 2 * cols, BF, seed))
        offs[1:] = torch.tensor(np.cumsum(counts), dtype=torch.int32).cuda()
        for t in (q, xq):
            t.fill_(9)
        for t in (s, xs, dx, v):
            t.fill_(7.0)
        graph.replay()
        got = [t.clone() for t in (q, s, xq, xs, dx, v)]
        for t in (q, xq):
            t.fill_(9)
        for t in (s, xs, dx, v):
            t.fill_(7.0)
        calls()
        for a, b in zip(got, (q, s, xq, xs, dx, v)):
            assert torch.equal(a, b)
        held = torch.zeros(rows, dtype=torch.bool)
        for e, n in enumerate(counts):
            held[e * 24:e * 24 + min(n, 24)] = True
        assert ((dx == 7.0).all(1).cpu() == ~held).all() and ((v == 7.0).all(1).cpu() == ~held).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (37, 48), (19, 144), (9, 1440), (5, 2896), (3, 6096),
                                       (3, 6160), (3, 8176), (3, 8208)])
def test_checkpoint_whose_blocks_straddle_the_halves(rows, cols, dtype):
    """One call writes what two calls write."""
    x = rows_of(rows, 2 * cols, dtype, cols).cuda()
    x[0, 5], x[-1, cols + 7] = float("nan"), float("inf")
    xq = torch.full((rows + 1, 2 * cols), 9, dtype=torch.uint8, device="cuda")
    xs = torch.full((rows + 1, ep.scale_blocks(2 * cols)), 7.0, device="cuda")
    q, s = ep.ep_quantize_blocks(x, act=ep.EP_ACT_SWIGLU, x_q=xq[:rows], x_scales=xs[:rows])
    for a, b in zip((q, s), ep.ep_quantize_blocks(x, act=ep.EP_ACT_SWIGLU)):
        assert torch.equal(a, b)
    wq, wsc = ep.ep_quantize_blocks(x)
    same = (xq[:rows] == wq) | (((xq[:rows] & 127) == 127) & ((wq & 127) == 127))  # NaN of any sign
    assert same.all() and torch.equal(xs[:rows], wsc)
    assert (xq[rows] == 9).all() and (xs[rows] == 7.0).all()
