"""ep_rms_norm and ep_rms_norm_backward against the plain 64-bit forms.

Sums over a row run over at most 64 terms a thread, 5 steps of a warp and 16 warps:
SUM = 96 roundings of 2^-24 cover them with their products.  rstd halves the sum's
error and adds a quotient, a sum, a root and a quotient; y adds two products and its
type's half step; a gradient's terms carry a sum's error each.  d_weight's sums
have one rounding per row and join 32 strands."""
import numpy as np
import pytest
import torch

import _fp8_ref as ref
import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu
EPS = 1e-6
U = 2.0 ** -24
SUM = 96 * U
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 16), (1, 7168), (5, 48), (9, 272), (17, 512), (3, 1024), (7, 1040), (33, 2880),
         (13, 4096), (3, 8192), (2, 8208), (3, 16384), (1300, 112), (700, 528)]


def n64(t):
    return t.double().cpu().numpy()


def rows_of(rows, cols, dtype, seed, loud=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * (0.1 + torch.rand((rows, 1), generator=g)) * loud
    if rows > 2:
        x[1] = 0.0
    return x.to(dtype)


def weight_of(cols, dtype):
    return (1.0 + 0.3 * torch.randn((cols,), generator=torch.Generator().manual_seed(cols))).to(dtype)


def half(dtype):
    return 2.0 ** -8 if dtype == BF else U


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_against_plain(rows, cols, dtype, wdtype, residual):
    x, w = rows_of(rows, cols, dtype, cols), weight_of(cols, wdtype)
    r = rows_of(rows, cols, dtype, cols + 1) if residual else None
    out = ep.alloc_norm(rows, cols, dtype, "cuda", residual=True, codes=True, rstd=True)
    ep.ep_rms_norm(x.cuda(), w.cuda(), None if r is None else r.cuda(), EPS, out)
    z = (x.float() + r.float()).to(dtype) if residual else x
    assert torch.equal(out.residual.cpu(), z)
    y, rstd = ref.norm(n64(z), n64(w), EPS)
    np.testing.assert_allclose(n64(out.rstd), rstd, rtol=SUM / 2 + 4 * U)
    tol = SUM / 2 + 8 * U
    assert (np.abs(n64(out.y) - y) <= (tol + half(dtype)) * np.abs(y)).all()
    scale = ref.block_scales(y)
    np.testing.assert_allclose(n64(out.scales), scale, rtol=tol + U)
    t = y / ref.widen(scale, cols)
    off = np.abs(ref.values(out.q.cpu().numpy(), n64(out.scales)) / ref.widen(scale, cols) - t)
    assert (off <= ref.half_step(np.abs(t) * (1 + 4 * tol)) + 4 * tol * np.abs(t)).all()


def test_each_output_alone_and_in_place():
    rows, cols = 11, 336
    x, r, w = (t.cuda() for t in (rows_of(rows, cols, BF, 1), rows_of(rows, cols, BF, 2),
                                  weight_of(cols, F32)))
    every = ep.ep_rms_norm(x, w, r, out=ep.alloc_norm(rows, cols, BF, "cuda", residual=True,
                                                      codes=True, rstd=True))
    for on in (dict(y=True), dict(y=False, residual=True), dict(y=False, codes=True),
               dict(y=False, rstd=True)):
        one = ep.ep_rms_norm(x, w, r, out=ep.alloc_norm(rows, cols, BF, "cuda", **on))
        for a, b in zip(one, every):
            assert a is None or torch.equal(a, b)
    plain = ep.ep_rms_norm(x, w, r)
    assert torch.equal(plain.y, every.y) and torch.equal(plain.rstd, every.rstd)
    assert torch.equal(plain.residual, every.residual) and plain.q is None
    # the residual stream updated in place, y over x
    x2, r2 = x.clone(), r.clone()
    ep.ep_rms_norm(x2, w, r2, out=ep.Norm(x2, r2, None, None, None))
    assert torch.equal(x2, every.y) and torch.equal(r2, every.residual)


def test_codes_feed_the_expert_product_like_quantized_rows():
    """float32 rows: the codes are ep_quantize_blocks's of y, bit for bit."""
    x, w = rows_of(9, 400, F32, 3).cuda(), weight_of(400, F32).cuda()
    out = ep.ep_rms_norm(x, w, out=ep.alloc_norm(9, 400, F32, "cuda", codes=True))
    q, s = ep.ep_quantize_blocks(out.y)
    assert torch.equal(out.q, q) and torch.equal(out.scales, s)


def test_nan_infinity_and_overflow():
    x = torch.ones((4, 256))
    x[0, 7], x[1, 9], x[2] = float("nan"), float("inf"), 1e30
    w = torch.ones(256)
    out = ep.ep_rms_norm(x.cuda(), w.cuda())
    y = out.y.cpu()
    assert torch.isnan(y[0]).all()
    assert torch.isnan(y[1, 9]) and (y[1, :9] == 0).all() and float(out.rstd[1]) == 0
    assert (y[2] == 0).all() and float(out.rstd[2]) == 0  # the sum of squares overflows
    want = 1.0 / np.sqrt(1 + EPS)
    assert np.abs(n64(out.y[3]) - want).max() <= want * (SUM / 2 + 6 * U)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_gradient_against_plain(rows, cols, dtype, wdtype, residual):
    z, dy, w = rows_of(rows, cols, dtype, cols), rows_of(rows, cols, dtype, cols + 1), weight_of(cols, wdtype)
    dres = rows_of(rows, cols, dtype, cols + 2) if residual else None
    rstd = torch.from_numpy(ref.norm(n64(z), n64(w), EPS)[1]).float()
    dx, dw = ep.ep_rms_norm_backward(dy.cuda(), z.cuda(), w.cuda(), rstd.cuda(),
                                     None if dres is None else dres.cuda())
    assert dx.dtype == dtype and dw.dtype == F32
    want, mag, wdw, mdw = ref.norm_grad(n64(dy), n64(z), n64(w), n64(rstd),
                                        None if dres is None else n64(dres))
    assert (np.abs(n64(dx) - want) <= (2 * SUM + 8 * U) * mag + half(dtype) * np.abs(want)).all()
    assert (np.abs(n64(dw) - wdw) <= (rows + 40) * U * mdw).all()
    again, none = ep.ep_rms_norm_backward(dy.cuda(), z.cuda(), w.cuda(), rstd.cuda(),
                                          None if dres is None else dres.cuda(), weight_grad=False)
    assert none is None and torch.equal(again, dx)


def test_gradient_against_differences():
    """Central differences of the plain norm in 64 bits, the loss being sum(d y): the
    step's own error is of the order h^2 = 1e-8 of the gradient's terms."""
    rows, cols, h = 3, 48, 1e-4
    z, dy, w = rows_of(rows, cols, F32, 4) + 0.5, rows_of(rows, cols, F32, 5), weight_of(cols, F32)
    y, r = ref.norm(n64(z), n64(w), EPS)
    dx, dw = ep.ep_rms_norm_backward(dy.cuda(), z.cuda(), w.cuda(), torch.from_numpy(r).float().cuda())
    _, mag, _, mdw = ref.norm_grad(n64(dy), n64(z), n64(w), r, None)
    for c in range(cols):
        at = np.zeros(cols)
        at[c] = h
        f = lambda zz, ww: (n64(dy) * ref.norm(zz, ww, EPS)[0]).sum(1)  # noqa: E731
        num = (f(n64(z) + at, n64(w)) - f(n64(z) - at, n64(w))) / (2 * h)
        # third derivatives are bounded by some 20 / rms^2 of the terms; rms > 0.1 here
        assert (np.abs(n64(dx)[:, c] - num) <= 2 * SUM * mag[:, c] + 1e-4 * mag.max(1)).all()
        num = (f(n64(z), n64(w) + at) - f(n64(z), n64(w) - at)).sum() / (2 * h)
        assert abs(n64(dw)[c] - num) <= 40 * U * mdw[c] + 1e-9


def test_gradient_is_the_same_every_time_and_in_place():
    rows, cols = 5003, 528
    z, dy, w = (t.cuda() for t in (rows_of(rows, cols, BF, 6), rows_of(rows, cols, BF, 7), weight_of(cols, F32)))
    dres = rows_of(rows, cols, BF, 8).cuda()
    rstd = ep.ep_rms_norm(z, w).rstd
    dx, dw = ep.ep_rms_norm_backward(dy, z, w, rstd, dres)
    ws = torch.full((ep.ep_rms_norm_backward_workspace_size(rows, cols),), 255, dtype=torch.uint8, device="cuda")
    for over in (dy.clone(), z.clone(), dres.clone()):
        args = [dy, z, w, rstd, dres]
        for i, t in enumerate((dy, z, None, None, dres)):
            if t is not None and torch.equal(t, over):
                args[i] = over
        got, dw2 = ep.ep_rms_norm_backward(*args, d_x=over, workspace=ws)
        assert torch.equal(got, dx) and torch.equal(dw2, dw)


def test_no_rows():
    z, w = torch.zeros((0, 64), device="cuda"), torch.ones(64, device="cuda")
    out = ep.ep_rms_norm(z, w)
    assert out.y.shape == (0, 64)
    dx, dw = ep.ep_rms_norm_backward(z, z, w, out.rstd, d_weight=torch.full((64,), 3.0, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_norm_and_gradient_in_a_graph():
    rows, cols = 130, 1040
    x, r, dy = (rows_of(rows, cols, BF, s).cuda() for s in (1, 2, 3))
    w = weight_of(cols, F32).cuda()
    out = ep.alloc_norm(rows, cols, BF, "cuda", residual=True, codes=True, rstd=True)
    ws = torch.empty((ep.ep_rms_norm_backward_workspace_size(rows, cols),), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty((cols,), device="cuda")

    def step():
        ep.ep_rms_norm(x, w, r, out=out)
        ep.ep_rms_norm_backward(dy, out.residual, w, out.rstd, r, d_x=dx, d_weight=dw, workspace=ws)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        step()
    x.copy_(rows_of(rows, cols, BF, 11))
    dy.copy_(rows_of(rows, cols, BF, 12))
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (*out, dx, dw)]
    step()
    for a, b in zip(got, (*out, dx, dw)):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    cols, rows = 16384, 270000
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free memory")
    x = torch.zeros((rows, cols), dtype=BF, device="cuda")
    last = rows_of(7, cols, BF, 8).cuda()
    x[-7:] = last
    w = weight_of(cols, BF).cuda()
    want = ep.ep_rms_norm(last, w)
    out = ep.alloc_norm(rows, cols, BF, "cuda", rstd=True)
    ep.ep_rms_norm(x, w, out=out)
    assert torch.equal(out.y[-7:], want.y)
    dx, dw = ep.ep_rms_norm_backward(x, x, w, out.rstd, d_x=out.y)
    dx7, dw7 = ep.ep_rms_norm_backward(last, last, w, want.rstd)
    assert torch.equal(dx[-7:], dx7)
    assert (dw - dw7).abs().max() <= 16 * U * dw7.abs().max()  # seven terms, in another order
