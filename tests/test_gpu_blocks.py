"""ep_quantize_blocks, ep_dequantize_blocks and ep_swiglu_backward against the plain
forms.

Codes of rows (EP_ACT_NONE) and restored values are defined bit for bit and compared
so.  SwiGLU's values carry, beside a code's half step, the float32 form's error: the
product with log2 e rounds at 2^-24 of |g| <= 100, which the exponential turns into
100 * 1.45 * 2^-24 relative; exponential, sum, reciprocal (2^-22 each) and three
products add less than 2^-20: RTOL = 2^-16 in all.  The gradient has the same and
five more roundings, on the magnitudes of its terms."""
import numpy as np
import pytest
import torch

import _fp8_ref as ref
import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu
CONTIG, MASKED = ep.EP_LAYOUT_CONTIG, ep.EP_LAYOUT_MASKED
SWIGLU = ep.EP_ACT_SWIGLU
RTOL = 2.0 ** -16
SIZES = [(1, 16), (1, 128), (5, 48), (3, 1024), (7, 1040), (33, 2880), (2, 7168), (3, 20000),
         (700, 112), (257, 1440)]


def rows_of(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.rand((rows, 1), generator=g) * 5
    if rows > 2:
        x[1] = 0.0
        x[2] *= 1e-12
    return x.to(dtype)


def n64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_codes_of_rows_bit_for_bit(rows, cols, dtype):
    x = rows_of(rows, cols, dtype, rows + cols)
    q, s = ep.ep_quantize_blocks(x.cuda())
    want_q, want_s = ref.quantize32(x)
    assert torch.equal(s.cpu(), want_s)
    assert torch.equal(q.cpu(), want_q)
    out = ep.ep_dequantize_blocks(q, s, out_dtype=torch.float32)
    v = torch.from_numpy(ref.e4m3(want_q.numpy())).float() * \
        torch.from_numpy(ref.widen(want_s.numpy(), cols))
    assert torch.equal(out.cpu(), v)
    assert torch.equal(ep.ep_dequantize_blocks(q.view(torch.float8_e4m3fn), s).cpu(),
                       v.to(torch.bfloat16))


def test_codes_are_those_of_dispatch():
    N, E, K, H = 40, 8, 2, 384
    x = rows_of(N, H, torch.bfloat16, 1).cuda()
    idx, _ = ep.ep_route_topk(torch.randn((N, E), generator=torch.Generator().manual_seed(2)).cuda(), K)
    lay = ep.ep_dispatch_layout(idx, torch.tensor([0, N], dtype=torch.int32, device="cuda"), E)
    out, scales = ep.ep_dispatch(x, idx, lay.pos, lay.expert_offsets, E,
                                 dtype=ep.EP_DTYPE_FP8_E4M3_B128)
    q, s = ep.ep_quantize_blocks(x)
    src = lay.row_src.long()
    assert torch.equal(out, q[src]) and torch.equal(scales, s[src])


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_swiglu_codes_and_checkpoint(rows, cols, dtype, keep):
    x = rows_of(rows, 2 * cols, dtype, rows + cols)
    x_q = x_s = None
    if keep:
        x_q = torch.zeros((rows, 2 * cols), dtype=torch.uint8, device="cuda")
        x_s = torch.zeros((rows, ep.scale_blocks(2 * cols)), device="cuda")
    q, s = ep.ep_quantize_blocks(x.cuda(), act=SWIGLU, x_q=x_q, x_scales=x_s)
    v = ref.swiglu(n64(x))
    scale = ref.block_scales(v)
    np.testing.assert_allclose(n64(s), scale, rtol=RTOL)
    t = v / ref.widen(scale, cols)
    off = np.abs(ref.values(q.cpu().numpy(), n64(s)) / ref.widen(scale, cols) - t)
    # the code of a value RTOL away, times a scale RTOL away
    assert (off <= ref.half_step(np.abs(t) * (1 + 2 * RTOL)) + 4 * RTOL * np.abs(t)).all()
    if keep:
        want_q, want_s = ref.quantize32(x)
        assert torch.equal(x_q.cpu(), want_q) and torch.equal(x_s.cpu(), want_s)


def test_codes_round_ties_to_even():
    x = torch.zeros((1, 128))
    x[0, 0] = 448.0
    # steps of 1/8 .. of 32: halfway points go to the even mantissa
    x[0, 1:9] = torch.tensor([1.0625, 1.1875, -1.0625, 17.0, 19.0, 432.0, 2.0 ** -10, 3 * 2.0 ** -10])
    q, s = ep.ep_quantize_blocks(x.cuda())
    assert float(s[0, 0]) == 1.0
    got = ref.e4m3(q.cpu().numpy())[0, :9].tolist()
    assert got == [448.0, 1.0, 1.25, -1.0, 16.0, 20.0, 448.0, 0.0, 2.0 ** -8]


def test_signs_of_zeros_and_quotients_at_borders():
    """-0 keeps its sign; multiples of a scale that lie between two codes, with scales
    whose reciprocals are not exact (amax = 448 m for odd m, and m / 7)."""
    x = torch.zeros((64, 256))
    x[:, ::3] = -0.0
    mids = torch.from_numpy(ref.e4m3(np.arange(8, 0x7e, dtype=np.uint8)))
    mids = ((mids[1:] + mids[:-1]) / 2).float()  # 117 values between two codes
    for r in range(64):
        x[r, :117] = mids * (r + 1 if r < 32 else (r - 31) / 7)
        x[r, 127] = 448.0 * (r + 1 if r < 32 else (r - 31) / 7)
    x[5, 128:] = -0.0
    for dtype in (torch.float32, torch.bfloat16):
        q, s = ep.ep_quantize_blocks(x.to(dtype).cuda())
        want_q, want_s = ref.quantize32(x.to(dtype))
        assert torch.equal(s.cpu(), want_s) and torch.equal(q.cpu(), want_q)


def test_tiny_rows_and_zeros():
    x = torch.zeros((4, 256))
    x[0, 5] = 1e-44     # its quotient by 448 is 0
    x[1, 5] = 1e-38
    x[2, 200] = -3e38
    q, s = ep.ep_quantize_blocks(x.cuda())
    q2, s2 = ref.quantize32(x)
    assert torch.equal(q.cpu(), q2) and torch.equal(s.cpu(), s2)
    assert not torch.isnan(ep.ep_dequantize_blocks(q, s)).any()


def test_nan_and_infinity_stay_visible():
    x = torch.ones((3, 272))
    x[0, 3] = float("nan")
    x[1, 130] = -float("inf")
    out = ep.ep_dequantize_blocks(*ep.ep_quantize_blocks(x.cuda()), out_dtype=torch.float32).cpu()
    assert torch.isnan(out[0, 3]) and (torch.isnan(out[0]).sum() == 1)
    assert torch.isnan(out[1, 128:256]).all()
    assert torch.equal(out[1, :128], x[1, :128]) and torch.equal(out[2], x[2])


def holds(layout, cap, offs, r):
    if layout == CONTIG:
        return r < int(offs[-1])
    return r % cap < int(offs[r // cap + 1] - offs[r // cap])


@pytest.mark.parametrize("layout", [CONTIG, MASKED])
def test_rows_without_a_token_are_left(layout):
    cap, cols = 6, 48
    offs = torch.tensor([0, 3, 3, 11, 13], dtype=torch.int32)
    rows = 4 * cap
    x = rows_of(rows, 2 * cols, torch.bfloat16, 3).cuda()
    d = rows_of(rows, cols, torch.bfloat16, 4).cuda()
    kw = dict(expert_offsets=offs.cuda(), layout=layout, cap=cap)

    def fill(shape, t, v):
        return torch.full(shape, v, dtype=t, device="cuda")

    def run(**kw):
        q, s = fill((rows, cols), torch.uint8, 9), fill((rows, 1), torch.float32, -5.0)
        xq, xs = fill((rows, 2 * cols), torch.uint8, 9), fill((rows, 1), torch.float32, -5.0)
        ep.ep_quantize_blocks(x, act=SWIGLU, q=q, scales=s, x_q=xq, x_scales=xs, **kw)
        v = ep.ep_dequantize_blocks(q, s, out=fill((rows, cols), torch.float32, -7.0), **kw)
        a = ep.ep_swiglu_backward(d, x, d_x=fill((rows, 2 * cols), torch.bfloat16, -7.0), **kw)
        b = ep.ep_swiglu_backward(d, xq, xs, d_x=fill((rows, 2 * cols), torch.bfloat16, -7.0), **kw)
        return q, s, xq, xs, v, a, b
    some, every = run(**kw), run()
    before = (9, -5.0, 9, -5.0, -7.0, -7.0, -7.0)
    for r in range(rows):
        for t, full, old in zip(some, every, before):
            if holds(layout, cap, offs, r):
                assert torch.equal(t[r], full[r])
            else:
                assert (t[r] == old).all()


@pytest.mark.parametrize("saved", ["rows", "codes"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_swiglu_gradient(rows, cols, dtype, saved):
    x = rows_of(rows, 2 * cols, dtype, rows + cols)
    d = rows_of(rows, cols, dtype, rows + cols + 1)
    if saved == "rows":
        v = n64(x)
        got = ep.ep_swiglu_backward(d.cuda(), x.cuda())
    else:
        q, s = ref.quantize32(x)
        v = ref.values(q.numpy(), n64(s))
        got = ep.ep_swiglu_backward(d.cuda(), q.cuda(), s.cuda())
    assert got.dtype == dtype
    want, mag = ref.swiglu_grad(v, n64(d))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert (np.abs(n64(got) - want) <= RTOL * mag + half * np.abs(want) + 1e-37).all()


def test_swiglu_gradient_against_differences():
    """Central differences of the plain SwiGLU in 64 bits: their own error is below
    h^2 |f'''| / 6 < 1e-9 of |d u|, and 1e-16 / h = 1e-11."""
    rows, cols, h = 9, 80, 1e-5
    x, d = rows_of(rows, 2 * cols, torch.float32, 5), rows_of(rows, cols, torch.float32, 6)
    got = n64(ep.ep_swiglu_backward(d.cuda(), x.cuda()))
    v, dd = n64(x), n64(d)
    for half in (0, 1):
        step = np.zeros_like(v)
        step[:, half * cols:(half + 1) * cols] = h  # every column moves its own output only
        want = dd * (ref.swiglu(v + step) - ref.swiglu(v - step)) / (2 * h)
        part = slice(half * cols, (half + 1) * cols)
        _, mag = ref.swiglu_grad(v, dd)
        assert (np.abs(got[:, part] - want) <= (RTOL + 2.0 ** -24) * mag[:, part]
                + 1e-8 * np.abs(dd) * (1 + np.abs(v[:, cols:]) + np.abs(v[:, :cols]))).all()


def test_swiglu_gradient_far_out_and_in_place():
    """Gates far from zero: the gradient neither overflows nor cancels; d_x may be x."""
    g = torch.tensor([-200.0, -90.0, -30.0, -1.2784645, 0.0, 30.0, 90.0, 3e38, 1.0, -1.0] + [0.5] * 6)
    x = torch.cat([g, torch.linspace(-2, 2, 16)])[None].contiguous()
    d = torch.full((1, 16), 0.75)
    want, mag = ref.swiglu_grad(n64(x), n64(d))
    xc = x.cuda()
    got = ep.ep_swiglu_backward(d.cuda(), xc)
    assert (np.abs(n64(got) - want) <= (RTOL + 2.0 ** -24) * mag + 1e-34).all()
    assert ep.ep_swiglu_backward(d.cuda(), xc, d_x=xc) is xc
    assert torch.equal(xc, got)


def test_no_rows():
    z = torch.zeros((0, 64), device="cuda")
    q, s = ep.ep_quantize_blocks(z, act=SWIGLU)
    assert q.shape == (0, 32) and s.shape == (0, 1)
    assert ep.ep_dequantize_blocks(q, s).shape == (0, 32)
    assert ep.ep_swiglu_backward(torch.zeros((0, 32), device="cuda"), z).shape == (0, 64)


def test_offsets_past_32_bits():
    """Rows whose elements pass 2^32: the last rows are those of a small call."""
    cols, rows = 16384, 270000
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free memory")
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    last = rows_of(7, cols, torch.bfloat16, 8).cuda()
    x[-7:] = last
    q, s = ep.ep_quantize_blocks(x)
    want_q, want_s = ep.ep_quantize_blocks(last)
    assert torch.equal(q[-7:], want_q) and torch.equal(s[-7:], want_s)
    assert torch.equal(ep.ep_dequantize_blocks(q, s, out=x)[-7:],
                       ep.ep_dequantize_blocks(want_q, want_s))
