"""SwiGLU and its gradient on float32 rows keep float32's precision for gates far from
zero, where an exponent rounded before the exponential would cost |g| 2^-24.

Roundings, relative, with U = 2^-24: expf 4 U (two last places), 1 + e U, reciprocal 2 U
(one last place), a product U each, the scale's quotient U.  A value: 4 + 1 + 2 + 2 + 1 =
10 U.  The gradient, on its terms' magnitudes: the larger of s and 1 - s takes half of e's
error, 2 + 1 + 2 = 5 U, the smaller 4 + 5 + 1 = 10 U; the multiply-add and three products
add 4: 19 U."""
import numpy as np
import pytest
import torch

import _fp8_ref as ref
import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SWIGLU = ep.EP_ACT_SWIGLU


def n64(t):
    return t.double().cpu().numpy()


def gates(rows, cols, seed):
    """Float32 rows whose gates cover -80 .. 80, where neither silu nor its gradient nears
    the smallest float32, and factors 0.5 .. 2 of either sign."""
    g = torch.Generator().manual_seed(seed)
    gate = (torch.rand((rows, cols), generator=g) * 2 - 1) * 80
    factor = 2.0 ** (torch.rand((rows, cols), generator=g) * 2 - 1)
    return gate, factor * (1 - 2.0 * (torch.rand((rows, cols), generator=g) < 0.5))


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("blocks", [1, 11])
def test_values_of_float32_rows(blocks, keep):
    """One value a block of 128, so that its scale tells it in float32."""
    rows, cols = 500, 128 * blocks
    gate, factor = gates(rows, blocks, blocks)
    x = torch.zeros((rows, 2 * cols))
    at = torch.arange(blocks) * 128 + 16 * torch.arange(blocks) % 128 + 5
    x[:, at], x[:, cols + at] = gate, factor
    kw = {}
    if keep:
        kw = dict(x_q=torch.zeros((rows, 2 * cols), dtype=torch.uint8, device="cuda"),
                  x_scales=torch.zeros((rows, 2 * blocks), device="cuda"))
    _, scales = ep.ep_quantize_blocks(x.cuda(), act=SWIGLU, **kw)
    g = n64(gate)
    want = np.abs(g / (1.0 + np.exp(-g)) * n64(factor)) / 448.0
    assert (np.abs(n64(scales) - want) <= 10 * U * want).all()


@pytest.mark.parametrize("saved", ["rows", "codes"])
@pytest.mark.parametrize("rows,cols", [(40, 1040), (3, 16), (257, 48)])
def test_gradient_of_float32_rows(rows, cols, saved):
    gate, factor = gates(rows, cols, cols)
    x = torch.cat([gate, factor], 1)
    d = gates(rows, cols, cols + 1)[1]
    if saved == "rows":
        v = n64(x)
        got = ep.ep_swiglu_backward(d.cuda(), x.cuda())
    else:
        q, s = ref.quantize32(x)
        # what float32 holds of a code times its scale
        v = n64(torch.from_numpy(ref.e4m3(q.numpy())).float() *
                torch.from_numpy(ref.widen(s.numpy(), 2 * cols)))
        got = ep.ep_swiglu_backward(d.cuda(), q.cuda(), s.cuda())
    want, mag = ref.swiglu_grad(v, n64(d))
    assert (np.abs(n64(got) - want) <= 19 * U * mag).all()


def test_far_gates_end_in_zeros_or_the_factor():
    """Where the sigmoid passes below 2^-126 it is 0 or nearly so, and nothing overflows;
    infinite and NaN gates stay visible."""
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([-3e38, -1000.0, -120.0, 120.0, 1000.0, 3e38, inf, -inf, nan, 0.0])
    x = torch.zeros((10, 256))
    x[:, 0], x[:, 128] = g, 1.0
    _, scales = ep.ep_quantize_blocks(x.cuda(), act=SWIGLU)
    s = scales.cpu()[:, 0]
    assert (s[:3] == 1.0).all()                       # zeros: scale 1
    assert (np.abs(n64(s[3:6]) * 448.0 - n64(g[3:6])) <= 10 * U * n64(g[3:6])).all()
    assert torch.isinf(s[6]) and s[9] == 1.0
    out = ep.ep_dequantize_blocks(*ep.ep_quantize_blocks(x.cuda(), act=SWIGLU), out_dtype=torch.float32)
    assert torch.isnan(out[6]).all() and torch.isnan(out[7, 0]) and torch.isnan(out[8, 0])
    d = torch.ones((10, 128))
    dx = ep.ep_swiglu_backward(d.cuda(), x.cuda()).cpu()
    assert (dx[:3, 0].abs() < 1e-30).all() and (dx[:3, 128].abs() < 1e-30).all()
    assert (dx[3:6, 0] == 1.0).all() and torch.equal(dx[3:6, 128], g[3:6])
    assert torch.isnan(dx[8, 0]) and torch.isnan(dx[8, 128])
    assert dx[9, 0] == 0.5 and dx[9, 128] == 0.0
