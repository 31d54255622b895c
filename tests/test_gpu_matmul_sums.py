"""The sums of ep_expert_matmul, float32 out and scales of 1, against integers.

Exact while partial sums stay below 2^24.  Codes drawn evenly from -128 .. 127
have products of standard deviation 5461, so sums of 65536 of them stay within
1.4e6 (sigma), a twelfth of 2^24: they are required bit for bit, at every length.
Codes of one sign pass 2^24 from Kd = 1040 on.  The kernel for few rows adds
integers: one rounding, to the output.  The tensor cores add 16 products at a time
to a float32, and an addition may lose up to 2^-23 of the sum so far; with P_b the
sum through block b of 128 K, whose 8 additions come in any order, that is at most
8 * 2^-23 * sum_b |P_b|, for codes of one sign."""
import numpy as np
import pytest
import torch

import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu
Nc = 200


def product(x, w, row_src=None, cap=0):
    E, rows = w.shape[0], x.shape[0]
    counts = torch.full((E,), rows // E)
    counts[-1] += rows - rows // E * E
    offs = torch.zeros(E + 1, dtype=torch.int32)
    offs[1:] = torch.cumsum(counts, 0)
    out = ep.ep_expert_matmul(x.cuda(), torch.ones(rows, device="cuda"), w.cuda(),
                              torch.ones((E, Nc), device="cuda"), offs.cuda(), out_dtype=torch.float32)
    want = torch.cat([x[offs[e]:offs[e + 1]].cuda().double() @ w[e].cuda().double().T for e in range(E)])
    return out.double(), want


@pytest.mark.parametrize("Kd", [1040, 2048, 7168, 16400, 65536])
@pytest.mark.parametrize("E,rows", [(1, 1), (1, 4), (1, 5), (1, 64), (2, 40), (3, 150), (2, 500), (1, 700), (7, 130)])
def test_sums_of_mixed_signs_are_exact(E, rows, Kd):
    g = torch.Generator().manual_seed(rows + Kd)
    x = torch.randint(-128, 128, (rows, Kd), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (E, Nc, Kd), generator=g, dtype=torch.int8)
    got, want = product(x, w)
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(got, want)


def one_sign(kind, rows, Kd):
    g = torch.Generator().manual_seed(Kd)
    if kind == "largest":
        return torch.full((rows, Kd), 127, dtype=torch.int8), torch.full((1, Nc, Kd), 127, dtype=torch.int8)
    if kind == "lowest":
        return torch.full((rows, Kd), -128, dtype=torch.int8), torch.full((1, Nc, Kd), -128, dtype=torch.int8)
    x = torch.randint(1, 128, (rows, Kd), generator=g, dtype=torch.int8)
    w = torch.randint(1, 128, (1, Nc, Kd), generator=g, dtype=torch.int8)
    return x, -w if kind == "negative" else w


@pytest.mark.parametrize("kind", ["largest", "lowest", "positive", "negative"])
@pytest.mark.parametrize("Kd", [1040, 2048, 7168, 65536])
@pytest.mark.parametrize("rows", [3, 40, 150, 300])
def test_sums_of_one_sign(rows, Kd, kind):
    x, w = one_sign(kind, rows, Kd)
    got, want = product(x, w)
    if rows <= 4:
        assert torch.equal(got, want.float().double())
        return
    # the block sums of every row and channel, added up
    bound = torch.zeros_like(want)
    prefix = torch.zeros_like(want)
    xc, wc = x.cuda().double(), w[0].cuda().double()
    for k in range(0, Kd, 128):
        prefix += xc[:, k:k + 128] @ wc[:, k:k + 128].T
        bound += 8 * 2.0 ** -23 * prefix.abs()
    bound[want.abs() <= 2 ** 24] = 0.0
    assert ((got - want).abs() <= bound).all()
    assert float((bound / want.abs()).max()) <= 1.2 * Kd / 16 / 2 * 2.0 ** -23 + 8 * 2.0 ** -23


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_sums_that_cancel(rows):
    """Partial sums of 5.8e7 that come back to small ones: what is lost is relative
    to the partial sums (each addition past 2^24 loses up to 2^-23 of 5.8e7)."""
    Kd = 7168
    g = torch.Generator().manual_seed(1)
    x = torch.full((rows, Kd), 127, dtype=torch.int8)
    w = torch.full((1, Nc, Kd), 127, dtype=torch.int8)
    w[:, :, Kd // 2:] = -127
    w[0, :, 100] = torch.randint(-127, 127, (Nc,), generator=g, dtype=torch.int8)
    got, want = product(x, w)
    lost = 0.0 if rows <= 4 else Kd / 16 * 2.0 ** -23 * 127 * 127 * Kd / 2
    assert float((got - want).abs().max()) <= lost
