"""ep_quantize_rows' codes, bit for bit: rne(v * (127 / max|v|)) with the quotient
and the product each rounded to float32 before the code is.  In bf16 rows
products that lie exactly between two codes are common (2 in 1000)."""
import numpy as np
import pytest
import torch

import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1024, 256), (1024, 512), (4096, 1024), (4096, 1536), (256, 1024),
                                       (256, 2048), (4096, 4096), (128, 4096), (256, 7168), (64, 16384),
                                       (32, 20000)])
def test_codes_are_the_two_step_formula(rows, cols, dtype):
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn((rows, cols), generator=g) * (0.5 + torch.rand((rows, 1), generator=g))).to(dtype)
    q, s = ep.ep_quantize_rows(x.cuda())
    v = x.float().numpy()
    top = np.abs(v).max(1, keepdims=True)
    want = np.rint(v * (np.float32(127) / top))
    assert want.dtype == np.float32
    assert np.array_equal(q.cpu().numpy(), want.astype(np.int8))
    assert np.array_equal(s.cpu().numpy(), (top / np.float32(127))[:, 0])


def test_products_that_round_to_a_tie():
    """1.5 times the rounded 127 / 3 is 63.499998: the nearest float32 is the tie
    63.5, which goes to the even 64; its negative likewise."""
    x = torch.zeros((1, 16))
    x[0, :5] = torch.tensor([3.0, 1.5, -1.5, 0.0118110236, -3.0])
    q, _ = ep.ep_quantize_rows(x.cuda())
    p = x.numpy() * (np.float32(127) / np.float32(3))
    assert np.array_equal(q.cpu().numpy(), np.rint(p).astype(np.int8))
