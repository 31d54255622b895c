"""A row's products do not depend on what else a call holds: codes over the whole range and
scales that are no powers of two, whose sums round differently in another order, compared
bit for bit in float32 between calls of few rows (tiles of 128 channels), of many (256),
of rows that lie together and of rows read through row_src, in both layouts."""
import pytest
import torch

import combine_ep_route_topk_gb300 as ep
from test_gpu_matmul_fp8 import wide_codes

pytestmark = pytest.mark.gpu
F32 = torch.float32
E, NC, KD = 40, 1000, 656  # four tiles of 256 channels an expert, a short last block of K


@pytest.fixture(scope="module")
def parts():
    g = torch.Generator().manual_seed(3)
    kb = ep.scale_blocks(KD)
    w, ws = wide_codes((E, NC, KD), g), (0.5 + torch.rand((E, ep.scale_blocks(NC), kb), generator=g)) / 120
    x, xs = wide_codes((4400, KD), g), (0.5 + torch.rand((4400, kb), generator=g)) / 120
    return tuple(t.cuda() for t in (w, ws, x, xs))


def offsets(counts):
    return torch.tensor([0] + list(counts), dtype=torch.int32).cumsum(0).int().cuda()


def alone(parts, expert, row):
    w, ws, x, xs = parts
    return ep.ep_expert_matmul_fp8(x[row:row + 1], xs[row:row + 1], w[expert:expert + 1],
                                   ws[expert:expert + 1], offsets([1]), out_dtype=F32)[0]


def test_order_matters_to_these_rows(parts):
    """In another order of the blocks of K the same sums round to other bits."""
    w, ws, x, xs = (t[:1] for t in parts)
    n = KD // 128 * 128
    flip = lambda t: t[..., :n].unflatten(-1, (-1, 128)).flip(-2).flatten(-2).contiguous()  # noqa: E731
    k = n // 128
    a = ep.ep_expert_matmul_fp8(x[..., :n].contiguous(), xs[..., :k].contiguous(), w[..., :n].contiguous(),
                                ws[..., :k].contiguous(), offsets([1]), out_dtype=F32)
    b = ep.ep_expert_matmul_fp8(flip(x), xs[..., :k].flip(-1).contiguous(), flip(w),
                                ws[..., :k].flip(-1).contiguous(), offsets([1]), out_dtype=F32)
    assert (a != b).float().mean() > 0.25


@pytest.mark.parametrize("counts", [[2] * E, [33, 0] * (E // 2), [110] * E, [5, 300, 0, 1, 129] * (E // 5)])
def test_rows_are_those_of_a_call_of_their_own(parts, counts):
    w, ws, x, xs = parts
    offs, n = offsets(counts), sum(counts)
    together = ep.ep_expert_matmul_fp8(x[:n], xs[:n], w, ws, offs, out_dtype=F32)
    src = torch.randperm(x.shape[0], generator=torch.Generator().manual_seed(n))[:n].int().cuda()
    anywhere = ep.ep_expert_matmul_fp8(x, xs, w, ws, offs, row_src=src, out_dtype=F32)
    copied = ep.ep_expert_matmul_fp8(x[src.long()], xs[src.long()], w, ws, offs, out_dtype=F32)
    assert torch.equal(anywhere, copied)
    cap = max(counts)
    masked = ep.ep_expert_matmul_fp8(x, xs, w, ws, offs, layout=ep.EP_LAYOUT_MASKED, cap=cap,
                                     row_src=src, out_dtype=F32)
    starts = offs.tolist()
    for e in range(0, E, 3):
        at = slice(starts[e], starts[e + 1])
        assert torch.equal(masked[e * cap:e * cap + counts[e]], anywhere[at])
        for i in {0, counts[e] // 2, counts[e] - 1} if counts[e] else ():
            assert torch.equal(together[starts[e] + i], alone(parts, e, starts[e] + i))
            assert torch.equal(anywhere[starts[e] + i], alone(parts, e, int(src[starts[e] + i])))
