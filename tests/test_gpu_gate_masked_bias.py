"""A bias of -inf or NaN forbids a pick and nothing else: the softmax goes over the
experts whose logit is available.  Weights computed by hand, over a total of 8."""
import math

import pytest
import torch

import combine_ep_route_topk_gb300 as ep

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("groups", [1, 2])
@pytest.mark.parametrize("mask", [-INF, NAN])
def test_softmax_weights_under_a_masked_bias(mask, groups):
    logits = torch.tensor([[0.0, math.log(2.0), math.log(4.0), 0.0]], device="cuda")
    bias = torch.tensor([0.0, 0.0, mask, mask], device="cuda")
    idx, w = ep.ep_gate_topk(logits, 3, ep.EP_SCORE_SOFTMAX, bias=bias, groups=groups, renorm=False)
    assert idx.tolist() == [[1, 0, -1]]
    torch.testing.assert_close(w.cpu(), torch.tensor([[2 / 8, 1 / 8, 0.0]]), rtol=1e-6, atol=0)
    _, w = ep.ep_gate_topk(logits, 3, ep.EP_SCORE_SOFTMAX, bias=bias, groups=groups, renorm=True)
    torch.testing.assert_close(w.cpu(), torch.tensor([[2 / 3, 1 / 3, 0.0]]), rtol=1e-6, atol=0)


@pytest.mark.parametrize("mask", [-INF, NAN])
def test_softmax_weights_under_masked_logits(mask):
    logits = torch.tensor([[0.0, math.log(2.0), mask, 0.0, mask]], device="cuda")
    idx, w = ep.ep_gate_topk(logits, 2, ep.EP_SCORE_SOFTMAX, bias=torch.zeros(5, device="cuda"), renorm=False)
    assert idx.tolist() == [[1, 0]]
    torch.testing.assert_close(w.cpu(), torch.tensor([[2 / 4, 1 / 4]]), rtol=1e-6, atol=0)
