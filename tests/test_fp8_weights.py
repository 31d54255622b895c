"""pipeline.quantize_expert_weights_fp8 at blocks that its formula alone does not settle
(elementary torch operations, so on the CPU too): the scale is 1 where max / 448 is 0,
and a NaN takes no part in the maximum, as ep_quantize_blocks has it."""
import numpy as np
import torch

import _fp8_ref as ref
from combine_ep_route_topk_gb300 import pipeline as pl


def weights():
    g = torch.Generator().manual_seed(5)
    up = torch.randn((2, 2 * 144, 272), generator=g)
    down = torch.randn((2, 272, 144), generator=g)
    return up, down


def test_blocks_whose_scale_would_be_zero():
    up, down = weights()
    up[0, :128, :128] = 0.0
    up[0, 3, 5] = 2.0 ** -149  # the smallest float32: / 448 it is 0
    w = pl.quantize_expert_weights_fp8(up, down)
    assert float(w.up_scales[0, 0, 0]) == 1.0
    assert (w.up[0, :128, :128] == 0).all()


def test_nan_stays_alone_and_infinity_takes_its_block():
    up, down = weights()
    clean = pl.quantize_expert_weights_fp8(up, down)
    up[1, 2, 3] = float("nan")
    down[0, 200, 140] = float("inf")  # in a short block of K
    w = pl.quantize_expert_weights_fp8(up, down)
    top = up[1, :128, :128].nan_to_num(0.0).abs().max()
    assert float(w.up_scales[1, 0, 0]) == float((top / torch.tensor(448.0)))
    codes = ref.e4m3(w.up.numpy())
    assert np.isnan(codes[1, 2, 3]) and np.isnan(codes).sum() == 1
    moved = w.up != clean.up
    moved[1, :128, :128] = False
    assert not moved.any()
    v = ref.e4m3(w.down.numpy()[0, 128:256, 128:])
    with np.errstate(invalid="ignore"):
        assert np.isnan(v * np.float64(w.down_scales[0, 1, 1])).all()
    assert torch.isinf(w.down_scales).sum() == 1
