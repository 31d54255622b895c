"""ep_rms_norm and its gradient where every block takes several rows in turn, some one more
than others: each row count is no multiple of the rows that the GPU holds at once (some
300 to 10,000).  The bounds are test_gpu_norm's."""
import pytest
import torch

import combine_ep_route_topk_gb300 as ep
import test_gpu_norm as base

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("wdtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(5003, 1040), (1999, 7168), (1201, 8192), (3001, 2880)])
def test_norm_of_several_turns(rows, cols, wdtype):
    base.test_norm_against_plain(rows, cols, BF, wdtype, False)


@pytest.mark.parametrize("outputs", [dict(y=True), dict(y=False, codes=True), dict(y=False, rstd=True)])
@pytest.mark.parametrize("rows,cols", [(5003, 1040), (1999, 7168)])
def test_norm_of_several_turns_one_output(rows, cols, outputs):
    x, w = base.rows_of(rows, cols, BF, 1).cuda(), base.weight_of(cols, F32).cuda()
    every = ep.ep_rms_norm(x, w, out=ep.alloc_norm(rows, cols, BF, "cuda", residual=True, codes=True,
                                                   rstd=True))
    one = ep.ep_rms_norm(x, w, out=ep.alloc_norm(rows, cols, BF, "cuda", **outputs))
    for a, b in zip(one, every):
        assert a is None or torch.equal(a, b)
    assert torch.equal(every.residual, x)
    # y over x: the row behind the one that is written is on its way already
    over = x.clone()
    ep.ep_rms_norm(over, w, out=ep.Norm(over, None, None, None, None))
    assert torch.equal(over, every.y)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(20011, 112), (15001, 256), (9001, 512), (5003, 528),
                                       (1003, 7168), (701, 8208), (333, 16384)])
def test_gradient_of_several_turns(rows, cols, dtype, residual):
    base.test_gradient_against_plain(rows, cols, dtype, F32, residual)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(20011, 112), (9001, 512), (1003, 7168), (333, 16384)])
def test_gradient_of_several_turns_in_place(rows, cols, dtype):
    z, dy, dres = (base.rows_of(rows, cols, dtype, s).cuda() for s in (1, 2, 3))
    w = base.weight_of(cols, F32).cuda()
    rstd = ep.ep_rms_norm(z, w).rstd
    dx, dw = ep.ep_rms_norm_backward(dy, z, w, rstd, dres)
    for i in (0, 1, 4):
        args = [dy, z, w, rstd, dres]
        args[i] = args[i].clone()
        got, dw2 = ep.ep_rms_norm_backward(*args, d_x=args[i])
        assert torch.equal(got, dx) and torch.equal(dw2, dw)
