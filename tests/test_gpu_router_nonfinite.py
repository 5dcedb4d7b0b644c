"""gmm_router_topk_bwd where a logit is not finite: a softmax over a row with a
NaN or +inf has no value, so every gradient of the row that it reaches is NaN,
as autograd of the formula gives; other rows are untouched."""
import math

import pytest
import torch

import moe_fp8_grouped_b200 as gm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("E,dtype", [(6, torch.float32), (70, torch.bfloat16)])
def test_softmax_gradient_is_nan_in_the_whole_row(bad, E, dtype):
    x = torch.randn(3, E, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    ids = torch.tensor([[0, 2], [1, 3], [4, 5]], dtype=torch.int32, device=DEV)  # not the bad one
    dw = torch.tensor([[0.5, -1.0], [2.0, 1.0], [0.25, 3.0]], device=DEV)
    clean = gm.gmm_router_topk_bwd(dw, x, ids)
    x[1, 0] = bad
    dl = gm.gmm_router_topk_bwd(dw, x, ids)
    leaf = x.double().requires_grad_(True)
    ref, = torch.autograd.grad((torch.softmax(leaf, 1).gather(1, ids.long()) * dw.double()).sum(), leaf)
    assert bool(torch.isnan(ref[1]).all())
    assert bool(torch.isnan(dl[1]).all())
    assert torch.equal(dl[0], clean[0]) and torch.equal(dl[2], clean[2])


def test_a_row_with_every_expert_masked_has_no_gradient():
    x = torch.full((1, 5), -math.inf, device=DEV)
    dl = gm.gmm_router_topk_bwd(torch.ones(1, 2, device=DEV), x,
                                torch.tensor([[0, 1]], dtype=torch.int32, device=DEV))
    assert not bool(torch.isnan(dl).any()) and not bool(dl.any())
