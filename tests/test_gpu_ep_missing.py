"""The expert-parallel layer on one rank fed by gmm_router_topk where masks
leave tokens fewer than k experts, or none: the forward, its captured graph and
the backward against the same layer with the missing choices sent to expert 0
with weight 0, and against the formula in 64 bits."""
import math

import pytest
import torch

import moe_fp8_grouped_b200 as gm
from moe_fp8_grouped_b200 import ep
from parity import TOL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, E, k, K, N = 24, 6, 3, 256, 384


def _case():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, K, generator=g).bfloat16().to(DEV)
    w = (torch.randn(E, K, N, generator=g) * 0.02).bfloat16().to(DEV)
    logits = torch.randn(T, E, generator=g)
    logits[3, 1:] = -math.inf   # one expert left
    logits[4, :4] = -math.inf   # two left
    logits[5] = -math.inf       # none
    logits = logits.to(DEV)
    s = torch.tensor([4.0 / 448.0], device=DEV)
    xq, _ = gm.gmm_quantize(x, "static", axis=1, static_scale=s)
    ids, wts = gm.gmm_router_topk(logits, k, normalize=True)
    assert (ids == -1).sum(1).tolist()[3:6] == [2, 1, 3] and int((ids == -1).sum()) == 6
    return xq, s, ids, wts, *gm.gmm_quantize_rhs(w), torch.randn(T, N, generator=g).bfloat16().to(DEV), logits


def _ref(xq, s, ids, wts, codes, scales):
    """h [T, k, N] of the formula and its magnitudes (0 for a missing choice)."""
    xd = xq.view(torch.float8_e4m3fn).double() * s.double()
    wd = codes.view(torch.float8_e4m3fn).double() * scales.double()[:, None, :]
    at = ids.long().clamp(min=0)
    there = (ids >= 0)[:, :, None]
    h = torch.einsum("tk,tjkn->tjn", xd, wd[at]) * there
    return h, torch.einsum("tk,tjkn->tjn", xd.abs(), wd[at].abs()) * there


@pytest.mark.parametrize("junk", [0.0, math.nan])
def test_forward(junk):
    xq, s, ids, wts, codes, scales, dy, _ = _case()
    wts = torch.where(ids < 0, torch.full_like(wts, junk), wts)  # whatever stands there is not used
    y, h, slot = ep.ep_moe_fwd(xq, s, ids, wts, codes, scales, out_dtype=torch.float32, keep_rows=True)
    hd, ab = _ref(xq, s, ids, wts, codes, scales)
    wd = torch.where(ids < 0, torch.zeros_like(wts), wts).double()[:, :, None]
    # products 2e-3 * A, their rows rounded to bf16 (2^-8), fp32 sums
    tol = (wd * (TOL * ab + (2.0 ** -8 + 1e-6) * hd.abs())).sum(1)
    assert bool(((y.double() - (wd * hd).sum(1)).abs() <= tol).all())
    assert not bool(y[5].any())
    assert torch.equal(slot == -1, ids == -1)
    dw = gm.gmm_combine_dweight(dy, h, slot)
    ref = torch.einsum("tn,tjn->tj", dy.double(), hd)
    tol = torch.einsum("tn,tjn->tj", dy.double().abs(), TOL * ab + (2.0 ** -8 + 1e-6) * hd.abs())
    assert bool(((dw.double() - ref).abs() <= tol).all()) and not bool(dw[ids < 0].any())
    assert torch.equal(y, ep.ep_moe_fwd(xq, s, ids, wts, codes, scales, out_dtype=torch.float32, validate=False))


def test_every_choice_missing():
    xq, s, ids, wts, codes, scales, dy, _ = _case()
    ids = torch.full_like(ids, -1)
    assert not bool(ep.ep_moe_fwd(xq, s, ids, wts, codes, scales).any())
    dx, dW = ep.ep_moe_bwd(xq, s, ids, wts, dy, codes, scales)
    assert not bool(dx.any()) and not bool(dW.any())


def test_captured_forward_takes_new_masks():
    xq, s, ids, wts, codes, scales, _, _ = _case()
    graph = ep.EPForwardGraph(xq, s, ids, wts, codes, scales)
    assert torch.equal(graph.replay(), ep.ep_moe_fwd(xq, s, ids, wts, codes, scales))
    ids.copy_(ids.flip(0).clone())
    ids[7, 1] = -1
    wts.copy_(wts.flip(0).clone())
    assert torch.equal(graph.replay(), ep.ep_moe_fwd(xq, s, ids, wts, codes, scales))


def test_backward():
    """Missing choices add nothing: the gradients are bit for bit those of a
    batch in which the tokens' missing choices do not exist (one choice a
    token), and dx of a token without experts is 0."""
    xq, s, ids, wts, codes, scales, dy, logits = _case()
    # one choice a token: the same rows with and without the tokens that have none
    one, w1 = ids[:, :1].contiguous(), wts[:, :1].contiguous()
    dx, dW = ep.ep_moe_bwd(xq, s, one, w1, dy, codes, scales)
    keep = [t for t in range(T) if t != 5]
    dx2, dW2 = ep.ep_moe_bwd(xq[keep], s, one[keep], w1[keep], dy[keep], codes, scales)
    assert torch.equal(dx[keep], dx2) and torch.equal(dW, dW2) and not bool(dx[5].any())
    # all choices: the router's gradient runs through without NaN, masked logits get none
    y, h, slot = ep.ep_moe_fwd(xq, s, ids, wts, codes, scales, keep_rows=True)
    dl = gm.gmm_router_topk_bwd(gm.gmm_combine_dweight(dy, h, slot), logits, ids, normalize=True)
    assert not bool(torch.isnan(dl).any()) and not bool(dl[logits == -math.inf].any())
    dx, _ = ep.ep_moe_bwd(xq, s, ids, wts, dy, codes, scales)
    assert not bool(dx[5].any()) and not bool(torch.isnan(dx).any())


def test_ids_out_of_range_are_still_refused():
    xq, s, ids, wts, codes, scales, dy, _ = _case()
    for bad in (E, -2):
        ids[0, 0] = bad
        with pytest.raises(ValueError, match="out of range"):
            ep.ep_moe_fwd(xq, s, ids, wts, codes, scales)
        with pytest.raises(ValueError, match="out of range"):
            ep.ep_moe_bwd(xq, s, ids, wts, dy, codes, scales)
