"""The router, the expert-parallel forward on one rank and their gradients run
together, as a training step uses them, against 64-bit autograd of the layer

  w = normalised weights of the chosen experts (softmax scores),
  y[t] = sum_j w[t, j] * (x[t] @ W[e(t, j)])

with x and W the values their E4M3 codes stand for.  dy . h uses rows h rounded
to bf16 (2^-8 |h|) whose product carries 2e-3 * A; the router's gradient passes
an error d of dw on as w (|d| + sum w |d|), plus 256 * 2^-23 of its terms.
"""
import pytest
import torch

import moe_fp8_grouped_b200 as gm
from moe_fp8_grouped_b200 import ep
from parity import TOL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_gradient_through_the_layer(score):
    T, E, k, K, N = 24, 6, 2, 256, 384
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, K, generator=g).bfloat16().to(DEV)
    w = (torch.randn(E, K, N, generator=g) * 0.02).bfloat16().to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    dy = torch.randn(T, N, generator=g).bfloat16().to(DEV)
    s = torch.tensor([4.0 / 448.0], device=DEV)
    xq, _ = gm.gmm_quantize(x, "static", axis=1, static_scale=s)
    codes, scales = gm.gmm_quantize_rhs(w)

    ids, wts = gm.gmm_router_topk(logits, k, score=score, normalize=True)
    y, h, slot = ep.ep_moe_fwd(xq, s, ids, wts, codes, scales, keep_rows=True)
    assert torch.equal(y, ep.ep_moe_fwd(xq, s, ids, wts, codes, scales))
    dw = gm.gmm_combine_dweight(dy, h, slot)
    dl = gm.gmm_router_topk_bwd(dw, logits, ids, score=score, normalize=True)
    dx, dW = ep.ep_moe_bwd(xq, s, ids, wts, dy, codes, scales)
    assert dx.shape == (T, K) and dW.shape == (E, K, N)

    xd = xq.view(torch.float8_e4m3fn).double() * s.double()
    wd = codes.view(torch.float8_e4m3fn).double() * scales.double()[:, None, :]
    leaf = logits.double().requires_grad_(True)
    p = torch.softmax(leaf, 1) if score == "softmax" else torch.sigmoid(leaf)
    q = torch.gather(p, 1, ids.long())
    wt = q / q.sum(1, keepdim=True)
    hd = torch.einsum("tk,tjkn->tjn", xd, wd[ids.long()])
    ab = torch.einsum("tk,tjkn->tjn", xd.abs(), wd[ids.long()].abs())
    dwd = torch.einsum("tn,tjn->tj", dy.double(), hd)
    err = torch.einsum("tn,tjn->tj", dy.double().abs(), TOL * ab + 2.0 ** -8 * hd.abs())
    assert bool(((dw.double() - dwd).abs() <= err + 1e-6 * dwd.abs()).all())
    ref, = torch.autograd.grad((wt * dwd).sum(), leaf)
    wv = wt.detach()
    tol = wv * (err + (wv * err).sum(1, keepdim=True)) + 256 * 2.0 ** -23 * wv * \
        (dwd.abs() + (wv * dwd.abs()).sum(1, keepdim=True))
    full = torch.zeros_like(ref).scatter_add_(1, ids.long(), tol) + 1e-12
    assert bool(((dl.double() - ref).abs() <= full).all())


def test_step_in_a_captured_graph_beside_an_eager_one():
    """Router, layer for few tokens and the router's gradient in one graph,
    replayed while the same calls run eagerly on another stream."""
    T, E, k, K, F, N = 8, 4, 2, 256, 128, 256
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, K, generator=g).bfloat16().to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    w1 = (torch.randn(E, K, 2 * F, generator=g) * 0.05).bfloat16().to(DEV)
    w2 = (torch.randn(E, F, N, generator=g) * 0.05).bfloat16().to(DEV)
    c1, s1 = gm.gmm_quantize_rhs(w1)
    c2, s2 = gm.gmm_quantize_rhs(w2)

    def step():
        ids, wts = gm.gmm_router_topk(logits, k, normalize=True)
        y = gm.gmm_moe_few(x, ids, wts, c1, s1, c2, s2)
        return ids, wts, y, gm.gmm_router_topk_bwd(wts, logits, ids, normalize=True)

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    eager = []
    for _ in range(10):
        graph.replay()
        with torch.cuda.stream(side):
            eager.append(step())
    torch.cuda.synchronize()
    for out in [got, *eager]:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
