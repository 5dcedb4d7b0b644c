"""The router (gmm_router_topk), its gradient and the combine's weight
gradient against their formulas in 64 bits.

Bounds.  Choices are compared exactly.  A weight is a few fp32 operations on
exp: expf is within 2 ulp, the sum of E <= 1024 positive terms within
(log2 E + 4) ulp (warp tree over per-lane sums), the division and the scale 1
ulp each; an exponent x - m is rounded once, which costs |x - m| ulp.  With
|x - m| <= 30 that stays below 64 ulp = 64 * 2^-23; a bf16 gradient adds
2^-8 of itself.  Products of these formulas with dweights sum k or E terms, so
their bound is 64 * 2^-23 of the terms' magnitudes times 4, and 2^-49 of a
row's magnitudes for the rounding of the 64-bit reference itself.
"""
import math

import pytest
import torch

import moe_fp8_grouped_b200 as gm
from parity import check_guards, guarded  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ULP = 2.0 ** -23


def _scores(x, score):
    x = x.double()
    if score == "sigmoid":
        return torch.sigmoid(x)
    m = x.amax(1, keepdim=True)
    e = torch.where(torch.isinf(x) & (x < 0), torch.zeros_like(x), torch.exp(x - m))
    return e / e.sum(1, keepdim=True)


def _ref(x, k, score, bias, normalize, scale):
    """ids and weights of the definition, one token at a time."""
    p = _scores(x, score).cpu()
    xd = x.double().cpu()
    key = xd if bias is None else p + bias.double().cpu()
    ids = torch.full((x.shape[0], k), -1, dtype=torch.int32)
    w = torch.zeros(x.shape[0], k, dtype=torch.float64)
    for t in range(x.shape[0]):
        order = sorted((e for e in range(x.shape[1]) if xd[t, e] != -math.inf and key[t, e] != -math.inf),
                       key=lambda e: (-float(key[t, e]), e))[:k]
        for j, e in enumerate(order):
            ids[t, j] = e
            w[t, j] = p[t, e]
        if normalize and order:
            l = torch.nn.functional.logsigmoid(xd[t, order]) if score == "sigmoid" else xd[t, order]
            w[t, :len(order)] = torch.softmax(l, 0)
    return ids, w * scale


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 31, 31), (5, 33, 4), (130, 64, 6), (257, 256, 8),
                                   (9, 511, 32), (4, 1024, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
def test_topk(T, E, k, score, normalize, dtype, with_bias):
    g = torch.Generator().manual_seed(T * 7 + E)
    x = (torch.randn(T, E, generator=g) * 2).to(dtype).to(DEV)
    bias = (torch.randn(E, generator=g) * 0.1).to(DEV) if with_bias else None
    ids, w = gm.gmm_router_topk(x, k, score=score, select_bias=bias, normalize=normalize, scale=2.5)
    rid, rw = _ref(x, k, score, bias, normalize, 2.5)
    assert torch.equal(ids.cpu(), rid)
    err = (w.double().cpu() - rw).abs()
    assert bool((err <= 64 * ULP * rw.abs() + 1e-40).all()), float((err / rw.abs().clamp(min=1e-30)).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masks_ties_and_signed_zero(score, with_bias):
    inf = math.inf
    low = torch.finfo(torch.float32).min
    x = torch.tensor([[0.5, 0.5, 0.5, 0.5, 0.5],       # all tied: lowest indices
                      [-inf, 1.0, -inf, 2.0, -inf],    # fewer left than k
                      [-inf] * 5,                      # none left
                      [low, low, 1.0, low, low],       # masked by the type's lowest value: still a choice
                      [0.0, -0.0, -1.0, 0.0, -0.0],    # zeros of either sign tie
                      [3.0, -inf, 3.0, 2.0, 3.0]], device=DEV)
    bias = torch.zeros(5, device=DEV) if with_bias else None
    ids, w = gm.gmm_router_topk(x, 3, score=score, select_bias=bias)
    want = [[0, 1, 2], [3, 1, -1], [-1, -1, -1], [2, 0, 1], [0, 1, 3], [0, 2, 4]]
    assert ids.tolist() == want
    assert w[1, 2] == 0 and bool((w[2] == 0).all()) and not bool(torch.isnan(w).any())
    _, rw = _ref(x, 3, score, bias, False, 1.0)
    assert bool(((w.double().cpu() - rw).abs() <= 64 * ULP * rw.abs() + 1e-40).all())
    if with_bias:  # a bias of -inf masks an expert for every token
        bias[0] = -inf
        ids, _ = gm.gmm_router_topk(x, 3, score=score, select_bias=bias)
        assert ids.tolist()[0] == [1, 2, 3] and 0 not in ids.flatten().tolist()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties_are_decided_exactly(score):
    """Experts 0 and 1 get the same bias and logits that are equal (odd tokens)
    or one fp32 step apart (even tokens), so that fp32 cannot tell their keys
    p + bias apart."""
    g = torch.Generator().manual_seed(0)
    T, E, k = 64, 16, 4
    x = torch.randn(T, E, generator=g).double()
    x32 = x.float().to(DEV)
    bias = torch.zeros(E)
    bias[0], bias[1] = 0.5, 0.5
    x32[:, 1] = x32[:, 0]
    x32[::2, 1] = torch.nextafter(x32[::2, 0], torch.full_like(x32[::2, 0], 100.0))
    ids, _ = gm.gmm_router_topk(x32, k, score=score, select_bias=bias.to(DEV))
    rid, _ = _ref(x32, k, score, bias, False, 1.0)
    assert torch.equal(ids.cpu(), rid)
    for t, row in enumerate(ids.tolist()):  # the larger logit first; exactly tied: the lower index
        at0, at1 = (row.index(e) if e in row else k for e in (0, 1))
        assert at1 < at0 or at0 == at1 == k if t % 2 == 0 else at0 < at1 or at0 == at1 == k


def test_nan_shows_in_the_weights():
    x = torch.tensor([[1.0, math.nan, 2.0, 0.0], [1.0, 3.0, 2.0, 0.0]], device=DEV)
    for score in ("softmax", "sigmoid"):
        ids, w = gm.gmm_router_topk(x, 2, score=score)
        assert ids.tolist() == [[1, 2], [1, 2]]
        assert bool(torch.isnan(w[0, 0])) and not bool(torch.isnan(w[1]).any())


def test_normalised_weights_where_every_score_underflows():
    x = torch.full((2, 8), -300.0, device=DEV)
    x[:, 3] = -299.0
    _, w = gm.gmm_router_topk(x, 2, score="sigmoid", normalize=True)
    want = torch.softmax(torch.tensor([1.0, 0.0], dtype=torch.float64), 0)
    assert bool(((w.double().cpu() - want).abs() <= 64 * ULP * want).all())


def _grad_ref(x, ids, dw, score, normalize, scale):
    """dlogits by autograd of the formula in 64 bits, and the terms' magnitude."""
    leaf = x.double().clone().requires_grad_(True)
    T, E = x.shape
    valid = (ids >= 0) & (ids < E)
    idx = ids.long().clamp(0, E - 1)
    valid &= torch.gather(x, 1, idx) != -math.inf
    z = torch.where(x == -math.inf, torch.full_like(leaf, -1e4), leaf)  # no slope where masked
    p = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    q = torch.where(valid, torch.gather(p, 1, idx), torch.zeros(1, dtype=torch.float64, device=x.device))
    w = q / q.sum(1, keepdim=True).clamp(min=1e-300) if normalize else q
    d = torch.where(valid, dw.double(), torch.zeros(1, dtype=torch.float64, device=x.device))
    gr, = torch.autograd.grad((w * d).sum() * scale, leaf)
    mag = (w * d).abs().sum(1, keepdim=True) * (p if score == "softmax" and not normalize else 0.0)
    mag = mag.expand(T, E).clone().detach() if torch.is_tensor(mag) else torch.zeros(T, E)
    own = (w * (d.abs() + (w * d).abs().sum(1, keepdim=True))).detach()
    mag = mag.scatter_add(1, idx, own)
    # the reference's own fp64 rounding: where the full softmax's terms cancel
    # (normalised weights of experts not chosen) it leaves up to a few 2^-53 of
    # the row's terms, 2^-49 of them at most; in units of the 256 ulp below
    return gr, scale * (mag + 2.0 ** -49 / (256 * ULP) * mag.sum(1, keepdim=True))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (2, 5, 3), (67, 64, 4), (33, 257, 8), (3, 1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_topk_bwd(T, E, k, score, normalize, dtype):
    g = torch.Generator().manual_seed(E)
    x = (torch.randn(T, E, generator=g) * 2).to(dtype).to(DEV)
    if E > 4:
        x[:, 3] = -math.inf
    ids, _ = gm.gmm_router_topk(x, min(k, E - (E > 4)), score=score, normalize=normalize)
    dw = torch.randn(ids.shape, generator=g).to(DEV)
    dl = gm.gmm_router_topk_bwd(dw, x, ids, score=score, normalize=normalize, scale=2.5)
    ref, mag = _grad_ref(x, ids, dw, score, normalize, 2.5)
    err = (dl.double() - ref).abs()
    tol = 256 * ULP * mag.to(DEV) + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0.0) + 1e-38
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_bwd_skips_missing_choices_and_counts_repeats(score, normalize):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4, 6, generator=g).to(DEV)
    ids = torch.tensor([[0, -1, 2], [7, 6, -5], [1, 1, 4], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    dw = torch.randn(4, 3, generator=g).to(DEV)
    ref, mag = _grad_ref(x, ids, dw, score, normalize, 1.0)
    dw = torch.where((ids >= 0) & (ids < 6), dw, torch.full_like(dw, math.nan))  # must not be read into the sum
    dl = gm.gmm_router_topk_bwd(dw, x, ids, score=score, normalize=normalize)
    assert bool(((dl.double() - ref).abs() <= 256 * ULP * mag.to(DEV) + 1e-38).all())
    assert bool((dl[3] == 0).all()) and bool((dl[1] == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_bwd_against_differences(score, normalize):
    """Central differences of the library's own forward.  A weight is within
    64 ulp of its value (<= 1), so a difference over 2 h with h = 2^-7 is off
    by 64 * 2^-23 / h plus the cube term h^2 / 6 * |w'''| (third derivatives of
    these weights are below 1): 1e-3 + 1e-4 in all, times sum |dw|."""
    g = torch.Generator().manual_seed(8)
    E, k, h = 12, 3, 2.0 ** -7
    x = torch.randn(1, E, generator=g).to(DEV)
    dw = torch.randn(1, k, generator=g).to(DEV)
    ids, _ = gm.gmm_router_topk(x, k, score=score, normalize=normalize)
    dl = gm.gmm_router_topk_bwd(dw, x, ids, score=score, normalize=normalize)

    def loss(xx):
        i2, w2 = gm.gmm_router_topk(xx, k, score=score, normalize=normalize)
        assert sorted(i2[0].tolist()) == sorted(ids[0].tolist())
        by = dict(zip(i2[0].tolist(), w2[0].double().tolist()))
        return sum(float(dw[0, j]) * by[int(ids[0, j])] for j in range(k))

    for e in range(E):
        a, b = x.clone(), x.clone()
        a[0, e] += h
        b[0, e] -= h
        num = (loss(a) - loss(b)) / float(a[0, e].double() - b[0, e].double())
        assert abs(num - float(dl[0, e])) <= 1.1e-3 * float(dw.abs().sum())


@pytest.mark.parametrize("T,k,N,R", [(1, 1, 8, 1), (5, 3, 72, 9), (64, 8, 7168, 512), (3, 9, 1032, 40), (2, 32, 256, 64)])
def test_combine_dweight(T, k, N, R):
    g = torch.Generator().manual_seed(N)
    dy = torch.randn(T, N, generator=g).bfloat16().to(DEV)
    rows = torch.randn(R, N, generator=g).bfloat16().to(DEV)
    slot = torch.randint(0, R, (T, k), generator=g, dtype=torch.int32).to(DEV)  # slots may repeat
    slot[0, 0] = -1
    slot[-1, -1] = R
    dw = gm.gmm_combine_dweight(dy, rows, slot)
    ok = (slot >= 0) & (slot < R)
    terms = dy.double()[:, None, :] * rows.double()[slot.long().clamp(0, R - 1)]
    ref = torch.where(ok, terms.sum(2), torch.zeros(1, dtype=torch.float64, device=DEV))
    # fp32 chain of N / 128 + 16 products a thread, then a tree of 9 levels
    tol = (N / 128 + 26) * 2.0 ** -24 * terms.abs().sum(2)
    assert bool(((dw.double() - ref).abs() <= tol).all())
    assert dw[0, 0] == 0 and dw[-1, -1] == 0
    assert torch.equal(dw, gm.gmm_combine_dweight(dy, rows, slot))


def test_combine_dweight_empty():
    dy = torch.zeros(0, 16, dtype=torch.bfloat16, device=DEV)
    rows = torch.zeros(4, 16, dtype=torch.bfloat16, device=DEV)
    assert gm.gmm_combine_dweight(dy, rows, torch.zeros(0, 2, dtype=torch.int32, device=DEV)).shape == (0, 2)
    out = gm.gmm_combine_dweight(torch.ones(2, 16, dtype=torch.bfloat16, device=DEV), rows[:0],
                                 torch.zeros(2, 2, dtype=torch.int32, device=DEV))
    assert bool((out == 0).all())


def test_the_most_tokens():
    T = 1 << 24
    x = torch.randn(T, 2, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV)
    ids, w = gm.gmm_router_topk(x, 1)
    assert torch.equal(ids[:, 0], (x[:, 1] > x[:, 0]).int())
    p = torch.softmax(x.double(), 1)
    # an exponential (4 ulp) over a sum of two, and a division
    assert bool(((w.double() - p.amax(1, keepdim=True)).abs() <= 1e-6).all())
    dl = gm.gmm_router_topk_bwd(torch.ones_like(w), x, ids)
    ref = p[:, 0] * p[:, 1] * torch.where(ids[:, 0] == 0, 1.0, -1.0)  # d p_max / d x_0
    assert bool(((dl[:, 0].double() - ref).abs() <= 1e-6).all()) and bool(((dl[:, 1].double() + ref).abs() <= 1e-6).all())


def test_combine_dweight_offsets_beyond_31_bits():
    R, N = 300_000, 8192
    g = torch.Generator(device=DEV).manual_seed(6)
    rows = torch.empty(R, N, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    dy = torch.randn(2, N, generator=g, device=DEV).bfloat16()
    slot = torch.tensor([[R - 1, 0], [R - 2, 280_000]], dtype=torch.int32, device=DEV)
    dw = gm.gmm_combine_dweight(dy, rows, slot)
    terms = dy.double()[:, None, :] * rows[slot.long()].double()
    assert bool(((dw.double() - terms.sum(2)).abs() <= (N / 128 + 26) * 2.0 ** -24 * terms.abs().sum(2)).all())
