"""gmm_moe_few (a whole mixture-of-experts layer for a few tokens) against the
formula in 64 bits.

Bound: gate, up and down products carry the library's 2e-3 * A (A the sum of
the magnitudes of the terms), SwiGLU passes the first two on as swiglu_bound
does, h is rounded to bf16 (2^-8 |h|), and the down product sums |W2| times
h's error.  The weighted sum adds its weights' magnitudes, fp32 rounding, and
a bf16 result 2^-8 |y|.
"""
import numpy as np
import pytest
import torch

import moe_fp8_grouped_b200 as gm
import oracle
from moe_fp8_grouped_b200 import _binding as B
from moe_fp8_grouped_b200 import ep
from parity import TOL, assert_within, check_guards, guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _layer(G, K, F, N, kind, trans, seed=0, std=0.02):
    """(w1, s1, w2, s2) on the GPU and the float64 weights they stand for."""
    g = torch.Generator().manual_seed(seed)
    w1 = (torch.randn(G, K, 2 * F, generator=g) * std).bfloat16().to(DEV)
    w2 = (torch.randn(G, F, N, generator=g) * std).bfloat16().to(DEV)
    if kind == "bf16":
        d1, d2 = w1.double(), w2.double()
        if trans:
            w1, w2 = w1.transpose(1, 2).contiguous(), w2.transpose(1, 2).contiguous()
        return (w1, None, w2, None), d1, d2
    c1, s1 = gm.gmm_quantize_rhs(w1, transpose_out=trans)
    c2, s2 = gm.gmm_quantize_rhs(w2, transpose_out=trans)
    dec = lambda c: c.view(torch.float8_e4m3fn).double()  # noqa: E731
    t = (lambda c: c.transpose(1, 2)) if trans else (lambda c: c)
    return (c1, s1, c2, s2), t(dec(c1)) * s1.double()[:, None, :], t(dec(c2)) * s2.double()[:, None, :]


def _ref(x, ids, wts, d1, d2):
    """y and its error bound (without the output's own rounding), float64."""
    T, k = ids.shape
    G, _, F2 = d1.shape
    F = F2 // 2
    y = torch.zeros(T, d2.shape[2], dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(y)
    L = oracle.SILU_LIPSCHITZ
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if not 0 <= e < G:
                continue
            xr = x[t].double()
            h, ab = xr @ d1[e], xr.abs() @ d1[e].abs()
            g, u, ag, au = h[:F], h[F:], ab[:F], ab[F:]
            sg = g * torch.sigmoid(g)
            hh = sg * u
            dh = L * TOL * ag * u.abs() + (sg.abs() + L * TOL * ag) * TOL * au + (1e-5 + 2.0 ** -8) * hh.abs()
            w = float(wts[t, j])
            y[t] += w * (hh @ d2[e])
            bound[t] += abs(w) * (dh @ d2[e].abs() + TOL * (hh.abs() @ d2[e].abs()))
    return y, bound


def _check(out, ref, bound, what):
    b = bound + (2.0 ** -8 * ref.abs() if out.dtype == torch.bfloat16 else 1e-6 * ref.abs())
    assert_within(out, ref.cpu().numpy(), b.cpu().numpy(), what)


def _inputs(T, k, G, K, seed, distinct=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).bfloat16().to(DEV)
    if distinct:
        ids = torch.stack([torch.randperm(G, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    else:
        ids = torch.randint(0, G, (T, k), generator=g, dtype=torch.int32)
    wts = torch.softmax(torch.randn(T, k, generator=g), 1).to(DEV)
    return x, ids.to(DEV), wts


CASES = [  # T, k, G, K, F, N
    (1, 1, 1, 128, 128, 128),     # the smallest call
    (1, 2, 8, 512, 256, 512),
    (2, 2, 3, 384, 128, 640),
    (7, 3, 5, 256, 384, 128),     # fewer units than SMs in the down product
    (8, 4, 4, 640, 256, 384),     # every expert has 8 rows
    (9, 2, 4, 256, 256, 256),     # the 32-row variant
    (33, 2, 2, 384, 256, 256),    # 33 rows an expert: two groups
    (64, 8, 16, 256, 128, 384),
    (128, 8, 9, 128, 256, 128),   # 1024 pairs, up to 128 rows an expert
    (1, 2, 4, 2048, 1024, 1024),  # several partial sums a tile
    (16, 8, 256, 256, 128, 256),  # many experts, most empty
]


@pytest.mark.parametrize("T,k,G,K,F,N", CASES)
@pytest.mark.parametrize("kind,trans", [("e4m3", False), ("e4m3", True), ("bf16", False), ("bf16", True)])
def test_matches_the_formula(T, k, G, K, F, N, kind, trans):
    w, d1, d2 = _layer(G, K, F, N, kind, trans, seed=T + G)
    x, ids, wts = _inputs(T, k, G, K, seed=K + F)
    ref, bound = _ref(x, ids, wts, d1, d2)
    for dt in (torch.float32, torch.bfloat16):
        raw, out, pad, n = guarded((T, N), dt)
        y = gm.gmm_moe_few(x, ids, wts, *w, transpose_rhs=trans, out=out)
        torch.cuda.synchronize()
        assert y.data_ptr() == out.data_ptr()
        _check(out, ref, bound, f"{kind} trans={trans} {dt}")
        check_guards(raw, pad, n)


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_ids_named_twice_and_out_of_range(kind):
    T, k, G, K, F, N = 5, 4, 3, 256, 128, 256
    w, d1, d2 = _layer(G, K, F, N, kind, False)
    x, ids, wts = _inputs(T, k, G, K, seed=3, distinct=False)
    ids[0] = torch.tensor([1, 1, 1, 1])
    ids[1] = torch.tensor([-1, 2, G, 2])
    ids[2] = torch.tensor([-1, -1, -1, -1])  # no expert at all: zeros
    ids[3] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 0])
    y = gm.gmm_moe_few(x, ids, wts, *w, out_dtype=torch.float32)
    ref, bound = _ref(x, ids, wts, d1, d2)
    _check(y, ref, bound, kind)
    assert bool((y[2] == 0).all())


def test_no_token_has_an_expert():
    w, _, _ = _layer(2, 128, 128, 128, "e4m3", False)
    x, ids, wts = _inputs(3, 2, 2, 128, seed=1)
    y = gm.gmm_moe_few(x, torch.full_like(ids, -1), wts, *w)
    assert bool((y == 0).all())


def test_activation_magnitudes():
    """Rows of very different size, outliers within a block, zeros, bf16
    subnormals and the largest values: the E4M3 pair keeps each value to 2^-22
    of its row's largest, below the 2e-3 * A of the bound."""
    T, k, G, K, F, N = 8, 1, 2, 512, 128, 256
    w, d1, d2 = _layer(G, K, F, N, "e4m3", False)
    x, ids, wts = _inputs(T, k, G, K, seed=5)
    x[1] *= 1e-3
    x[2, 7] = 3000.0
    x[3] = 0.0
    x[4] *= 1e-30
    x[5] = 1e-39
    x[6, ::128] = 1e4
    x[7, 128:] = 0.0
    y = gm.gmm_moe_few(x, ids, wts, *w, out_dtype=torch.float32)
    ref, bound = _ref(x, ids, wts, d1, d2)
    _check(y, ref, bound + 1e-30, "magnitudes")
    assert bool((y[3] == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_value_that_is_not_finite_stays_in_its_row(bad):
    T, k, G, K, F, N = 4, 2, 2, 256, 128, 256
    w, d1, d2 = _layer(G, K, F, N, "e4m3", True)
    x, ids, wts = _inputs(T, k, G, K, seed=6)
    x[2, 100] = bad
    y = gm.gmm_moe_few(x, ids, wts, *w, transpose_rhs=True, out_dtype=torch.float32)
    assert bool(torch.isnan(y[2]).all())
    keep = [0, 1, 3]
    ref, bound = _ref(x[keep], ids[keep], wts[keep], d1, d2)
    _check(y[keep], ref, bound, "other rows")


def test_repeated_calls_and_captured_graphs_give_the_same_bits():
    T, k, G, K, F, N = 12, 4, 8, 1024, 512, 768
    w, _, _ = _layer(G, K, F, N, "e4m3", False)
    x, ids, wts = _inputs(T, k, G, K, seed=7)
    first = gm.gmm_moe_few(x, ids, wts, *w)
    for _ in range(5):
        assert torch.equal(gm.gmm_moe_few(x, ids, wts, *w), first)
    outs, graphs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gm.gmm_moe_few(x, ids, wts, *w)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):  # two graphs, neither may share the other's workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gm.gmm_moe_few(x, ids, wts, *w))
        graphs.append(g)
    for o in outs:
        o.zero_()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    # new routing through the same graph
    ids.copy_(ids.flip(0).clone())
    want = gm.gmm_moe_few(x, ids, wts, *w)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)


def test_two_streams_at_once():
    T, k, G, K, F, N = 4, 2, 8, 512, 256, 512
    w, _, _ = _layer(G, K, F, N, "bf16", False)
    ins = [_inputs(T, k, G, K, seed=s) for s in (1, 2)]
    want = [gm.gmm_moe_few(*i, *w) for i in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(gm.gmm_moe_few(*ins[i], *w))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_agrees_with_the_routed_products():
    """The same layer through gmm_router_topk, the grouped products and the
    combine: the bf16 family rounds the same h, so only summation order
    differs."""
    T, k, G, K, F, N = 24, 3, 6, 512, 256, 384
    (w1, _, w2, _), d1, d2 = _layer(G, K, F, N, "bf16", False)
    g = torch.Generator().manual_seed(11)
    x = torch.randn(T, K, generator=g).bfloat16().to(DEV)
    ids, wts = gm.gmm_router_topk(torch.randn(T, G, generator=g).to(DEV), k, normalize=True)
    y = gm.gmm_moe_few(x, ids, wts, w1, None, w2, None, out_dtype=torch.float32)
    rt = ep.route(ids, G, 1)
    gs = rt.counts.to(torch.int32)
    h = gm.gmm_fwd_act(ep.gather_rows(x, rt.order // k), w1, None, gs, act="swiglu", rule="none")
    r = gm.gmm_fwd_act(h, w2, None, gs, rule="none")
    slot = torch.empty_like(rt.order).scatter_(0, rt.order, torch.arange(T * k, device=DEV))
    z = ep.combine_rows(r, slot.view(T, k), wts, torch.float32)
    ref, bound = _ref(x, ids.cpu(), wts, d1, d2)
    _check(y, ref, bound, "few")
    # the combine's rows are rounded to bf16: 2^-8 of each
    rows = 2.0 ** -8 * (wts.double()[:, :, None] * r.double()[slot.view(T, k)].abs()).sum(1)
    _check(z, ref, bound + rows, "grouped")


def test_device_status_is_clean():
    w, _, _ = _layer(4, 256, 128, 256, "e4m3", False)
    x, ids, wts = _inputs(4, 2, 4, 256, seed=2)
    need = B.lib().gmm_moe_few_workspace_bytes(4, 2, 4, 256, 128, 256, B.DT_E4M3)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)  # contents do not matter
    y = gm.gmm_moe_few(x, ids, wts, *w, ws=ws)
    assert gm.gmm_read_device_status(ws) == (0, 0)
    assert torch.equal(y, gm.gmm_moe_few(x, ids, wts, *w))


def test_thousand_experts_and_single_ones():
    T, k, G, K, F, N = 6, 5, 1000, 128, 128, 128
    w, d1, d2 = _layer(G, K, F, N, "e4m3", False)
    x, ids, wts = _inputs(T, k, G, K, seed=4)
    ids[0, 0], ids[1, 0] = 0, G - 1
    y = gm.gmm_moe_few(x, ids, wts, *w, out_dtype=torch.float32)
    ref, bound = _ref(x, ids, wts, d1, d2)
    _check(y, ref, bound, "G = 1000")


@pytest.mark.parametrize("T,k", [(40, 2), (1, 32)])
def test_many_tokens_share_row_maxima_and_one_token_many_choices(T, k):
    G, K, F, N = 3, 1152, 256, 384  # 1152: a row of more than one piece, the last one short
    w, d1, d2 = _layer(G, K, F, N, "e4m3", True)
    x, ids, wts = _inputs(T, k, G, K, seed=8, distinct=False)
    x[0] *= 1e4
    x[-1, -1] = 250.0  # the largest value in the short piece
    y = gm.gmm_moe_few(x, ids, wts, *w, transpose_rhs=True, out_dtype=torch.float32)
    ref, bound = _ref(x, ids, wts, d1, d2)
    _check(y, ref, bound, f"T={T} k={k}")


def test_bf16_weights_take_any_value():
    T, k, G, K, F, N = 3, 1, 2, 256, 128, 128
    w, d1, d2 = _layer(G, K, F, N, "bf16", False)
    x, ids, wts = _inputs(T, k, G, K, seed=9)
    x[0] *= 1e-20
    x[1, 5] = 1e6
    x[2, 9] = float("inf")
    y = gm.gmm_moe_few(x, ids, wts, *w, out_dtype=torch.float32)
    ref, bound = _ref(x[:2], ids[:2], wts[:2], d1, d2)
    _check(y[:2], ref, bound + 1e-30, "bf16")
    assert not bool(torch.isfinite(y[2]).all())


def test_no_tokens():
    w, _, _ = _layer(2, 128, 128, 256, "e4m3", False)
    y = gm.gmm_moe_few(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV),
                       torch.empty(0, 2, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV), *w)
    assert y.shape == (0, 256)


def test_results_do_not_depend_on_the_other_tokens():
    """A token's row is the same whatever else is in the batch, up to the order
    of the sums (which depends on the routing): 2e-3 * A of the bound is far
    above it; tokens that choose no expert change nothing at all."""
    T, k, G, K, F, N = 6, 2, 4, 512, 256, 256
    w, d1, d2 = _layer(G, K, F, N, "e4m3", False)
    x, ids, wts = _inputs(T, k, G, K, seed=10)
    alone = gm.gmm_moe_few(x, ids, wts, *w, out_dtype=torch.float32)
    pad_x = torch.cat([x, torch.randn(2, K, device=DEV).bfloat16()])
    pad_ids = torch.cat([ids, torch.full((2, k), -1, dtype=torch.int32, device=DEV)])
    padded = gm.gmm_moe_few(pad_x, pad_ids, torch.cat([wts, wts[:2]]), *w, out_dtype=torch.float32)
    assert torch.equal(padded[:T], alone) and bool((padded[T:] == 0).all())


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_one_expert_with_every_row(kind):
    T, k, G, K, F, N = 1024, 1, 1, 128, 128, 128
    w, d1, d2 = _layer(G, K, F, N, kind, False)
    x, ids, wts = _inputs(T, k, G, K, seed=12)
    y = gm.gmm_moe_few(x, ids, wts, *w, out_dtype=torch.float32)
    ref, bound = _ref(x, ids, wts, d1, d2)
    _check(y, ref, bound, kind)


def _sparse(C, cols, kind, trans, seed):
    """A weight [1, C, cols] whose columns have 8 entries of +-1 (an entry hit
    twice is their sum), the entries' rows [8, cols] and signs."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows = torch.randint(0, C, (8, cols), generator=g, device=DEV)
    rows[0, ::2], rows[1, 1::2] = C - 1, 0
    sign = torch.randint(0, 2, (8, cols), generator=g, device=DEV).float() * 2 - 1
    w = torch.zeros(C, cols, device=DEV)
    w.index_put_((rows, torch.arange(cols, device=DEV).expand(8, -1)), sign, accumulate=True)
    w = (w.t() if trans else w).contiguous()
    w = w.to(torch.float8_e4m3fn).view(torch.uint8) if kind == "e4m3" else w.bfloat16()
    return w[None], rows, sign.double()


@pytest.mark.parametrize("K,F,N", [(1 << 20, 128, 128), (128, 1 << 19, 128), (128, 128, 1 << 20)])
@pytest.mark.parametrize("kind,trans", [("e4m3", False), ("e4m3", True), ("bf16", False), ("bf16", True)])
def test_largest_sizes(K, F, N, kind, trans):
    """The longest contractions and widest rows, with weights sparse enough that
    every entry shows: x holds integers up to 8, so gate and up are exact; h is
    rounded to bf16 (2^-8) after 1e-5 of SwiGLU, and split for E4M3 weights to
    2^-22 of its row's largest."""
    w1, r1, s1 = _sparse(K, 2 * F, kind, trans, 1)
    w2, r2, s2 = _sparse(F, N, kind, trans, 2)
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-8, 9, (2, K), generator=g).bfloat16().to(DEV)
    ids = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    wts = torch.tensor([[1.0], [-0.5]], device=DEV)
    one = lambda n: torch.ones(1, n, device=DEV) if kind == "e4m3" else None  # noqa: E731
    y = gm.gmm_moe_few(x, ids, wts, w1, one(2 * F), w2, one(N), transpose_rhs=trans, out_dtype=torch.float32)
    for t in range(2):
        z = (x[t].double()[r1] * s1).sum(0)
        h = z[:F] * torch.sigmoid(z[:F]) * z[F:]
        terms = h[r2] * s2
        bound = (2.0 ** -8 + 1e-5) * terms.abs().sum(0) + 8 * 2.0 ** -22 * h.abs().max()
        assert_within(y[t], (wts[t, 0].double() * terms.sum(0)).cpu().numpy(), bound.cpu().numpy(), f"token {t}")
