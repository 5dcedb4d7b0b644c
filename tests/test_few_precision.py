"""gmm_moe_few with E4M3 weights uses the bf16 activations in full: rows of 8
significant bits over six binades, multiplied with weights of eight +-1 a
column, so that gate and up are exact sums and the down product adds eight
values of h.

Bound.  x, scaled by a power of two, is hi + lo / 16 exactly (its values are
multiples of 2^-13 of the row's largest), fp32 sums of eight are exact, and
h = bf16(silu(gate) * up) is the reference's unless the fp32 evaluation (within
1e-5 of the value) crosses a rounding boundary, which costs one step, 2^-7 of
the value.  h is split exactly down to 2^-13 of its row's largest and within
2^-21 of that below: scaled, the largest is at least 2^7, and lo, in steps of
2^-9, is off by at most 2^-10, which is 2^-14 of x.  fp32 sums of up to 16
weighted terms: 2^-20 of them.

The CPU test runs the same arithmetic in torch, whole and with the lo codes of
x or of h left out, and shows that the bound tells them apart."""
import pytest
import torch

T, K, G, F, N, TERMS = 6, 512, 3, 256, 384, 8


def _inputs():
    g = torch.Generator().manual_seed(21)
    x = torch.randint(-255, 256, (T, K), generator=g).double() * 2.0 ** -7
    x *= 2.0 ** -torch.randint(0, 6, (T, K), generator=g).double()
    x[:, 0] = 255 * 2.0 ** -7
    assert torch.equal(x.bfloat16().double(), x)

    def sparse(C, cols):
        w = torch.zeros(G, C, cols, dtype=torch.float64)
        for e in range(G):
            for c in range(cols):
                at = torch.randperm(C, generator=g)[:TERMS]
                w[e, at, c] = torch.randint(0, 2, (TERMS,), generator=g).double() * 2 - 1
        return w

    ids = torch.tensor([[0, 1], [2, 0], [1, -1], [2, 2], [0, 2], [1, 0]], dtype=torch.int32)
    wts = torch.tensor([[1.0, -0.5], [0.25, 1.0], [2.0, 1.0], [1.0, 0.5], [-1.0, -1.0], [0.5, 0.5]])
    return x, ids, wts, sparse(K, 2 * F), sparse(F, N)


def _split(v, with_lo=True):
    """The values hi + lo / 16 of a row of bf16 values (or hi alone)."""
    up = 2.0 ** (7 - torch.floor(torch.log2(v.abs().amax(-1, keepdim=True))))
    s = v * up
    hi = s.to(torch.float8_e4m3fn).double()
    lo = ((s - hi) * 16).to(torch.float8_e4m3fn).double() / 16 if with_lo else 0.0
    return (hi + lo) / up


def _layer(x, ids, wts, w1, w2, lo_x=True, lo_h=True, split=False):
    """y, and the bound of the docstring (both float64)."""
    y = torch.zeros(T, N, dtype=torch.float64)
    bound = torch.zeros_like(y)
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0:
                continue
            gu = (_split(x[t], lo_x) if split else x[t]) @ w1[e]
            h = gu[:F] * torch.sigmoid(gu[:F]) * gu[F:]
            hb = h.bfloat16().double()
            crossing = (h * (1 - 1e-5)).bfloat16() != (h * (1 + 1e-5)).bfloat16()
            w = float(wts[t, j])
            y[t] += w * ((_split(hb, lo_h) if split else hb) @ w2[e])
            off = 2.0 ** -7 * h.abs() * crossing + 2.0 ** -20 * h.abs() + 2.0 ** -21 * h.abs().max()
            bound[t] += abs(w) * (off @ w2[e].abs())
    return y, bound


def test_the_bound_holds_for_the_split_and_for_nothing_less():
    a = _inputs()
    y, bound = _layer(*a)
    off = lambda **kw: ((_layer(*a, split=True, **kw)[0] - y).abs() > bound).double().mean()  # noqa: E731
    assert off() == 0
    assert off(lo_x=False) > 0.5 and off(lo_h=False) > 0.5


def test_the_split_of_every_bf16_value():
    """Against row maxima of every exponent (significands 1.0, 1.4375 and the
    largest): exact from 2^-13 of the largest on, within 2^-21 of it below, which
    is reached; rows below 2^-119 keep every value (the power of two stops at
    2^126, where bf16's last place is 2^-7)."""
    v = (torch.arange(0x7f80, dtype=torch.int32) << 16).view(torch.float32).double()
    worst = 0.0
    for bits in [(e << 7) + m for e in range(0xff) for m in (0, 56, 127)][1:]:
        up = 2.0 ** min(134 - (bits >> 7), 126)
        x = v[:bits + 1] * up
        hi = x.to(torch.float8_e4m3fn).double()
        err = (hi + ((x - hi) * 16).to(torch.float8_e4m3fn).double() / 16 - x).abs() / up
        assert not bool(err[v[:bits + 1] >= 2.0 ** -13 * v[bits]].any())
        if bits < 8 << 7:
            assert not bool(err.any())
        else:
            worst = max(worst, float(err.max() / v[bits]))
    assert worst == 2.0 ** -21


@pytest.mark.gpu
@pytest.mark.parametrize("trans", [False, True])
def test_activations_are_used_in_full(trans):
    import moe_fp8_grouped_b200 as gm
    x, ids, wts, w1, w2 = _inputs()
    y, bound = _layer(x, ids, wts, w1, w2)
    dev = "cuda:0"

    def codes(w):
        w = w.transpose(1, 2) if trans else w
        return w.float().contiguous().to(torch.float8_e4m3fn).view(torch.uint8).to(dev)

    got = gm.gmm_moe_few(x.bfloat16().to(dev), ids.to(dev), wts.to(dev), codes(w1), torch.ones(G, 2 * F, device=dev),
                         codes(w2), torch.ones(G, N, device=dev), transpose_rhs=trans, out_dtype=torch.float32)
    err = (got.double().cpu() - y).abs()
    assert bool((err <= bound).all()), f"{int((err > bound).sum())} outside, worst {float((err - bound).max())}"


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,width", [(45, 1024), (46, 1024), (30, 1152), (31, 1152), (15, 65664), (16, 65664)])
def test_row_maxima_on_either_side_of_the_rule(tokens, width):
    """The largest magnitude of a row, found by every CTA or shared: rows whose
    only value other than 0 lies at a different place each, the last one too,
    and of different sizes.  Gate and up are that value, h its SwiGLU rounded to
    bf16 (one step where fp32 crosses a boundary), y that h."""
    import moe_fp8_grouped_b200 as gm
    dev = "cuda:0"
    x = torch.zeros(tokens, width)
    at = torch.arange(tokens) * 997 % width
    at[0] = width - 1
    v = (1 + torch.arange(tokens) % 128 / 128.0) * 2.0 ** (torch.arange(tokens) % 5 - 1)
    x[torch.arange(tokens), at] = v
    one = 0x38  # E4M3 code of 1
    w1 = torch.full((1, width, 256), one, dtype=torch.uint8, device=dev)
    w2 = torch.zeros(1, 128, 128, dtype=torch.uint8, device=dev)
    w2[:, 7] = one
    y = gm.gmm_moe_few(x.bfloat16().to(dev), torch.zeros(tokens, 1, dtype=torch.int32, device=dev),
                       torch.ones(tokens, 1, device=dev), w1, torch.ones(1, 256, device=dev), w2,
                       torch.ones(1, 128, device=dev), out_dtype=torch.float32)
    h = v.double() * torch.sigmoid(v.double()) * v.double()
    lo, hi = (h * (1 - 1e-5)).bfloat16().double(), (h * (1 + 1e-5)).bfloat16().double()
    got = y.double().cpu()
    assert bool(((got == lo[:, None]) | (got == hi[:, None])).all())
