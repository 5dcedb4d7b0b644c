"""gmm_fwd_act (product with bias, activation and residual in its epilogue)
and gmm_act_bwd against the formulas in 64 bits.

Bounds.  The product carries the library's 2e-3 * A; an activation passes an
error of z on times its largest slope (L); SwiGLU as swiglu_bound.  fp32
evaluation of an activation: 1e-5 of the value plus 1e-6 of |z| (erfc and exp
are within a few ulp; z sigmoid(z) keeps their relative error).  bf16 results
add 2^-8 of themselves.
"""
import math

import numpy as np
import pytest
import torch

import moe_fp8_grouped_b200 as gm
import oracle
from parity import TOL, assert_within, check_guards, guarded, swiglu_bound

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"]
SLOPE = {"none": 1.0, "relu": 1.0, "silu": oracle.SILU_LIPSCHITZ, "gelu": 1.13, "gelu_tanh": 1.13}
C = math.sqrt(2.0 / math.pi)


def act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))  # slope 0 at 0
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * C * (z + 0.044715 * z ** 3))
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        return g * torch.sigmoid(g) * u
    return z


def torch_quantize(x):
    """The dynamic rule of gmm_fwd_act in torch: codes [M, K], scales [K/128, M]."""
    b = x.float().view(x.shape[0], -1, 128)
    s = b.abs().amax(2, keepdim=True) / 448.0  # torch: times fl32(1/448)
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    q = (b * inv).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape)
    return q, s[:, :, 0].t().contiguous()


def _product(lhs, w, sizes, rule, trans, s):
    """rhs operands on the GPU, z64 and A of the product (rows outside groups 0)."""
    M, K = lhs.shape
    G, _, N = w.shape
    if rule == "none":
        rhs, sc = (w.transpose(1, 2).contiguous() if trans else w), None
        a, wd = lhs.double(), w.double()
    else:
        rhs, sc = gm.gmm_quantize_rhs(w, transpose_out=trans)
        c, _ = gm.gmm_quantize_rhs(w)
        wd = c.view(torch.float8_e4m3fn).double() * sc.double()[:, None, :]
        q, bs = torch_quantize(lhs) if rule == "dynamic" else (*gm.gmm_quantize(lhs, rule, axis=1, static_scale=s)[:1], s)
        a = q.view(torch.float8_e4m3fn).double()
        a = a * s.double() if rule == "static" else (a.view(M, K // 128, 128) * bs.t().double()[:, :, None]).view(M, K)
    z = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    ab = torch.zeros_like(z)
    r = 0
    for g, n in enumerate(sizes):
        z[r:r + n] = a[r:r + n] @ wd[g]
        ab[r:r + n] = a[r:r + n].abs() @ wd[g].abs()
        r += n
    return rhs, sc, z, ab


def _bias_rows(bias, sizes, M):
    out = torch.zeros(M, bias.shape[1], dtype=torch.float64, device=DEV)
    r = 0
    for g, n in enumerate(sizes):
        out[r:r + n] = bias[g].double()
        r += n
    return out


def _out_bound(z, ab, act, out_dtype, residual):
    if act == "swiglu":
        zc, ac = z.cpu().numpy(), ab.cpu().numpy()
        f = zc.shape[1] // 2
        ref = act64(z, act).cpu().numpy()
        b = swiglu_bound(torch.float32, (zc[:, :f], zc[:, f:], ac[:, :f], ac[:, f:]), ref)
    else:
        ref = act64(z, act).cpu().numpy()
        b = SLOPE[act] * TOL * ab.cpu().numpy() + 1e-5 * np.abs(ref) + 1e-6 * np.abs(z.cpu().numpy())
    if residual is not None:
        ref = ref + residual.double().cpu().numpy()
        b = b + 1e-6 * np.abs(ref)
    if out_dtype == torch.bfloat16:
        b = b + 2.0 ** -8 * np.abs(ref)
    return ref, b


def _case(sizes, M, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    G = len(sizes)
    lhs = torch.randn(M, K, generator=g).bfloat16().to(DEV)
    w = (torch.randn(G, K, N, generator=g) * 0.02).bfloat16().to(DEV)
    bias = (torch.randn(G, N, generator=g) * 0.5).to(DEV)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    s = torch.tensor([4.0 / 448.0], device=DEV)
    return lhs, w, bias, gs, s


def _run(sizes, M, K, N, rule, trans, act, with_bias, res_dtype, keep, out_dtype, seed=0):
    lhs, w, bias, gs, s = _case(sizes, M, K, N, seed)
    rhs, sc, z, ab = _product(lhs, w, sizes, rule, trans, s)
    rows = sum(sizes)
    inside = (torch.arange(M, device=DEV) < rows)[:, None]
    if with_bias:
        z = z + _bias_rows(bias, sizes, M)
    out_n = N // 2 if act == "swiglu" else N
    res = None
    if res_dtype is not None:
        res = torch.randn(M, out_n, generator=torch.Generator().manual_seed(9)).to(res_dtype).to(DEV)
    raw, out, pad, n = guarded((M, out_n), out_dtype)
    zraw, zk, zpad, zn = guarded((M, N), torch.bfloat16)
    got = gm.gmm_fwd_act(lhs, rhs, sc, gs, act=act, bias=bias if with_bias else None, residual=res, rule=rule,
                         static_scale=s if rule == "static" else None, transpose_rhs=trans, out=out,
                         preact=zk if keep else None)
    torch.cuda.synchronize()
    assert isinstance(got, tuple) == keep
    ref, b = _out_bound(z, ab, act, out_dtype, torch.where(inside, res.double(), 0.0) if res is not None else None)
    assert_within(out, ref, b, f"{act} {rule} trans={trans}")
    assert bool((out[rows:] == 0).all())
    check_guards(raw, pad, n)
    if keep:
        zr = z.cpu().numpy()
        assert_within(zk, zr, TOL * ab.cpu().numpy() + (2.0 ** -8 + 1e-6) * np.abs(zr), "z")
        assert bool((zk[rows:] == 0).all())
    check_guards(zraw, zpad, zn)


SIZES = {"one": ([1], 1), "dense": ([300], 300), "ragged": ([5, 0, 129, 64, 0, 257], 455), "tail": ([70, 0, 31], 140),
         "none": ([0, 0], 65)}


@pytest.mark.parametrize("which", list(SIZES))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rule", ["static", "dynamic", "none"])
@pytest.mark.parametrize("trans", [False, True])
def test_fwd(which, act, rule, trans):
    sizes, M = SIZES[which]
    N = 768 if act == "swiglu" else 640
    _run(sizes, M, 384, N, rule, trans, act, True, torch.bfloat16, True, torch.bfloat16, seed=M)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("res_dtype", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
def test_fwd_parts(with_bias, res_dtype, keep, act):
    _run([100, 3, 0, 260], 400, 256, 512, "static", False, act, with_bias, res_dtype, keep, torch.float32)


@pytest.mark.parametrize("tiles", ["one_cta", "cta_pairs", "cta_pairs_narrow"])
@pytest.mark.parametrize("rule", ["static", "dynamic", "none"])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("trans", [False, True])
def test_fwd_every_tile(tiles, rule, act, trans):
    gm.gmm_set_tiles(tiles)
    try:
        _run([40, 700, 0, 129], 900, 512, 768, rule, trans, act, True, torch.bfloat16, True, torch.bfloat16)
    finally:
        gm.gmm_set_tiles("auto")


def test_plain_epilogue_equals_gmm_fwd():
    """No bias, no activation, no residual: the bits of gmm_fwd; with SwiGLU
    gmm_fwd_swiglu up to the evaluation of silu (1e-5 of the value each, so
    that a bf16 result differs by one step at most: 2^-7 of itself)."""
    lhs, w, _, gs, s = _case([200, 0, 56], 300, 384, 512, 3)
    codes, sc = gm.gmm_quantize_rhs(w)
    for rule in ("static", "dynamic"):
        kw = dict(rule=rule, static_scale=s if rule == "static" else None)
        if rule == "dynamic":  # the same codes for both (the scales' one ulp aside)
            lhs, kw["lhs_scales"] = gm.gmm_quantize(lhs, "dynamic", axis=1)
        assert torch.equal(gm.gmm_fwd_act(lhs, codes, sc, gs, **kw), gm.gmm_fwd(lhs, codes, sc, gs, **kw))
        a = gm.gmm_fwd_act(lhs, codes, sc, gs, act="swiglu", **kw).double()
        b = gm.gmm_fwd_swiglu(lhs, codes, sc, gs, **kw).double()
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs()).all())


def test_block_scaled_weights_and_quantized_lhs():
    sizes, M, K, N = [130, 20], 160, 384, 512
    lhs, w, bias, gs, s = _case(sizes, M, K, N, 4)
    codes, bs = gm.gmm_quantize_rhs_blocks(w, axis=0)
    for rule in ("static", "dynamic"):
        kw = dict(rule=rule, static_scale=s if rule == "static" else None)
        x = lhs
        if rule == "dynamic":
            x, kw["lhs_scales"] = gm.gmm_quantize(lhs, "dynamic", axis=1)
        z, ab0 = gm.gmm_fwd(x, codes, bs, gs, out_dtype=torch.float32, **kw).double(), None
        y = gm.gmm_fwd_act(x, codes, bs, gs, act="silu", bias=bias, out_dtype=torch.float32, **kw)
        ref = act64(z + _bias_rows(bias, sizes, M), "silu")
        ref[150:] = 0
        assert_within(y, ref.cpu().numpy(), (1e-5 * ref.abs() + 1e-6 * (z.abs() + 1)).cpu().numpy(), rule)
        assert ab0 is None
    q, qs = torch_quantize(lhs)  # bit for bit what the call makes of lhs
    c2, s2 = gm.gmm_quantize_rhs(w)
    a = gm.gmm_fwd_act(q, c2, s2, gs, act="gelu", bias=bias, rule="dynamic", lhs_scales=qs)
    assert torch.equal(a, gm.gmm_fwd_act(lhs, c2, s2, gs, act="gelu", bias=bias, rule="dynamic"))


def test_residual_may_be_the_output():
    lhs, w, bias, gs, s = _case([60, 200], 260, 256, 384, 5)
    codes, sc = gm.gmm_quantize_rhs(w)
    res = torch.randn(260, 384, device=DEV).bfloat16()
    want = gm.gmm_fwd_act(lhs, codes, sc, gs, act="relu", bias=bias, residual=res, static_scale=s)
    buf = res.clone()
    got = gm.gmm_fwd_act(lhs, codes, sc, gs, act="relu", bias=bias, residual=buf, static_scale=s, out=buf)
    assert got.data_ptr() == buf.data_ptr() and torch.equal(got, want)


def _bwd_ref(z, dout, sizes, act):
    zd = z.double().requires_grad_(True)
    rows = sum(sizes)
    dz, = torch.autograd.grad((act64(zd, act) * dout.double()).sum(), zd)
    dz[rows:] = 0
    mag = dout.double().abs() if act != "swiglu" else torch.cat([dout.double().abs()] * 2, 1) * \
        torch.cat([zd.detach().chunk(2, 1)[1].abs(), zd.detach().chunk(2, 1)[0].abs()], 1)
    db, dm = [], []
    r = 0
    for n in sizes:
        db.append(dz[r:r + n].sum(0))
        dm.append(mag[r:r + n].sum(0))
        r += n
    return dz, mag, torch.stack(db), torch.stack(dm)


@pytest.mark.parametrize("sizes,M,N", [([1], 1, 256), ([300], 300, 256), ([5, 0, 129, 64, 0, 257], 455, 768),
                                       ([70, 0, 31], 140, 512), ([0, 0], 65, 256), ([0] * 600 + [3], 200, 256),
                                       ([1] * 100, 100, 256)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("with_dbias", [False, True])
def test_bwd(sizes, M, N, act, with_dbias):
    g = torch.Generator().manual_seed(M)
    z = (torch.randn(M, N, generator=g) * 2).bfloat16().to(DEV)
    z[0, 0], z[-1, -1] = 40.0, -40.0
    if act == "relu":
        z[0, 1] = 0.0  # slope 0 at 0
    dout = torch.randn(M, N // 2 if act == "swiglu" else N, generator=g).bfloat16().to(DEV)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    raw, dz, pad, n = guarded((M, N), torch.bfloat16)
    braw, db, bpad, bn = guarded((len(sizes), N), torch.float32)
    a, b = gm.gmm_act_bwd(dout, z, gs, act=act, with_dbias=with_dbias, dz=dz, dbias=db if with_dbias else None)
    torch.cuda.synchronize()
    rz, mag, rb, bm = _bwd_ref(z, dout, sizes, act)
    # fp32 slopes: within 2e-6 of the factors' magnitudes (slopes are below 1.13)
    assert_within(dz, rz.cpu().numpy(), (2.0 ** -8 * rz.abs() + 2e-6 * mag).cpu().numpy(), act)
    if with_dbias:
        # 2e-6 a term, and an fp32 chain of at most 16 + 8 + 8 terms' roundings
        assert_within(db, rb.cpu().numpy(), ((2e-6 + 32 * 2.0 ** -24) * bm + 1e-30).cpu().numpy(), "dbias")
        check_guards(braw, bpad, bn)
    else:
        assert b is None
    assert bool((dz[sum(sizes):] == 0).all())
    check_guards(raw, pad, n)


@pytest.mark.parametrize("act", ACTS)
def test_bwd_against_differences(act):
    """Central differences of the fp64 formula at bf16 z: checks the slopes
    themselves.  h = 2^-10: the cube term is h^2 / 6 * 4 < 1e-6, fp64 rounding
    far below, the kernel's bf16 result 2^-8 of itself."""
    M, N, h = 8, 256, 2.0 ** -10
    g = torch.Generator().manual_seed(1)
    z = (torch.randn(M, N, generator=g) * 2).bfloat16().to(DEV)
    z[z.abs() < 2 * h] = 0.25  # relu's corner
    dout = torch.randn(M, N // 2 if act == "swiglu" else N, generator=g).bfloat16().to(DEV)
    gs = torch.tensor([M], dtype=torch.int32, device=DEV)
    dz, _ = gm.gmm_act_bwd(dout, z, gs, act=act)
    zd, d = z.double(), dout.double()
    f = N // 2
    num = torch.empty_like(zd)
    for part in (slice(0, f), slice(f, N)):
        a, b = zd.clone(), zd.clone()
        a[:, part] += h
        b[:, part] -= h
        diff = (act64(a, act) - act64(b, act)) / (2 * h) * d
        num[:, part] = diff if act == "swiglu" else diff[:, part]
    scale = d.abs().max() * (1 + zd.abs().max())
    assert bool(((dz.double() - num).abs() <= 2.0 ** -8 * num.abs() + 1e-5 * scale).all())


def test_bwd_extreme_values():
    """Slopes far out are 0 or 1, without NaN from overflowing powers."""
    v = torch.tensor([1e30, -1e30, 3e38, -3e38, 200.0, -200.0, 0.0, -0.0], device=DEV).bfloat16()
    z = v.repeat(16).view(1, 128).contiguous()
    dout = torch.ones(1, 128, dtype=torch.bfloat16, device=DEV)
    gs = torch.tensor([1], dtype=torch.int32, device=DEV)
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        dz, _ = gm.gmm_act_bwd(dout, z, gs, act=act)
        mid = 0.0 if act == "relu" else 0.5
        want = torch.tensor([1, 0, 1, 0, 1, 0, mid, mid], device=DEV).repeat(16).view(1, 128)
        assert torch.equal(dz.float(), want), act


def test_bwd_in_place_over_z_and_repeatable():
    g = torch.Generator().manual_seed(2)
    z = torch.randn(500, 512, generator=g).bfloat16().to(DEV)
    dout = torch.randn(500, 256, generator=g).bfloat16().to(DEV)
    gs = torch.tensor([130, 0, 350], dtype=torch.int32, device=DEV)
    dz, db = gm.gmm_act_bwd(dout, z, gs, act="swiglu")
    dz2, db2 = gm.gmm_act_bwd(dout, z, gs, act="swiglu")
    assert torch.equal(dz, dz2) and torch.equal(db, db2)
    buf = z.clone()
    dz3, db3 = gm.gmm_act_bwd(dout, buf, gs, act="swiglu", dz=buf)
    assert dz3.data_ptr() == buf.data_ptr() and torch.equal(dz3, dz) and torch.equal(db3, db)


def test_training_step_runs_together():
    """Forward with kept z, gradient of the epilogue, dlhs and dW, against
    autograd of the same layer in 64 bits (bf16 family).  Errors: z is rounded
    to bf16 before its slope is taken (2^-8 |z| times the second derivative,
    below 1.2 |dout|), dz is rounded to bf16, the products add 2e-3 * A."""
    sizes, M, K, N = [90, 0, 38], 128, 256, 384
    lhs, w, bias, gs, _ = _case(sizes, M, K, N, 6)
    out, z = gm.gmm_fwd_act(lhs, w, None, gs, act="gelu", bias=bias, rule="none", keep_preact=True)
    dout = torch.randn(M, N, device=DEV).bfloat16()
    dz, db = gm.gmm_act_bwd(dout, z, gs, act="gelu")
    dl, dw = gm.gmm_backward(lhs, dz, w, None, gs, rule="none", dlhs_dtype=torch.float32)
    ld, wd, bd = (t.double().requires_grad_(True) for t in (lhs, w, bias))
    parts, r = [], 0
    for g, n in enumerate(sizes):
        parts.append(ld[r:r + n] @ wd[g] + bd[g])
        r += n
    zz = torch.cat(parts)
    gl, gw, gb = torch.autograd.grad((act64(zz, "gelu") * dout.double()).sum(), (ld, wd, bd))
    ab = torch.cat([lhs[a:b].double().abs() @ w[g].double().abs() for g, (a, b) in enumerate([(0, 90), (90, 90), (90, 128)])])
    ddz = dout.double().abs() * (1.2 * (2.0 ** -8 * zz.detach().abs() + TOL * ab) + 1.13 * 2.0 ** -8)
    r = 0
    for g, n in enumerate(sizes):
        rows = slice(r, r + n)
        e = ddz[rows]
        assert bool(((db[g].double() - gb[g]).abs() <= e.sum(0) + 1e-9).all())
        assert bool(((dl[rows].double() - gl[rows]).abs() <=
                     (e + TOL * 1.13 * dout[rows].double().abs()) @ wd[g].detach().abs().t() + 1e-9).all())
        assert bool(((dw[g].double() - gw[g]).abs() <=
                     ld[rows].detach().abs().t() @ (e + TOL * 1.13 * dout[rows].double().abs()) + 1e-9).all())
        r += n


def test_streams_and_graphs():
    lhs, w, bias, gs, s = _case([60, 200], 260, 256, 384, 7)
    codes, sc = gm.gmm_quantize_rhs(w)
    z = torch.randn(260, 384, device=DEV).bfloat16()

    def both():
        return (gm.gmm_fwd_act(lhs, codes, sc, gs, act="silu", bias=bias, static_scale=s), *gm.gmm_act_bwd(lhs.new_ones(260, 384), z, gs, act="silu"))

    want = both()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(both())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_device_errors():
    lhs, w, bias, gs, s = _case([60, 200], 260, 256, 384, 8)
    codes, sc = gm.gmm_quantize_rhs(w)
    ws = torch.empty(gm.gmm_workspace_bytes(0, 260, 256, 384, 2), dtype=torch.uint8, device=DEV)
    gm.gmm_fwd_act(lhs, codes, sc, gs, act="silu", bias=bias, static_scale=s, ws=ws)
    assert gm.gmm_read_device_status(ws) == (0, 0)
    out = gm.gmm_fwd_act(lhs, codes, sc, gs, act="silu", static_scale=torch.zeros_like(s), ws=ws)
    assert gm.gmm_read_device_status(ws) == (4, 2) and bool((out == 0).all())  # an unusable scale
    gm.gmm_fwd_act(lhs, codes, sc, torch.tensor([-1, 200], dtype=torch.int32, device=DEV), static_scale=s, ws=ws)
    assert gm.gmm_read_device_status(ws)[0] == 7
    z = torch.zeros(260, 384, dtype=torch.bfloat16, device=DEV)
    ws2 = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    gm.gmm_act_bwd(z, z, torch.tensor([200, 200], dtype=torch.int32, device=DEV), act="gelu", ws=ws2)
    assert gm.gmm_read_device_status(ws2)[0] == 7  # clamped to the rows there are


def test_bwd_at_the_most_rows():
    """The largest row count that the library takes (ceil(M / 128) + G = 65535),
    rows behind the last group among them."""
    M, N, rows = 65534 * 128, 128, 8_000_001
    z = torch.full((M, N), -1.0, dtype=torch.bfloat16, device=DEV)
    z[::2] = 1.0
    dout = torch.ones(M, N, dtype=torch.bfloat16, device=DEV)
    gs = torch.tensor([rows], dtype=torch.int32, device=DEV)
    dz, db = gm.gmm_act_bwd(dout, z, gs, act="relu")
    assert bool((dz[0:rows:2] == 1).all()) and bool((dz[1:rows:2] == 0).all()) and bool((dz[rows:] == 0).all())
    assert bool((db == 4_000_001).all())  # sums of ones below 2^24 are exact


def test_bwd_many_tiles_in_a_graph():
    """Groups of many tiles, summed by whichever CTA ends last: the same bits
    from every call and every replay, and the empty groups' zeros each time."""
    sizes, M, N = [0, 5000, 0, 0, 129, 128, 0], 5300, 512
    g = torch.Generator().manual_seed(9)
    z = torch.randn(M, N, generator=g).bfloat16().to(DEV)
    dout = torch.randn(M, N, generator=g).bfloat16().to(DEV)
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    dz, db = gm.gmm_act_bwd(dout, z, gs, act="silu")
    _, mag, rb, bm = _bwd_ref(z, dout, sizes, "silu")
    # chains of 16 rows, 8 row threads, 5 tiles of each of 8 sums, those 8
    assert_within(db, rb.cpu().numpy(), ((2e-6 + 40 * 2.0 ** -24) * bm + 1e-30).cpu().numpy(), "dbias")
    out = torch.empty_like(db)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gm.gmm_act_bwd(dout, z, gs, act="silu", dbias=out)
    for _ in range(5):
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(out, db)


def test_wrong_scales_are_refused():
    """Scales of another shape than the codes' would be read out of bounds."""
    lhs, w, bias, gs, s = _case([60, 200], 260, 256, 384, 8)
    codes, sc = gm.gmm_quantize_rhs(w)
    with pytest.raises(ValueError, match="rhs_scales has shape"):
        gm.gmm_fwd_act(lhs, codes, sc[:1], gs, static_scale=s)
    with pytest.raises(ValueError, match="rhs_scales has shape"):
        gm.gmm_fwd_act(lhs, codes, sc[None], gs, static_scale=s)
    a, a_sc = gm.gmm_quantize(lhs, rule="dynamic", axis=1)
    with pytest.raises(ValueError, match="lhs scale has shape"):
        gm.gmm_fwd_act(a, codes, sc, gs, rule="dynamic", lhs_scales=a_sc[:, :100].contiguous())
    with pytest.raises(ValueError, match="bias has dtype"):
        gm.gmm_fwd_act(lhs, codes, sc, gs, bias=bias.bfloat16(), static_scale=s)
    with pytest.raises(ValueError, match="must be contiguous"):
        gm.gmm_fwd_act(lhs.t().contiguous().t(), codes, sc, gs, static_scale=s)
    with pytest.raises(ValueError, match="all must be on one device"):
        gm.gmm_fwd_act(lhs, codes, sc, gs.cpu(), static_scale=s)


@pytest.mark.parametrize("rule", ["static", "dynamic", "none"])
def test_offsets_beyond_31_bits(rule):
    """More than 2^31 values in out, z, residual and their gradients: the rows
    at the end have the bits of a call with those rows alone."""
    M, K, N, sizes = 1 << 18, 128, 8448, [100_000, 0, 160_000]
    g = torch.Generator(device=DEV).manual_seed(4)
    lhs = torch.randn(M, K, generator=g, device=DEV).bfloat16()
    w = (torch.randn(3, K, N, generator=g, device=DEV) * 0.1).bfloat16()
    bias = torch.randn(3, N, generator=g, device=DEV)
    res = torch.empty(M, N, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    rhs, sc = (w, None) if rule == "none" else gm.gmm_quantize_rhs(w)
    s = torch.tensor([4.0 / 448.0], device=DEV) if rule == "static" else None
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    out, z = gm.gmm_fwd_act(lhs, rhs, sc, gs, act="gelu", bias=bias, residual=res, rule=rule, static_scale=s,
                            keep_preact=True)
    dz, _ = gm.gmm_act_bwd(res, z, gs, act="gelu")
    for grp, a, b in ((0, 0, 300), (2, 259_700, 260_000)):
        one = torch.tensor([b - a], dtype=torch.int32, device=DEV)
        o2, z2 = gm.gmm_fwd_act(lhs[a:b], rhs[grp:grp + 1], sc[grp:grp + 1] if sc is not None else None, one,
                                act="gelu", bias=bias[grp:grp + 1], residual=res[a:b], rule=rule, static_scale=s,
                                keep_preact=True)
        assert torch.equal(out[a:b], o2) and torch.equal(z[a:b], z2)
        assert torch.equal(dz[a:b], gm.gmm_act_bwd(res[a:b], z2, one, act="gelu", with_dbias=False)[0])
    assert not bool(out[260_000:].any()) and not bool(z[260_000:].any()) and not bool(dz[260_000:].any())
