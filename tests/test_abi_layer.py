"""Host-side refusals of the fused epilogue, few-token layer and router calls:
each returns its status before any CUDA call (no GPU needed), and the Python
wrappers check shapes before they reach the library."""
import ctypes

import pytest
import torch

import moe_fp8_grouped_b200 as gm
from moe_fp8_grouped_b200 import _binding as B

FAKE = 0x100000  # a 16-byte aligned fake device address; never dereferenced
BIG = 1 << 40
INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 5, 9


@pytest.fixture(scope="module")
def L():
    from moe_fp8_grouped_b200 import build
    build.build()
    return B.lib()


def _op(data, dtype, scale, rule):
    return B.Operand(data, dtype, scale, rule)


def test_fwd_act(L):
    lhs, rhs = _op(FAKE, B.DT_BF16, FAKE, B.Q_STATIC), _op(FAKE, B.DT_E4M3, FAKE, B.Q_NONE)

    def call(act=B.ACT_SILU, bias=FAKE, res=FAKE, rdt=B.DT_BF16, pre=FAKE, M=256, K=512, N=512, G=8, epi=True, ws=FAKE,
             nbytes=BIG, out=FAKE):
        e = B.Epilogue(act, bias, res, rdt, pre)
        return L.gmm_fwd_act(lhs, rhs, 0, FAKE, G, M, K, N, ctypes.byref(e) if epi else None, out, B.DT_BF16, ws,
                             nbytes, None)

    assert call(epi=False) == INVALID
    assert call(act=6) == INVALID and call(act=-1) == INVALID
    assert call(act=B.ACT_SWIGLU, N=384) == SHAPE
    assert call(N=200) == SHAPE and call(K=500) == SHAPE and call(M=0) == SHAPE
    assert call(rdt=B.DT_E4M3) == INVALID
    assert call(bias=FAKE + 4) == ALIGN and call(res=FAKE + 2) == ALIGN and call(pre=FAKE + 8) == ALIGN
    assert call(G=2000) == UNSUPPORTED
    assert call(out=None) == INVALID
    assert call(nbytes=1024) == WORKSPACE and call(ws=None) == WORKSPACE


def test_act_bwd(L):
    def call(act=B.ACT_SILU, dout=FAKE, z=FAKE, gs=FAKE, dz=FAKE, db=FAKE, M=256, N=512, G=8, ws=FAKE, nbytes=BIG):
        return L.gmm_act_bwd(dout, z, act, gs, G, M, N, dz, db, ws, nbytes, None)

    assert call(act=9) == INVALID
    assert call(dout=None) == INVALID and call(z=None) == INVALID and call(gs=None) == INVALID
    assert call(dz=None) == INVALID
    assert call(N=300) == SHAPE and call(act=B.ACT_SWIGLU, N=384) == SHAPE and call(M=0) == SHAPE
    assert call(z=FAKE + 2) == ALIGN and call(db=FAKE + 4) == ALIGN
    assert call(nbytes=64) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(M=65528 * 128 + 1) == UNSUPPORTED
    assert L.gmm_act_bwd_workspace_bytes(256, 300, 8) == 0
    # one fp32 row of column sums per 128-row tile: at most ceil(M / 128) + G
    assert L.gmm_act_bwd_workspace_bytes(256, 512, 8) >= 4 * 512 * (2 + 8)


def test_moe_few(L):
    def op(dt=B.DT_E4M3, scale=FAKE, rule=B.Q_NONE, data=FAKE):
        return _op(data, dt, scale, rule)

    def call(T=4, k=2, w1=None, w2=None, G=8, K=256, F=128, N=256, x=FAKE, ids=FAKE, wts=FAKE, y=FAKE, ydt=B.DT_BF16,
             ws=FAKE, nbytes=BIG):
        return L.gmm_moe_few(x, ids, wts, T, k, w1 or op(), w2 or op(), 0, G, K, F, N, y, ydt, ws, nbytes, None)

    assert call(T=-1) == SHAPE and call(k=0) == SHAPE and call(G=0) == SHAPE
    assert call(T=0) == 0  # nothing to do
    assert call(K=200) == SHAPE and call(F=64) == SHAPE and call(N=100) == SHAPE
    assert call(T=513, k=2) == UNSUPPORTED and call(T=2 ** 40, k=2 ** 30) == UNSUPPORTED
    assert call(G=1025) == UNSUPPORTED and call(F=(1 << 19) + 128) == UNSUPPORTED
    for name in ("x", "ids", "wts", "y"):
        assert call(**{name: None}) == INVALID
    assert call(w1=op(data=None)) == INVALID
    assert call(ydt=B.DT_E4M3) == INVALID
    assert call(w1=op(dt=B.DT_BF16)) == INVALID  # one type for both
    assert call(w1=op(dt=B.DT_F32), w2=op(dt=B.DT_F32)) == INVALID
    assert call(w2=op(scale=None)) == INVALID
    assert call(w1=op(rule=B.Q_DYNAMIC)) == UNSUPPORTED  # block-wise scales
    assert call(x=FAKE + 2) == ALIGN and call(w1=op(scale=FAKE + 4)) == ALIGN
    need = L.gmm_moe_few_workspace_bytes(4, 2, 8, 256, 128, 256, B.DT_E4M3)
    assert need >= 4 * 2 * 128 * 2 + 4 * 2 * 256 * 4
    assert call(nbytes=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert L.gmm_moe_few_workspace_bytes(4, 2, 8, 256, 100, 256, B.DT_E4M3) == 0
    assert L.gmm_moe_few_workspace_bytes(4, 2, 8, 256, 128, 256, B.DT_F32) == 0


def test_router(L):
    def call(x=FAKE, dt=B.DT_F32, T=4, E=8, k=2, score=B.SCORE_SOFTMAX, bias=None, ids=FAKE, w=FAKE):
        return L.gmm_router_topk(x, dt, T, E, k, score, bias, 0, 1.0, ids, w, None)

    assert call(T=-1) == SHAPE and call(E=0) == SHAPE and call(k=0) == SHAPE and call(k=9) == SHAPE
    assert call(T=0) == 0 and call(T=0, x=None, ids=None, w=None) == 0  # nothing to do
    assert call(E=1025) == UNSUPPORTED and call(E=64, k=33) == UNSUPPORTED and call(T=(1 << 24) + 1) == UNSUPPORTED
    assert call(x=None) == INVALID and call(dt=B.DT_E4M3) == INVALID and call(score=2) == INVALID
    assert call(ids=None) == INVALID and call(w=None) == INVALID
    assert call(x=FAKE + 4) == ALIGN and call(bias=FAKE + 4) == ALIGN

    def bwd(dw=FAKE, x=FAKE, ids=FAKE, dl=FAKE, T=4, E=8, k=2):
        return L.gmm_router_topk_bwd(dw, x, B.DT_BF16, ids, T, E, k, B.SCORE_SIGMOID, 1, 1.0, dl, None)

    assert bwd(T=0) == 0
    assert bwd(k=9) == SHAPE and bwd(dw=None) == INVALID and bwd(ids=None) == INVALID and bwd(dl=None) == INVALID
    assert bwd(dl=FAKE + 2) == ALIGN


def test_combine_dweight(L):
    def call(dy=FAKE, rows=FAKE, nrows=8, slot=FAKE, T=4, k=2, N=64, dw=FAKE):
        return L.gmm_combine_dweight(dy, rows, nrows, slot, T, k, N, dw, None)

    assert call(N=20) == SHAPE and call(N=0) == INVALID and call(T=-1) == INVALID and call(nrows=-1) == INVALID
    assert call(dy=None) == INVALID and call(rows=None) == INVALID and call(dw=None) == INVALID
    assert call(dy=FAKE + 8) == ALIGN
    assert call(T=0) == 0 and call(k=0) == 0  # nothing to do


def test_wrapper_checks():
    z = torch.zeros
    with pytest.raises(ValueError, match="act must be one of"):
        gm.gmm_fwd_act(z(4, 128), z(1, 128, 128), None, z(1), act="tanh")
    with pytest.raises(ValueError, match="bias has shape"):
        gm.gmm_fwd_act(z(4, 128), z(1, 128, 128), None, z(1), bias=z(128))
    with pytest.raises(ValueError, match="residual has shape"):
        gm.gmm_fwd_act(z(4, 128), z(1, 128, 256), None, z(1), act="swiglu", residual=z(4, 256))
    with pytest.raises(ValueError, match="contracts over"):
        gm.gmm_fwd_act(z(4, 128), z(1, 256, 128), None, z(1))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        gm.gmm_fwd_act(z(4, 128).bfloat16(), z(1, 128, 128), None, z(1), rule="none")
    with pytest.raises(ValueError, match="dout has shape"):
        gm.gmm_act_bwd(z(4, 256), z(4, 256), z(1), act="swiglu")
    with pytest.raises(ValueError, match="do not fit together"):
        gm.gmm_moe_few(z(2, 128), z(2, 2), z(2, 2), z(4, 128, 256), None, z(4, 256, 128), None)
    with pytest.raises(ValueError, match="weights has shape"):
        gm.gmm_moe_few(z(2, 128), z(2, 2), z(2, 1), z(4, 128, 256), None, z(4, 128, 128), None)
    with pytest.raises(ValueError, match="select_bias has shape"):
        gm.gmm_router_topk(z(2, 8), 2, select_bias=z(7))
    with pytest.raises(ValueError, match="dweights has shape"):
        gm.gmm_router_topk_bwd(z(2, 3), z(2, 8), z(2, 2))
    with pytest.raises(ValueError, match="dy has shape"):
        gm.gmm_combine_dweight(z(2, 16), z(4, 8), z(2, 2))
