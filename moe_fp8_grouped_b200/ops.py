"""Torch-facing binding of the C-ABI in include/gmm_fp8.h, with the same names.

Marshalling only: every step runs in libgmm_fp8.so on the tensors' CUDA
device and on torch's current stream.  torch provides device memory (outputs
and a reusable workspace) and the stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import _binding as B


class GmmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = B.STATUS_NAMES.get(status, str(status))
        text = B.lib().gmm_status_string(status).decode()
        super().__init__(f"{where}: {name} ({text})")


class QRule:
    NONE, STATIC, DYNAMIC = B.Q_NONE, B.Q_STATIC, B.Q_DYNAMIC
    by_name = {"none": B.Q_NONE, "static": B.Q_STATIC, "dynamic": B.Q_DYNAMIC}


class DType:
    BF16, F32, E4M3 = B.DT_BF16, B.DT_F32, B.DT_E4M3


_TORCH_DT = {torch.bfloat16: B.DT_BF16, torch.float32: B.DT_F32, torch.uint8: B.DT_E4M3,
             torch.float8_e4m3fn: B.DT_E4M3}


def _rule(rule) -> int:
    return QRule.by_name[rule] if isinstance(rule, str) else int(rule)


def _check(status: int, where: str):
    if status != B.GMM_OK:
        raise GmmError(status, where)


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t.data_ptr()


_ws_cache: dict = {}


def workspace(nbytes: int, device) -> torch.Tensor:
    """A reusable uint8 workspace on ``device`` of at least ``nbytes``."""
    dev = torch.device(device)
    key = (dev.type, dev.index if dev.index is not None else torch.cuda.current_device())
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 1 << 16), dtype=torch.uint8, device=dev)
        _ws_cache[key] = ws
    return ws


def gmm_workspace_bytes(op: int, M: int, K: int, N: int, G: int) -> int:
    return int(B.lib().gmm_workspace_bytes(op, M, K, N, G))


def gmm_chunk_capacity(rows: int, G: int) -> int:
    return int(B.lib().gmm_chunk_capacity(rows, G))


def gmm_status_string(status: int) -> str:
    return B.lib().gmm_status_string(status).decode()


def last_launch_count() -> int:
    return int(B.lib().gmm_last_launch_count())


def gmm_quantize_rhs(w: torch.Tensor, transpose_out: bool = False):
    """W [G, K, N] bf16 -> (codes uint8 [G, K, N] or [G, N, K], scales fp32 [G, N])."""
    G, K, N = w.shape
    codes = torch.empty((G, N, K) if transpose_out else (G, K, N), dtype=torch.uint8, device=w.device)
    scales = torch.empty((G, N), dtype=torch.float32, device=w.device)
    st = B.lib().gmm_quantize_rhs(_dev(w, "w", torch.bfloat16), G, K, N, int(transpose_out), codes.data_ptr(),
                                  scales.data_ptr(), _stream(w))
    _check(st, "gmm_quantize_rhs")
    return codes, scales


def gmm_quantize(x: torch.Tensor, rule="dynamic", axis: int = 1, static_scale: torch.Tensor | None = None,
                 group_sizes: torch.Tensor | None = None, col_scale: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None):
    """Quantize x [rows, cols] bf16; see gmm_quantize in include/gmm_fp8.h for
    the layouts.  Returns (codes, scales)."""
    rows, cols = x.shape
    G = int(group_sizes.numel()) if group_sizes is not None else 1
    r = _rule(rule)
    if axis == 1:
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
        scales = torch.empty((cols // 128, rows), dtype=torch.float32, device=x.device)
    else:
        cap = gmm_chunk_capacity(rows, G)
        codes = torch.empty((cap, cols, 128), dtype=torch.uint8, device=x.device)
        scales = torch.empty((cap, cols), dtype=torch.float32, device=x.device)
    nbytes = gmm_workspace_bytes(B.OP_FWD, rows, cols, cols, G)
    if ws is None:
        ws = workspace(nbytes, x.device)
    st = B.lib().gmm_quantize(
        _dev(x, "x", torch.bfloat16), rows, cols, r, axis,
        _dev(static_scale, "static_scale", torch.float32) if static_scale is not None else None,
        _dev(group_sizes, "group_sizes", torch.int32) if group_sizes is not None else None, G,
        _dev(col_scale, "col_scale", torch.float32) if col_scale is not None else None,
        codes.data_ptr(), scales.data_ptr(), ws.data_ptr(), ws.numel(), _stream(x))
    _check(st, "gmm_quantize")
    return codes, scales


def _operand(data, dtype_code, scale, rule):
    return B.Operand(data, dtype_code, scale, rule)


def _rhs_operand(rhs, rhs_scales):
    """rhs with its scales: 2-D scales [G, N] are per channel (rule NONE), 3-D
    scales block-wise (rule DYNAMIC, from gmm_quantize_rhs_blocks)."""
    blockwise = rhs_scales is not None and rhs_scales.dim() == 3
    return _operand(_dev(rhs, "rhs"), _TORCH_DT[rhs.dtype],
                    _dev(rhs_scales, "rhs_scales", torch.float32) if rhs_scales is not None else None,
                    B.Q_DYNAMIC if blockwise else B.Q_NONE)


def gmm_quantize_rhs_blocks(w: torch.Tensor, axis: int = 0):
    """W [G, K, N] bf16 -> (codes uint8 [G, K, N], block-wise scales fp32):
    axis 0 [G, K/128, N] for gmm_fwd, axis 1 [G, N/128, K] for gmm_dlhs."""
    G, K, N = w.shape
    codes = torch.empty((G, K, N), dtype=torch.uint8, device=w.device)
    scales = torch.empty((G, K // 128, N) if axis == 0 else (G, N // 128, K), dtype=torch.float32, device=w.device)
    st = B.lib().gmm_quantize_rhs_blocks(_dev(w, "w", torch.bfloat16), G, K, N, int(axis), codes.data_ptr(),
                                         scales.data_ptr(), _stream(w))
    _check(st, "gmm_quantize_rhs_blocks")
    return codes, scales


def gmm_fwd(lhs: torch.Tensor, rhs: torch.Tensor, rhs_scales: torch.Tensor | None, group_sizes: torch.Tensor,
            rule="static", static_scale: torch.Tensor | None = None, transpose_rhs: bool = False,
            out_dtype=torch.bfloat16, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
            lhs_scales: torch.Tensor | None = None):
    """Forward gmm: out[m] = lhs[m] @ rhs[g(m)] with lhs quantized inside the
    call (rule "static" with ``static_scale``, or "dynamic"); rule "none"
    runs the bf16 family (rhs bf16, no scales).  A uint8 / float8 ``lhs`` is
    taken as already-quantized E4M3 codes: its scale is ``static_scale``
    (static) or ``lhs_scales`` [K/128, M] (dynamic, as gmm_quantize writes)."""
    return _fwd(lhs, rhs, rhs_scales, group_sizes, rule, static_scale, transpose_rhs, out_dtype, out, ws,
                lhs_scales, swiglu=False)


def gmm_fwd_keep_lhs(lhs: torch.Tensor, rhs: torch.Tensor, rhs_scales: torch.Tensor | None,
                     group_sizes: torch.Tensor, rule="static", static_scale: torch.Tensor | None = None,
                     transpose_rhs: bool = False, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None, lhs_codes: torch.Tensor | None = None,
                     lhs_scales: torch.Tensor | None = None):
    """gmm_fwd that also returns the E4M3 codes [M, K] (and, for the dynamic
    rule, the block scales [K/128, M]) it made for lhs: (out, codes, scales),
    written into ``lhs_codes`` / ``lhs_scales`` when given.
    With the static rule the codes can be passed as the lhs of tgmm_drhs /
    gmm_backward, which then skip their own quantization of lhs."""
    M, K = lhs.shape
    G, K2, N = (rhs.shape[0], rhs.shape[2], rhs.shape[1]) if transpose_rhs else rhs.shape
    assert K2 == K, "lhs / rhs contraction mismatch"
    r = _rule(rule)
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=lhs.device)
    if ws is None:
        ws = workspace(gmm_workspace_bytes(B.OP_FWD, M, K, N, G), lhs.device)
    codes = lhs_codes if lhs_codes is not None else torch.empty((M, K), dtype=torch.uint8, device=lhs.device)
    scales = None
    if r == B.Q_DYNAMIC:
        scales = lhs_scales if lhs_scales is not None else torch.empty((K // 128, M), dtype=torch.float32,
                                                                         device=lhs.device)
    a = _operand(_dev(lhs, "lhs", torch.bfloat16), B.DT_BF16,
                 _dev(static_scale, "static_scale", torch.float32) if static_scale is not None else None, r)
    st = B.lib().gmm_fwd_keep_lhs(a, _rhs_operand(rhs, rhs_scales), int(transpose_rhs),
                                  _dev(group_sizes, "group_sizes", torch.int32), G, M, K, N,
                                  _dev(out, "out", (torch.bfloat16, torch.float32)), _TORCH_DT[out.dtype],
                                  ws.data_ptr(), ws.numel(), _dev(codes, "lhs_codes", torch.uint8),
                                  _dev(scales, "lhs_scales", torch.float32) if scales is not None else None,
                                  _stream(lhs))
    _check(st, "gmm_fwd_keep_lhs")
    return out, codes, scales


def gmm_fwd_swiglu(lhs: torch.Tensor, rhs: torch.Tensor, rhs_scales: torch.Tensor | None,
                   group_sizes: torch.Tensor, rule="static", static_scale: torch.Tensor | None = None,
                   transpose_rhs: bool = False, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                   ws: torch.Tensor | None = None, lhs_scales: torch.Tensor | None = None):
    """Merged gate|up forward with SwiGLU fused: rhs is [W0 | W1] along N
    (N = 2F); returns out[M, F] = silu(h[:, :F]) * h[:, F:] with h the merged
    product, which is never written.  Arguments as for gmm_fwd."""
    return _fwd(lhs, rhs, rhs_scales, group_sizes, rule, static_scale, transpose_rhs, out_dtype, out, ws,
                lhs_scales, swiglu=True)


def _fwd(lhs, rhs, rhs_scales, group_sizes, rule, static_scale, transpose_rhs, out_dtype, out, ws, lhs_scales,
         swiglu):
    M, K = lhs.shape
    if transpose_rhs:
        G, N, K2 = rhs.shape
    else:
        G, K2, N = rhs.shape
    assert K2 == K, "lhs / rhs contraction mismatch"
    r = _rule(rule)
    if out is None:
        out = torch.empty((M, N // 2 if swiglu else N), dtype=out_dtype, device=lhs.device)
    if ws is None:
        ws = workspace(gmm_workspace_bytes(B.OP_FWD, M, K, N, G), lhs.device)
    if lhs.dtype in (torch.uint8, torch.float8_e4m3fn):
        sc = static_scale if r == B.Q_STATIC else lhs_scales
        a = _operand(_dev(lhs, "lhs"), B.DT_E4M3, _dev(sc, "lhs scale", torch.float32) if sc is not None else None, r)
    else:
        a = _operand(_dev(lhs, "lhs", torch.bfloat16), B.DT_BF16,
                     _dev(static_scale, "static_scale", torch.float32) if static_scale is not None else None, r)
    b = _rhs_operand(rhs, rhs_scales)
    fn = B.lib().gmm_fwd_swiglu if swiglu else B.lib().gmm_fwd
    st = fn(a, b, int(transpose_rhs), _dev(group_sizes, "group_sizes", torch.int32), G, M, K, N,
            _dev(out, "out", (torch.bfloat16, torch.float32)), _TORCH_DT[out.dtype], ws.data_ptr(),
            ws.numel(), _stream(lhs))
    _check(st, "gmm_fwd_swiglu" if swiglu else "gmm_fwd")
    return out


def gmm_dlhs(dout: torch.Tensor, rhs: torch.Tensor, rhs_scales: torch.Tensor | None, group_sizes: torch.Tensor,
             transpose_rhs: bool = False, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
             ws: torch.Tensor | None = None, rule="dynamic"):
    """Backward gmm wrt lhs: dlhs[m] = dout[m] @ rhs[g(m)]^T, dout quantized
    with dynamic 128-blocks after folding the rhs column scale in."""
    M, N = dout.shape
    if transpose_rhs:
        G, N2, K = rhs.shape
    else:
        G, K, N2 = rhs.shape
    assert N2 == N, "dout / rhs mismatch"
    r = _rule(rule)
    if out is None:
        out = torch.empty((M, K), dtype=out_dtype, device=dout.device)
    if ws is None:
        ws = workspace(gmm_workspace_bytes(B.OP_DLHS, M, K, N, G), dout.device)
    a = _operand(_dev(dout, "dout", torch.bfloat16), B.DT_BF16, None, r)
    b = _rhs_operand(rhs, rhs_scales)
    st = B.lib().gmm_dlhs(a, b, int(transpose_rhs), _dev(group_sizes, "group_sizes", torch.int32), G, M, K, N,
                          _dev(out, "out", (torch.bfloat16, torch.float32)), _TORCH_DT[out.dtype], ws.data_ptr(),
                          ws.numel(), _stream(dout))
    _check(st, "gmm_dlhs")
    return out


def tgmm_drhs(lhs: torch.Tensor, dout: torch.Tensor, group_sizes: torch.Tensor, rule="static",
              static_scale: torch.Tensor | None = None, out_dtype=torch.float32, out: torch.Tensor | None = None,
              ws: torch.Tensor | None = None):
    """Weight gradient dW[g] = lhs[rows of g]^T @ dout[rows of g] ([G, K, N]),
    both operands quantized per 128-row chunk of each group.  With rule
    "static" a uint8 / float8 ``lhs`` is taken as the forward's E4M3 codes
    (scale ``static_scale``) and only re-laid out."""
    M, K = lhs.shape
    M2, N = dout.shape
    assert M2 == M
    G = int(group_sizes.numel())
    r = _rule(rule)
    if out is None:
        out = torch.empty((G, K, N), dtype=out_dtype, device=lhs.device)
    if ws is None:
        ws = workspace(gmm_workspace_bytes(B.OP_DRHS, M, K, N, G), lhs.device)
    sc = _dev(static_scale, "static_scale", torch.float32) if static_scale is not None else None
    if lhs.dtype in (torch.uint8, torch.float8_e4m3fn):
        a = _operand(_dev(lhs, "lhs"), B.DT_E4M3, sc, r)
    else:
        a = _operand(_dev(lhs, "lhs", torch.bfloat16), B.DT_BF16, sc, r)
    d = _operand(_dev(dout, "dout", torch.bfloat16), B.DT_BF16, None, B.Q_NONE if r == B.Q_NONE else B.Q_DYNAMIC)
    st = B.lib().tgmm_drhs(a, d, _dev(group_sizes, "group_sizes", torch.int32), G, M, K, N,
                           _dev(out, "out", (torch.bfloat16, torch.float32)), _TORCH_DT[out.dtype], ws.data_ptr(),
                           ws.numel(), _stream(lhs))
    _check(st, "tgmm_drhs")
    return out


def gmm_backward(lhs: torch.Tensor, dout: torch.Tensor, rhs: torch.Tensor, rhs_scales: torch.Tensor | None,
                 group_sizes: torch.Tensor, rule="static", static_scale: torch.Tensor | None = None,
                 transpose_rhs: bool = False, dlhs_dtype=torch.bfloat16, drhs_dtype=torch.float32,
                 dlhs: torch.Tensor | None = None, drhs: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Both backward passes in one call (dout read once): returns (dlhs [M, K],
    dW [G, K, N]) equal bit for bit to gmm_dlhs and tgmm_drhs.  ``rule`` and
    ``static_scale`` describe lhs as for tgmm_drhs ("none": bf16 family)."""
    M, K = lhs.shape
    M2, N = dout.shape
    assert M2 == M
    G = int(group_sizes.numel())
    r = _rule(rule)
    if dlhs is None:
        dlhs = torch.empty((M, K), dtype=dlhs_dtype, device=lhs.device)
    if drhs is None:
        drhs = torch.empty((G, K, N), dtype=drhs_dtype, device=lhs.device)
    if ws is None:
        ws = workspace(gmm_workspace_bytes(B.OP_BWD, M, K, N, G), lhs.device)
    sc = _dev(static_scale, "static_scale", torch.float32) if static_scale is not None else None
    if lhs.dtype in (torch.uint8, torch.float8_e4m3fn):
        a = _operand(_dev(lhs, "lhs"), B.DT_E4M3, sc, r)
    else:
        a = _operand(_dev(lhs, "lhs", torch.bfloat16), B.DT_BF16, sc, r)
    d = _operand(_dev(dout, "dout", torch.bfloat16), B.DT_BF16, None, B.Q_NONE if r == B.Q_NONE else B.Q_DYNAMIC)
    b = _rhs_operand(rhs, rhs_scales)
    st = B.lib().gmm_backward(a, d, b, int(transpose_rhs), _dev(group_sizes, "group_sizes", torch.int32), G, M, K, N,
                              _dev(dlhs, "dlhs", (torch.bfloat16, torch.float32)), _TORCH_DT[dlhs.dtype],
                              _dev(drhs, "drhs", (torch.bfloat16, torch.float32)), _TORCH_DT[drhs.dtype],
                              ws.data_ptr(), ws.numel(), _stream(lhs))
    _check(st, "gmm_backward")
    return dlhs, drhs


ACTS = {"none": B.ACT_NONE, "relu": B.ACT_RELU, "silu": B.ACT_SILU, "gelu": B.ACT_GELU,
        "gelu_tanh": B.ACT_GELU_TANH, "swiglu": B.ACT_SWIGLU}
SCORES = {"softmax": B.SCORE_SOFTMAX, "sigmoid": B.SCORE_SIGMOID}


def _name(table: dict, name, what: str) -> int:
    if name not in table:
        raise ValueError(f"{what} must be one of {sorted(table)}, not {name!r}")
    return table[name]


def _same_device(first: torch.Tensor, *others):
    dev = first.device
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {t.device} and {dev}: all must be on one device")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_here = contextlib.nullcontext()


def _on(t: torch.Tensor):
    """Makes t's device current for the call (nothing to do when it is)."""
    return _here if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)


def _current(t: torch.Tensor) -> int:
    """The raw handle of torch's current stream on t's device, without the
    Python stream object (a microsecond of the smallest calls)."""
    return _raw_stream(t.device.index) if _raw_stream else _stream(t)


@functools.lru_cache(maxsize=4096)
def _fwd_bytes(M: int, K: int, N: int, G: int) -> int:
    return gmm_workspace_bytes(B.OP_FWD, M, K, N, G)


@functools.lru_cache(maxsize=4096)
def _act_bwd_bytes(M: int, N: int, G: int) -> int:
    return int(B.lib().gmm_act_bwd_workspace_bytes(M, N, G))


@functools.lru_cache(maxsize=4096)
def _few_bytes(T: int, k: int, G: int, K: int, F: int, N: int, dtype: int) -> int:
    return int(B.lib().gmm_moe_few_workspace_bytes(T, k, G, K, F, N, dtype))


def _shape(t: torch.Tensor | None, name: str, shape):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _empty(like: torch.Tensor, shape, dtype) -> torch.Tensor:
    """like.new_empty for two dimensions, in 1.4 us of the host instead of 2."""
    return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=like.device)


_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_FLOAT = (torch.bfloat16, torch.float32)
_OPERAND = (torch.bfloat16, torch.uint8, torch.float8_e4m3fn)
_U8 = (torch.uint8,)


def _pointers(*args):
    """Device pointers of a call's tensors.  Each argument: (tensor or None,
    name, shape or None for any, dtypes).  All must be contiguous and on the
    first tensor's CUDA device; _refuse words what is not so.  (One pass of
    attribute reads: a check a function cost the smallest calls 4 us.)"""
    dev = args[0][0].get_device()  # -1 for the CPU
    ptrs = []
    for t, name, shape, dtypes in args:
        if t is None:
            ptrs.append(None)
            continue
        if dev < 0 or t.get_device() != dev or t.dtype not in dtypes or not t.is_contiguous() or \
                (shape is not None and t.shape != shape):
            _refuse(args)
        ptrs.append(t.data_ptr())
    return ptrs


def _refuse(args):
    for t, name, shape, _ in args:
        if shape is not None:
            _shape(t, name, shape)
    _same_device(*(a[0] for a in args))
    for t, name, _, dtypes in args:
        _dev(t, name, dtypes)
    raise ValueError("unusable tensors")


def _scratch(nbytes: int, like: torch.Tensor) -> torch.Tensor:
    """A workspace from torch's caching allocator for one call alone: the
    allocator keeps it apart per stream and per captured graph, so that calls
    on several streams or in several graphs share none."""
    return like.new_empty(max(nbytes, 256), dtype=torch.uint8)


def gmm_fwd_act(lhs: torch.Tensor, rhs: torch.Tensor, rhs_scales: torch.Tensor | None, group_sizes: torch.Tensor,
                act: str = "none", bias: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                rule="static", static_scale: torch.Tensor | None = None, transpose_rhs: bool = False,
                out_dtype=torch.bfloat16, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                lhs_scales: torch.Tensor | None = None, keep_preact: bool = False,
                preact: torch.Tensor | None = None):
    """gmm_fwd with bias, activation and residual in the epilogue:
    out = act(z) + residual, z = product + bias[g].  ``act``: "none", "relu",
    "silu", "gelu", "gelu_tanh" or "swiglu" (merged gate|up rhs; out is
    [M, N/2]).  bias: fp32 [G, N]; residual: bf16 or fp32, of out's shape (it
    may be ``out`` itself when of its type).  With keep_preact (or a bf16
    [M, N] buffer ``preact``) returns (out, z), z for gmm_act_bwd.  Other
    arguments as for gmm_fwd."""
    a_code = _name(ACTS, act, "act")
    M, K = lhs.shape
    G, K2, N = (rhs.shape[0], rhs.shape[2], rhs.shape[1]) if transpose_rhs else rhs.shape
    if K2 != K:
        raise ValueError(f"lhs contracts over {K}, rhs over {K2}")
    r = _rule(rule)
    out_shape = (M, N // 2 if act == "swiglu" else N)
    if out is None:
        out = _empty(lhs, out_shape, out_dtype)
    if preact is None and keep_preact:
        preact = _empty(lhs, (M, N), torch.bfloat16)
    if ws is None:
        ws = _scratch(_fwd_bytes(M, K, N, G), lhs)
    blockwise = rhs_scales is not None and rhs_scales.dim() == 3
    if lhs.dtype == torch.bfloat16:
        lhs_dt, sc, sc_shape = B.DT_BF16, static_scale, None
    else:
        lhs_dt, sc = B.DT_E4M3, static_scale if r == B.Q_STATIC else lhs_scales
        sc_shape = None if r == B.Q_STATIC else (K // 128, M)
    a_p, w_p, ws_p, gs_p, out_p, sc_p, wsc_p, bias_p, res_p, z_p = _pointers(
        (lhs, "lhs", None, _OPERAND), (rhs, "rhs", None, _OPERAND), (ws, "ws", None, _U8),
        (group_sizes, "group_sizes", (G,), _I32), (out, "out", out_shape, _FLOAT),
        (sc, "lhs scale", sc_shape, _F32),
        (rhs_scales, "rhs_scales", (G, K // 128, N) if blockwise else (G, N), _F32), (bias, "bias", (G, N), _F32),
        (residual, "residual", out_shape, _FLOAT), (preact, "preact", (M, N), _BF16))
    epi = B.Epilogue(a_code, bias_p, res_p, _TORCH_DT[residual.dtype] if res_p is not None else B.DT_BF16, z_p)
    with _on(lhs):
        st = B.lib().gmm_fwd_act(B.Operand(a_p, lhs_dt, sc_p, r),
                                 B.Operand(w_p, _TORCH_DT[rhs.dtype], wsc_p, B.Q_DYNAMIC if blockwise else B.Q_NONE),
                                 int(transpose_rhs), gs_p, G, M, K, N, ctypes.byref(epi), out_p,
                                 _TORCH_DT[out.dtype], ws_p, ws.numel(), _current(lhs))
    if st != B.GMM_OK:
        raise GmmError(st, "gmm_fwd_act")
    return out if preact is None else (out, preact)


def gmm_act_bwd(dout: torch.Tensor, preact: torch.Tensor, group_sizes: torch.Tensor, act: str = "none",
                with_dbias: bool = True, dz: torch.Tensor | None = None, dbias: torch.Tensor | None = None,
                ws: torch.Tensor | None = None):
    """Gradient of gmm_fwd_act's epilogue: (dz [M, N] bf16, dbias [G, N] fp32
    or None).  dz = dout * act'(z) is the dout of gmm_dlhs / tgmm_drhs /
    gmm_backward; the residual's gradient is dout itself."""
    a_code = _name(ACTS, act, "act")
    M, N = preact.shape
    G = int(group_sizes.numel())
    if dz is None:
        dz = _empty(dout, (M, N), torch.bfloat16)
    if dbias is None and with_dbias:
        dbias = _empty(dout, (G, N), torch.float32)
    if ws is None:
        ws = _scratch(_act_bwd_bytes(M, N, G), dout)
    dout_p, z_p, gs_p, dz_p, db_p, ws_p = _pointers(
        (dout, "dout", (M, N // 2 if act == "swiglu" else N), _BF16), (preact, "preact", None, _BF16),
        (group_sizes, "group_sizes", None, _I32), (dz, "dz", (M, N), _BF16), (dbias, "dbias", (G, N), _F32),
        (ws, "ws", None, _U8))
    with _on(dout):
        st = B.lib().gmm_act_bwd(dout_p, z_p, a_code, gs_p, G, M, N, dz_p, db_p, ws_p, ws.numel(), _current(dout))
    if st != B.GMM_OK:
        raise GmmError(st, "gmm_act_bwd")
    return dz, dbias


def gmm_moe_few(x: torch.Tensor, expert_ids: torch.Tensor, weights: torch.Tensor, w1: torch.Tensor,
                w1_scales: torch.Tensor | None, w2: torch.Tensor, w2_scales: torch.Tensor | None,
                transpose_rhs: bool = False, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                ws: torch.Tensor | None = None):
    """A whole mixture-of-experts layer for a few tokens in one kernel:
    y[t] = sum_j weights[t, j] * (silu(g) * u) @ W2[e], [g | u] = x[t] @ W1[e],
    e = expert_ids[t, j].  x: bf16 [T, K] (not quantized); expert_ids int32
    and weights fp32 [T, k] (as gmm_router_topk gives them); w1 [G, K, 2F]
    merged gate|up and w2 [G, F, N] (transpose_rhs: [G, 2F, K], [G, N, F]),
    both E4M3 codes with scales [G, 2F] and [G, N], or both bf16 with scales
    None.  T * k <= 1024.  Returns y [T, N]."""
    T, K = x.shape
    k = expert_ids.shape[1]
    G, K2, F2 = (w1.shape[0], w1.shape[2], w1.shape[1]) if transpose_rhs else w1.shape
    G2, F, N = (w2.shape[0], w2.shape[2], w2.shape[1]) if transpose_rhs else w2.shape
    if K2 != K or G2 != G or F2 != 2 * F:
        raise ValueError(f"x {tuple(x.shape)}, w1 {tuple(w1.shape)} and w2 {tuple(w2.shape)} do not fit together")
    if out is None:
        out = _empty(x, (T, N), out_dtype)
    dt = _TORCH_DT.get(w1.dtype, B.DT_F32)
    if ws is None:
        ws = _scratch(_few_bytes(T, k, G, K, F, N, dt), x)
    x_p, ids_p, wt_p, w1_p, s1_p, w2_p, s2_p, y_p, ws_p = _pointers(
        (x, "x", None, _BF16), (expert_ids, "expert_ids", (T, k), _I32), (weights, "weights", (T, k), _F32),
        (w1, "w1", None, _OPERAND), (w1_scales, "w1_scales", (G, F2), _F32), (w2, "w2", None, _OPERAND),
        (w2_scales, "w2_scales", (G, N), _F32), (out, "out", (T, N), _FLOAT), (ws, "ws", None, _U8))
    with _on(x):
        st = B.lib().gmm_moe_few(x_p, ids_p, wt_p, T, k, B.Operand(w1_p, dt, s1_p, B.Q_NONE),
                                 B.Operand(w2_p, _TORCH_DT[w2.dtype], s2_p, B.Q_NONE), int(transpose_rhs), G, K, F, N,
                                 y_p, _TORCH_DT[out.dtype], ws_p, ws.numel(), _current(x))
    if st != B.GMM_OK:
        raise GmmError(st, "gmm_moe_few")
    return out


def gmm_router_topk(logits: torch.Tensor, k: int, score: str = "softmax", select_bias: torch.Tensor | None = None,
                    normalize: bool = False, scale: float = 1.0):
    """The router: (expert_ids int32 [T, k], weights fp32 [T, k]) of the k
    experts of largest score (+ select_bias, fp32 [E], for the choice only),
    ties to the lowest index.  weights = scale * score, or with normalize
    scale * score / (sum of the chosen scores).  Experts masked with -inf are
    never chosen (id -1, weight 0 where fewer than k are left)."""
    T, E = logits.shape
    ids = _empty(logits, (T, k), torch.int32)
    weights = _empty(logits, (T, k), torch.float32)
    x_p, bias_p = _pointers((logits, "logits", None, _FLOAT), (select_bias, "select_bias", (E,), _F32))
    with _on(logits):
        st = B.lib().gmm_router_topk(x_p, _TORCH_DT[logits.dtype], T, E, k, _name(SCORES, score, "score"), bias_p,
                                     int(normalize), float(scale), ids.data_ptr(), weights.data_ptr(),
                                     _current(logits))
    if st != B.GMM_OK:
        raise GmmError(st, "gmm_router_topk")
    return ids, weights


def gmm_router_topk_bwd(dweights: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor,
                        score: str = "softmax", normalize: bool = False, scale: float = 1.0):
    """Gradient of gmm_router_topk's weights: dlogits [T, E] (logits' type)
    from dweights [T, k] fp32, the logits and the chosen expert_ids."""
    T, E = logits.shape
    k = expert_ids.shape[1]
    dlogits = torch.empty_like(logits)
    x_p, dw_p, ids_p = _pointers((logits, "logits", None, _FLOAT), (dweights, "dweights", (T, k), _F32),
                                 (expert_ids, "expert_ids", (T, k), _I32))
    with _on(logits):
        st = B.lib().gmm_router_topk_bwd(dw_p, x_p, _TORCH_DT[logits.dtype], ids_p, T, E, k,
                                         _name(SCORES, score, "score"), int(normalize), float(scale),
                                         dlogits.data_ptr(), _current(logits))
    if st != B.GMM_OK:
        raise GmmError(st, "gmm_router_topk_bwd")
    return dlogits


def gmm_combine_dweight(dy: torch.Tensor, rows: torch.Tensor, slot: torch.Tensor):
    """Gradient of the combine's routing weights: dweight[t, j] =
    sum_n dy[t, n] * rows[slot[t, j], n] (fp32 [T, k]; 0 for a slot outside
    rows).  dy [T, N] and rows [R, N] bf16, slot int32 [T, k]."""
    T, k = slot.shape
    R, N = rows.shape
    dw = _empty(dy, (T, k), torch.float32)
    dy_p, rows_p, slot_p = _pointers((dy, "dy", (T, N), _BF16), (rows, "rows", None, _BF16),
                                     (slot, "slot", None, _I32))
    with _on(dy):
        st = B.lib().gmm_combine_dweight(dy_p, rows_p, R, slot_p, T, k, N, dw.data_ptr(), _current(dy))
    if st != B.GMM_OK:
        raise GmmError(st, "gmm_combine_dweight")
    return dw


def gmm_read_device_status(ws: torch.Tensor):
    """(status, bits) left in ``ws`` by the last call; synchronizes the stream."""
    bits = ctypes.c_uint32(0)
    st = B.lib().gmm_read_device_status(ws.data_ptr(), ctypes.byref(bits), _stream(ws))
    return st, bits.value


def gmm_selftest_timeout(ws: torch.Tensor, limit_ns: int):
    _check(B.lib().gmm_selftest_timeout(ws.data_ptr(), limit_ns, _stream(ws)), "gmm_selftest_timeout")


def gmm_set_wait_limit_ns(limit_ns: int):
    B.lib().gmm_set_wait_limit_ns(limit_ns)


TILES = {"auto": B.TILES_AUTO, "one_cta": B.TILES_ONE_CTA, "cta_pairs": B.TILES_CTA_PAIRS,
         "cta_pairs_narrow": B.TILES_CTA_PAIRS_NARROW}


def gmm_set_tiles(mode="auto"):
    """GEMM tile choice for the calls that follow: "auto", "one_cta" (128-row
    tiles), "cta_pairs" (256-row tiles over a two-CTA cluster) or
    "cta_pairs_narrow" (CTA pairs; 256 x 128 tiles for the promoted passes
    with K-major weights)."""
    _check(B.lib().gmm_set_tiles(TILES[mode] if isinstance(mode, str) else int(mode)), "gmm_set_tiles")


def gmm_plan(group_sizes: torch.Tensor, M: int):
    """Host-side helper (no kernel): clamped row offsets of the groups, as
    int64 CPU tensor [G + 1] (same rule as the device plan)."""
    gs = group_sizes.detach().to("cpu", torch.int64).clamp(min=0)
    offs = torch.zeros(gs.numel() + 1, dtype=torch.int64)
    offs[1:] = torch.cumsum(gs, 0).clamp(max=M)
    return offs


def profile_enable(on: bool = True):
    """Bracket every library kernel launch with CUDA events (benchmarks)."""
    B.lib().gmm_profile_enable(int(on))


def profile_collect() -> dict:
    """{kernel name: (launches, total ms)} since the last collect."""
    arr = (B.ProfileEntry * 32)()
    n = B.lib().gmm_profile_collect(arr, 32)
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms)) for i in range(n)}
