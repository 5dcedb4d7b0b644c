"""Cases, inputs and plain forms of the operators around the expert products.

Four operators, each through the calls a user makes:

  act      gmm_fwd_act / gmm_act_bwd: the grouped (or, with one group, dense)
           product with bias, activation and residual in its epilogue, and the
           gradient of that epilogue
  few      gmm_moe_few: a whole mixture-of-experts layer (merged gate|up
           product, SwiGLU, down product, weighted sum) for a few tokens
  router   gmm_router_topk and gmm_router_topk_bwd with gmm_combine_dweight:
           the choice of k experts a token, and the gradient of its weights

With ``own`` false ``run`` computes the plain form in elementary torch
operations; with ``own`` true it calls this repository's package.
"""
import math

import torch

own = False

FP8_MAX = 448.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest training call: latency of one expert projection with bias
        {"name": "act_fwd_tiny", "op": "act", "dir": "fwd", "G": 8, "M": 256, "K": 512, "N": 512, "rule": "static",
         "act": "silu", "bias": True, "residual": False, "keep": False, "trans": False, "routing": "uniform"},
        # a dense feed-forward up projection in bf16 (one group), as beside the experts of a layer
        {"name": "act_fwd_dense_bf16", "op": "act", "dir": "fwd", "G": 1, "M": 4099, "K": 4096, "N": 14336, "rule": "none",
         "act": "gelu_tanh", "bias": True, "residual": False, "keep": False, "trans": True, "routing": "uniform"},
        # the Mixtral-like merged gate|up projection of a training forward, which keeps z for the backward
        {"name": "act_fwd_mixtral_swiglu", "op": "act", "dir": "fwd", "G": 8, "M": 16384, "K": 4096, "N": 28672,
         "rule": "static", "act": "swiglu", "bias": True, "residual": False, "keep": True, "trans": False,
         "routing": "uniform"},
        # the DeepSeek-V3-shaped down projection: many small ragged groups, residual added in place of a pass
        {"name": "act_fwd_dsv3_down", "op": "act", "dir": "fwd", "G": 256, "M": 32768, "K": 2048, "N": 7168,
         "rule": "dynamic", "act": "none", "bias": False, "residual": True, "keep": False, "trans": False,
         "routing": "zipf"},
        # gradient of the merged SwiGLU epilogue of the Mixtral-like step
        {"name": "act_bwd_mixtral_swiglu", "op": "act", "dir": "bwd", "G": 8, "M": 16384, "N": 28672, "act": "swiglu",
         "bias": True, "routing": "uniform"},
        # gradient of a bias + GELU epilogue over many ragged groups, some empty, with padded rows behind the last
        {"name": "act_bwd_ragged_gelu", "op": "act", "dir": "bwd", "G": 256, "M": 8195, "N": 2048, "act": "gelu",
         "bias": True, "routing": "tail"},
        # decoding one token through a tiny layer: latency
        {"name": "few_tiny_t1", "op": "few", "T": 1, "k": 2, "G": 8, "K": 512, "F": 256, "N": 512, "weights": "e4m3",
         "trans": False},
        # decoding one token through the Mixtral-like layer: the weights of two experts
        {"name": "few_mixtral_t1", "op": "few", "T": 1, "k": 2, "G": 8, "K": 4096, "F": 14336, "N": 4096,
         "weights": "e4m3", "trans": False},
        # a small decoding batch through the DeepSeek-V3-shaped layer: about a hundred experts, most with one row
        {"name": "few_dsv3_t16", "op": "few", "T": 16, "k": 8, "G": 256, "K": 7168, "F": 2048, "N": 7168,
         "weights": "e4m3", "trans": True},
        # bf16 weights, an odd batch over the experts of one expert-parallel rank
        {"name": "few_bf16_t5", "op": "few", "T": 5, "k": 4, "G": 32, "K": 7168, "F": 256, "N": 7168, "weights": "bf16",
         "trans": False},
        # routing of a training batch: sigmoid scores, a selection bias, normalised weights
        {"name": "router_fwd_t4096", "op": "router", "dir": "fwd", "T": 4096, "E": 256, "k": 8, "score": "sigmoid",
         "select_bias": True, "normalize": True, "dtype": "f32", "masked": 0},
        # gradient of the routing of that batch: from dy and the experts' rows to the logits
        {"name": "router_bwd_t4096", "op": "router", "dir": "bwd", "T": 4096, "E": 256, "k": 8, "N": 7168,
         "score": "softmax", "normalize": False, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_128(rng, lo, hi):
    return 128 * _log_int(rng, max(1, lo // 128), hi // 128)


def draw(rng):
    kind = rng.choice(["act_fwd", "act_fwd", "act_bwd", "few", "few", "router_fwd", "router_bwd"])
    if kind == "act_fwd":
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
        while True:
            G, M = _log_int(rng, 1, 256), _log_int(rng, 1, 32768)
            K, N = _log_128(rng, 128, 7168), _log_128(rng, 256, 28672)
            if act == "swiglu":
                N = max(256, N // 256 * 256)
            if M * K * N <= 16384 * 4096 * 28672 // 2 and G * K * N <= 256 * 2048 * 7168:
                break
        return {"op": "act", "dir": "fwd", "G": G, "M": M, "K": K, "N": N,
                "rule": rng.choice(["static", "dynamic", "none"]), "act": act, "bias": rng.random() < 0.6,
                "residual": rng.random() < 0.5, "keep": rng.random() < 0.4, "trans": rng.random() < 0.5,
                "routing": rng.choice(["uniform", "zipf", "tail"])}
    if kind == "act_bwd":
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
        G, M, N = _log_int(rng, 1, 256), _log_int(rng, 1, 16384), _log_128(rng, 256, 28672)
        if act == "swiglu":
            N = max(256, N // 256 * 256)
        return {"op": "act", "dir": "bwd", "G": G, "M": M, "N": N, "act": act, "bias": rng.random() < 0.7,
                "routing": rng.choice(["uniform", "zipf", "tail"])}
    if kind == "few":
        while True:
            G, T = _log_int(rng, 1, 256), _log_int(rng, 1, 64)
            k = min(G, _log_int(rng, 1, 8))
            K, F, N = _log_128(rng, 128, 7168), _log_128(rng, 128, 14336), _log_128(rng, 128, 7168)
            wt = rng.choice(["e4m3", "e4m3", "bf16"])
            each = (2 * K * F + F * N) * (1 if wt == "e4m3" else 2)
            if G * each <= 256 * (2 * 7168 * 2048 + 2048 * 7168) and T * k * (2 * K * F + F * N) <= 128 * 3 * 7168 * 2048:
                break
        return {"op": "few", "T": T, "k": k, "G": G, "K": K, "F": F, "N": N, "weights": wt, "trans": rng.random() < 0.5}
    E = _log_int(rng, 2, 512)
    k = min(E, _log_int(rng, 1, 8))
    case = {"op": "router", "T": _log_int(rng, 1, 8192 if kind == "router_fwd" else 4096), "E": E, "k": k,
            "score": rng.choice(["softmax", "sigmoid"]), "normalize": rng.random() < 0.5,
            "dtype": rng.choice(["f32", "bf16"])}
    if kind == "router_fwd":
        return {**case, "dir": "fwd", "select_bias": rng.random() < 0.5,
                "masked": rng.choice([0, 0, min(E // 4, E - k)])}
    return {**case, "dir": "bwd", "N": 8 * _log_int(rng, 16, 896)}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _sizes(case, seed):
    """Rows per group (host list): as a training step's routing leaves them."""
    G, M = case["G"], case["M"]
    g = torch.Generator().manual_seed(seed * 31 + 7)
    rows = M - M // 9 if case["routing"] == "tail" else M  # "tail": padded rows behind the last group
    if case["routing"] == "zipf":
        p = torch.arange(1, G + 1, dtype=torch.float64).pow(-1.2)[torch.randperm(G, generator=g)]
    else:
        p = torch.ones(G, dtype=torch.float64)
        if case["routing"] == "tail" and G > 2:
            p[torch.randperm(G, generator=g)[:G // 4]] = 0.0
    idx = torch.multinomial(p, max(rows, 1), replacement=True, generator=g)[:rows]
    return torch.bincount(idx, minlength=G).tolist()


def _e4m3(x):
    """Nearest E4M3 code (ties to even), saturating at +-448."""
    return x.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _quant_weights(w, axis):
    """Per-channel E4M3 codes (uint8) and fp32 scales over the contraction axis."""
    f = w.float()
    s = f.abs().amax(axis, keepdim=True) / FP8_MAX
    return _e4m3(f * (1.0 / s)).view(torch.uint8), s.squeeze(axis)


def _weights(g, G, K, N, trans, kind):
    """[G, K, N] (or [G, N, K] with trans) weights and their scales [G, N]."""
    shape = (G, N, K) if trans else (G, K, N)
    if kind == "bf16":
        w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        for e in range(G):
            w[e] = _normal(g, shape[1:], 0.02)
        return w, None
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    scales = torch.empty((G, N), dtype=torch.float32, device="cuda")
    for e in range(G):
        codes[e], scales[e] = _quant_weights(_normal(g, shape[1:], 0.02), 1 if trans else 0)
    return codes, scales


def _distinct(g, T, G, k):
    """k distinct experts a token (int32) and normalised weights."""
    logits = torch.randn((T, G), generator=g, device="cuda")
    v, i = torch.topk(logits, k, dim=1)
    return i.to(torch.int32).contiguous(), torch.softmax(v, 1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "act":
        G, M, N = case["G"], case["M"], case["N"]
        sizes = _sizes(case, seed)
        st["sizes"] = sizes
        st["group_sizes"] = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        out_n = N // 2 if case["act"] == "swiglu" else N
        if case["dir"] == "fwd":
            st["lhs"] = _normal(g, (M, case["K"]))
            st["rhs"], st["rhs_scales"] = _weights(g, G, case["K"], N, case["trans"],
                                                   "bf16" if case["rule"] == "none" else "e4m3")
            st["static_scale"] = torch.full((1,), 4.0 / FP8_MAX, device="cuda")
            st["bias"] = _normal(g, (G, N), 0.5, torch.float32) if case["bias"] else None
            st["residual"] = _normal(g, (M, out_n)) if case["residual"] else None
        else:
            st["dout"] = _normal(g, (M, out_n))
            st["z"] = _normal(g, (M, N), 1.5)
    elif case["op"] == "few":
        T, k, G = case["T"], case["k"], case["G"]
        st["x"] = _normal(g, (T, case["K"]))
        st["ids"], st["weights"] = _distinct(g, T, G, k)
        st["w1"], st["s1"] = _weights(g, G, case["K"], 2 * case["F"], case["trans"], case["weights"])
        st["w2"], st["s2"] = _weights(g, G, case["F"], case["N"], case["trans"], case["weights"])
    else:
        T, E, k = case["T"], case["E"], case["k"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        st["logits"] = _normal(g, (T, E), 1.5, dt)
        if case["dir"] == "fwd":
            st["select_bias"] = _normal(g, (E,), 0.05, torch.float32) if case["select_bias"] else None
            if case["masked"]:
                st["logits"][:, torch.randperm(E, generator=g, device="cuda")[:case["masked"]]] = -math.inf
        else:
            st["ids"], _ = _distinct(g, T, E, k)
            st["dy"] = _normal(g, (T, case["N"]))
            st["rows"] = _normal(g, (T * k, case["N"]))
            st["slot"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    return st


# ------------------------------------------------------------- plain forms

def _quant_lhs(x, rule, static_scale):
    """The values the quantized lhs stands for (fp32)."""
    f = x.float()
    if rule == "none":
        return f
    if rule == "static":
        return _e4m3(f * (1.0 / static_scale)).float() * static_scale
    b = f.view(f.shape[0], -1, 128)
    s = b.abs().amax(2, keepdim=True) / FP8_MAX
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    return (_e4m3(b * inv).float() * s).view(f.shape)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "swiglu":
        g, u = z.chunk(2, dim=1)
        return g / (1.0 + torch.exp(-g)) * u
    return z


def _act_grad(z, dout, act):
    if act == "relu":
        return torch.where(z > 0, dout, torch.zeros_like(dout))
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return dout * (s * (1.0 + z * (1.0 - s)))
    if act == "gelu":
        return dout * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return dout * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z))
    if act == "swiglu":
        g, u = z.chunk(2, dim=1)
        s = 1.0 / (1.0 + torch.exp(-g))
        return torch.cat([dout * u * (s * (1.0 + g * (1.0 - s))), dout * (g * s)], dim=1)
    return dout


def _group_of_row(st, M):
    """[M] group of each row, G for the rows behind the last group."""
    ends = torch.cumsum(st["group_sizes"].to(torch.int64), 0)
    return torch.searchsorted(ends, torch.arange(M, device="cuda"), right=True)


def _act_fwd(st, case):
    M, N = case["M"], case["N"]
    a = _quant_lhs(st["lhs"], case["rule"], st["static_scale"])
    z = torch.zeros((M, N), device="cuda")
    r0 = 0
    for e, n in enumerate(st["sizes"]):
        if n:
            w = st["rhs"][e] if case["rule"] == "none" else st["rhs"][e].view(torch.float8_e4m3fn)
            w = w.float().t() if case["trans"] else w.float()
            y = a[r0:r0 + n] @ w
            if st["rhs_scales"] is not None:
                y = y * st["rhs_scales"][e]
            z[r0:r0 + n] = y if st["bias"] is None else y + st["bias"][e]
            r0 += n
    out = _act(z, case["act"])
    if st["residual"] is not None:
        out[:r0] += st["residual"][:r0].float()
    out = out.to(torch.bfloat16)
    return (out, z.to(torch.bfloat16)) if case["keep"] else out


def _act_bwd(st, case):
    dz = _act_grad(st["z"].float(), st["dout"].float(), case["act"])
    g = _group_of_row(st, case["M"])
    dz = torch.where((g < case["G"])[:, None], dz, torch.zeros_like(dz))
    if not case["bias"]:
        return dz.to(torch.bfloat16)
    db = torch.zeros((case["G"] + 1, case["N"]), device="cuda").index_add_(0, g, dz)
    return dz.to(torch.bfloat16), db[:case["G"]]


def _pair_weights(w, ids, trans, dtype):
    """The experts' weights of every (token, choice): [T*k, contraction, columns]."""
    p = w.index_select(0, ids.reshape(-1).long())
    p = (p if p.dtype == torch.bfloat16 else p.view(torch.float8_e4m3fn)).to(dtype)
    return p.transpose(1, 2) if trans else p


def _few(st, case):
    T, k = case["T"], case["k"]
    idx = st["ids"].reshape(-1).long()
    xr = st["x"].float().repeat_interleave(k, 0)[:, None, :]
    h = torch.bmm(xr, _pair_weights(st["w1"], st["ids"], case["trans"], torch.float32))[:, 0]
    if st["s1"] is not None:
        h = h * st["s1"][idx]
    h = _act(h, "swiglu")[:, None, :]
    y = torch.bmm(h, _pair_weights(st["w2"], st["ids"], case["trans"], torch.float32))[:, 0]
    if st["s2"] is not None:
        y = y * st["s2"][idx]
    return (y.view(T, k, -1) * st["weights"][:, :, None]).sum(1).to(torch.bfloat16)


def _scores(logits, score):
    """Scores in 64 bits: the choice compares neighbouring values."""
    x = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _router_fwd(st, case):
    p = _scores(st["logits"], case["score"])
    key = p if st["select_bias"] is None else p + st["select_bias"].double()
    if st["select_bias"] is None:
        key = st["logits"].double()
    key = torch.where(st["logits"] == -math.inf, torch.full_like(key, -math.inf), key)
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :case["k"]]
    w = torch.gather(p, 1, ids)
    if case["normalize"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), w.float()


def _router_bwd(st, case):
    T, k = case["T"], case["k"]
    dw = (st["dy"].float()[:, None, :] * st["rows"].float().index_select(0, st["slot"].view(-1).long()).view(T, k, -1)).sum(2)
    x, idx = st["logits"].float(), st["ids"].long()
    p = _scores(x, case["score"]).float()
    q = torch.gather(p, 1, idx)
    if case["normalize"]:
        w = q / q.sum(1, keepdim=True)
        c = w * (dw - (w * dw).sum(1, keepdim=True))
        if case["score"] == "sigmoid":
            c = c * (1.0 - q)
        dl = torch.zeros_like(x).scatter_(1, idx, c)
    elif case["score"] == "sigmoid":
        dl = torch.zeros_like(x).scatter_(1, idx, dw * q * (1.0 - q))
    else:
        dl = torch.zeros_like(x).scatter_(1, idx, dw * q) - p * (q * dw).sum(1, keepdim=True)
    return dw, dl.to(st["logits"].dtype)


# --------------------------------------------------------------------- run

def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "act":
        return _act_fwd(st, case) if case["dir"] == "fwd" else _act_bwd(st, case)
    if case["op"] == "few":
        return _few(st, case)
    return _router_fwd(st, case) if case["dir"] == "fwd" else _router_bwd(st, case)


def _run_own(st, case):
    import moe_fp8_grouped_b200 as gm
    if case["op"] == "act" and case["dir"] == "fwd":
        out = gm.gmm_fwd_act(st["lhs"], st["rhs"], st["rhs_scales"], st["group_sizes"], act=case["act"],
                             bias=st["bias"], residual=st["residual"], rule=case["rule"],
                             static_scale=st["static_scale"] if case["rule"] == "static" else None,
                             transpose_rhs=case["trans"], keep_preact=case["keep"])
        return out
    if case["op"] == "act":
        dz, dbias = gm.gmm_act_bwd(st["dout"], st["z"], st["group_sizes"], act=case["act"], with_dbias=case["bias"])
        return (dz, dbias) if case["bias"] else dz
    if case["op"] == "few":
        return gm.gmm_moe_few(st["x"], st["ids"], st["weights"], st["w1"], st["s1"], st["w2"], st["s2"],
                              transpose_rhs=case["trans"])
    if case["dir"] == "fwd":
        return gm.gmm_router_topk(st["logits"], case["k"], score=case["score"], select_bias=st["select_bias"],
                                  normalize=case["normalize"])
    dw = gm.gmm_combine_dweight(st["dy"], st["rows"], st["slot"])
    return dw, gm.gmm_router_topk_bwd(dw, st["logits"], st["ids"], score=case["score"], normalize=case["normalize"])


# -------------------------------------------------------------------- work

def work(case):
    """Bytes and FLOPs of one pass, each input read and each output written once."""
    if case["op"] == "act":
        G, M, N = case["G"], case["M"], case["N"]
        out_n = N // 2 if case["act"] == "swiglu" else N
        if case["dir"] == "fwd":
            el = 2 if case["rule"] == "none" else 1
            used = min(G, M)  # groups that can have rows at all
            b = M * case["K"] * 2 + used * case["K"] * N * el + (0 if el == 2 else 4 * used * N)
            b += 4 * used * N * case["bias"] + 2 * M * out_n * (1 + case["residual"]) + 2 * M * N * case["keep"]
            return {"bytes": b, "flops": 2 * M * case["K"] * N}
        return {"bytes": 2 * M * out_n + 4 * M * N + 4 * G * N * case["bias"], "flops": 12 * M * N}
    if case["op"] == "few":
        T, k, G, K, F, N = (case[c] for c in ("T", "k", "G", "K", "F", "N"))
        el = 1 if case["weights"] == "e4m3" else 2
        active = G * (1.0 - (1.0 - k / G) ** T)  # experts that a batch of this size reaches
        each = (K * 2 * F + F * N) * el + (4 * (2 * F + N) if el == 1 else 0)
        return {"bytes": int(active * each) + 2 * T * (K + N) + 8 * T * k, "flops": 2 * T * k * (2 * K * F + F * N)}
    T, E, k = case["T"], case["E"], case["k"]
    el = 4 if case["dtype"] == "f32" else 2
    if case["dir"] == "fwd":
        return {"bytes": T * E * el + 8 * T * k + 4 * E * case["select_bias"], "flops": 8 * T * E}
    read = T * E * el if case["score"] == "softmax" and not case["normalize"] else T * k * el
    return {"bytes": 2 * T * case["N"] * (k + 1) + 12 * T * k + read + T * E * el,
            "flops": 2 * T * k * case["N"] + 6 * T * E}


# ------------------------------------------------------------------- exact

def _exact_codes(x, inv):
    """E4M3 values of fl32(x * inv), worked out from the format: a step of
    2^(e - 3) between 2^e and 2^(e + 1), 2^-9 below 2^-6, nearest even."""
    v = (x.float() * inv).double().clamp(-FP8_MAX, FP8_MAX)
    _, e = torch.frexp(v)  # v = m * 2^e, 0.5 <= |m| < 1
    step = torch.ldexp(torch.ones_like(v), (e - 4).clamp(min=-9))
    return torch.round(v / step) * step


def _exact_e4m3(codes):
    """Value of each E4M3 byte."""
    c = torch.arange(256, device="cuda")
    ex, m, sign = (c >> 3) & 15, (c & 7).double(), 1.0 - 2.0 * (c >> 7).double()
    table = sign * torch.where(ex == 0, m * 2.0 ** -9, torch.ldexp(1.0 + m / 8.0, ex - 7))
    return table[codes.long()]


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    f = z.shape[1] // 2
    return z[:, :f] * torch.special.expit(z[:, :f]) * z[:, f:]


def _exact_dact(z, act):
    """d act(z) / dz of the one-input activations."""
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.special.expit(z)
        return s + z * s * torch.special.expit(-z)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2.0 * math.pi)
    u = 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    du = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3 * 0.044715 * z ** 2)
    s = torch.special.expit(u)
    return s + z * s * torch.special.expit(-u) * du


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "act":
        G, M, N = case["G"], case["M"], case["N"]
        if case["dir"] == "fwd":
            x, rule = st["lhs"], case["rule"]
            if rule == "none":
                a = x.double()
            elif rule == "static":
                s = st["static_scale"]
                a = _exact_codes(x, 1.0 / s) * s.double()
            else:
                b = x.float().view(M, -1, 128)
                s = b.abs().amax(2, keepdim=True) / FP8_MAX
                a = (_exact_codes(b, torch.where(s > 0, 1.0 / s, torch.zeros_like(s))) * s.double()).view(M, -1)
            z = torch.zeros((M, N), dtype=torch.float64, device="cuda")
            ends = [sum(st["sizes"][:e + 1]) for e in range(G)]
            for e in range(G):
                lo, hi = (ends[e - 1] if e else 0), ends[e]
                if hi == lo:
                    continue
                w = st["rhs"][e].double() if rule == "none" else _exact_e4m3(st["rhs"][e])
                z[lo:hi] = torch.matmul(a[lo:hi], w.T if case["trans"] else w)
                if rule != "none":
                    z[lo:hi] *= st["rhs_scales"][e].double()
                if case["bias"]:
                    z[lo:hi] += st["bias"][e].double()
            out = _exact_act(z, case["act"])
            if case["residual"]:
                out[:ends[-1]] += st["residual"][:ends[-1]].double()
            return (out, z) if case["keep"] else out
        z, d = st["z"].double(), st["dout"].double()
        if case["act"] == "swiglu":
            f = N // 2
            dz = torch.cat([d * z[:, f:] * _exact_dact(z[:, :f], "silu"), d * _exact_act(z[:, :f], "silu")], 1)
        else:
            dz = d * _exact_dact(z, case["act"])
        rows = sum(st["sizes"])
        dz[rows:] = 0.0
        if not case["bias"]:
            return dz
        db = torch.zeros((G, N), dtype=torch.float64, device="cuda")
        lo = 0
        for e, n in enumerate(st["sizes"]):
            db[e] = dz[lo:lo + n].sum(0)
            lo += n
        return dz, db
    if case["op"] == "few":
        T, k = case["T"], case["k"]
        y = torch.zeros((T, case["N"]), dtype=torch.float64, device="cuda")
        ids = st["ids"].tolist()
        for e in sorted({i for r in ids for i in r}):
            at = [(t, j) for t in range(T) for j in range(k) if ids[t][j] == e]
            t_ = torch.tensor([t for t, _ in at], device="cuda")
            j_ = torch.tensor([j for _, j in at], device="cuda")
            one = (lambda w: w[e].double()) if case["weights"] == "bf16" else (lambda w: _exact_e4m3(w[e]))
            w1, w2 = one(st["w1"]), one(st["w2"])
            h = torch.matmul(st["x"][t_].double(), w1.T if case["trans"] else w1)
            if st["s1"] is not None:
                h *= st["s1"][e].double()
            v = torch.matmul(_exact_act(h, "swiglu"), w2.T if case["trans"] else w2)
            if st["s2"] is not None:
                v *= st["s2"][e].double()
            y.index_add_(0, t_, v * st["weights"][t_, j_].double()[:, None])
        return y
    T, E, k = case["T"], case["E"], case["k"]
    x = st["logits"].double()
    p = torch.special.expit(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    if case["dir"] == "fwd":
        key = x if st["select_bias"] is None else p + st["select_bias"].double()
        key = key.masked_fill(torch.isinf(x), -math.inf)
        ids = torch.argsort(-key, dim=1, stable=True)[:, :k]
        w = p.gather(1, ids)
        return ids.to(torch.int32), w / w.sum(1, keepdim=True) if case["normalize"] else w
    rows = st["rows"].double()[st["slot"].long()]
    dw = torch.einsum("tn,tkn->tk", st["dy"].double(), rows)
    leaf = x.clone().requires_grad_(True)
    p = torch.special.expit(leaf) if case["score"] == "sigmoid" else torch.softmax(leaf, 1)
    w = p.gather(1, st["ids"].long())
    if case["normalize"]:
        w = w / w.sum(1, keepdim=True)
    return dw, torch.autograd.grad((w * dw).sum(), leaf)[0]
