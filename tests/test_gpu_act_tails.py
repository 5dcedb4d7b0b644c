"""The activations of gmm_fwd_act far out on the negative side, where their
values are tiny and only a relative error says something: fp32 outputs of z that
are exact (one-hot rows pick single bf16 weights).

Relative bounds.  2^x and 1 / x come within 2 ulp and 1 ulp and the fit of
the Gaussian tail within 4.2e-7: 1e-6 with the multiplications.  The rounding of
an exponent w to fp32, and of its product with log2(e), costs a few 2^-24 of
|w|: |w| = |z| for SiLU (2 roundings), z^2 / 2 for GELU (3),
2 sqrt(2 / pi) |z + 0.044715 z^3| for the tanh form (5)."""
import math

import pytest
import torch

import moe_fp8_grouped_b200 as gm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("act,far", [("silu", 80.0), ("gelu", 12.0), ("gelu_tanh", 7.0)])
def test_tails_keep_their_relative_error(act, far):
    K, N = 128, 1024
    z = -(torch.rand(K, N, generator=torch.Generator().manual_seed(6)) * far + 0.01).bfloat16()
    out = gm.gmm_fwd_act(torch.eye(K).bfloat16().to(DEV), z[None].to(DEV), None,
                         torch.tensor([K], dtype=torch.int32, device=DEV), act=act, rule="none",
                         out_dtype=torch.float32)
    d = z.double()
    if act == "silu":
        w, roundings, ref = d.abs(), 2, d * torch.special.expit(d)
    elif act == "gelu":
        w, roundings, ref = d * d / 2, 3, d * 0.5 * torch.special.erfc(-d / math.sqrt(2))
    else:
        w = 2 * math.sqrt(2 / math.pi) * (d + 0.044715 * d ** 3).abs()
        roundings, ref = 5, d * torch.special.expit(-w)
    err = (out.double().cpu() - ref).abs() / ref.abs()
    assert bool((err <= 1e-6 + roundings * 2.0 ** -24 * w).all()), float((err / (1e-6 + roundings * 2.0 ** -24 * w)).max())
