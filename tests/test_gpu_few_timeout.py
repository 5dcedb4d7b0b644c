"""A wait of gmm_moe_few that runs out of its limit: the call ends, its status
word reads as a timeout (a report must survive the reset of the word at the
start of the call), and the workspace serves the next call."""
import pytest
import torch

import moe_fp8_grouped_b200 as gm
from moe_fp8_grouped_b200 import _binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TIMEOUT = 8, B.DEV_TIMEOUT  # GMM_ERR_TIMEOUT and its device bit


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_a_wait_that_runs_out_is_reported(kind):
    """The epilogue waits for the sum of a whole tile: 32 MB of weights a CTA,
    at least 0.6 ms at the copy rate of 148 CTAs.  A wait looks at its limit
    (1 ns here) after 64 polls, which take 0.27 ms."""
    T, K, F, N = 2, 1 << 18, 74 * 128, 128
    dt, code = (torch.uint8, B.DT_E4M3) if kind == "e4m3" else (torch.bfloat16, B.DT_BF16)
    one = 0x38 if kind == "e4m3" else 1.0  # E4M3 code of 1
    w1 = torch.zeros(1, K, 2 * F, dtype=dt, device=DEV)
    w1[:, ::1024] = one
    w2 = torch.zeros(1, F, N, dtype=dt, device=DEV)
    w2[:, 0] = one
    s1, s2 = (torch.ones(1, n, device=DEV) if kind == "e4m3" else None for n in (2 * F, N))
    x = torch.full((T, K), 2.0 ** -7, dtype=torch.bfloat16, device=DEV)  # gate = up = 256 * 2^-7 = 2
    ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    wts = torch.ones(T, 1, device=DEV)
    ws = torch.empty(B.lib().gmm_moe_few_workspace_bytes(T, 1, 1, K, F, N, code), dtype=torch.uint8, device=DEV)

    def call():
        return gm.gmm_moe_few(x, ids, wts, w1, s1, w2, s2, out_dtype=torch.float32, ws=ws)

    gm.gmm_set_wait_limit_ns(1)
    try:
        for _ in range(5):
            call()
            assert gm.gmm_read_device_status(ws) == TIMEOUT
    finally:
        gm.gmm_set_wait_limit_ns(0)
    y = call()
    assert gm.gmm_read_device_status(ws) == (0, 0)
    # 4 * sigmoid(2) = 3.5232 rounded to bf16, whose steps are 2^-6 there
    h = (4 * torch.sigmoid(torch.tensor(2.0, dtype=torch.float64))).bfloat16().float()
    assert bool((y == h.item()).all())
