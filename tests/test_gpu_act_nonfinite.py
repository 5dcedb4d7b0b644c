"""gmm_act_bwd where dout is not finite (an overflowed loss scale): the ReLU
gradient is a choice, dz = dout where z > 0 and 0 elsewhere, so an infinite or
NaN dout shows in dz and in its group's bias gradient only where z > 0."""
import math

import pytest
import torch

import moe_fp8_grouped_b200 as gm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("sizes,M", [([3], 4), ([130, 0, 70], 210)])
def test_relu_selects(bad, sizes, M):
    N = 384
    g = torch.Generator().manual_seed(1)
    z = torch.randint(-2, 3, (M, N), generator=g).bfloat16().to(DEV)  # many zeros of either sign
    z[0, 5] = -0.0
    dout = torch.randint(-3, 4, (M, N), generator=g).bfloat16().to(DEV)
    dout[z <= 0] = bad
    z[1, 7] = math.nan  # not above 0: no gradient
    dout[1, 7] = bad
    gs = torch.tensor(sizes, dtype=torch.int32, device=DEV)
    dz, db = gm.gmm_act_bwd(dout, z, gs, act="relu")
    rows = sum(sizes)
    want = torch.where(z > 0, dout, torch.zeros_like(dout))
    want[rows:] = 0
    assert torch.equal(dz, want)
    r = 0
    for i, n in enumerate(sizes):  # sums of small integers: exact
        assert torch.equal(db[i], want[r:r + n].float().sum(0))
        r += n


def test_relu_passes_it_on_where_z_is_positive():
    z = torch.full((2, 128), -1.0, dtype=torch.bfloat16, device=DEV)
    z[0, 3] = z[1, 4] = z[1, 9] = 2.0
    dout = torch.full((2, 128), math.inf, dtype=torch.bfloat16, device=DEV)
    dout[1, 9] = math.nan
    dz, db = gm.gmm_act_bwd(dout, z, torch.tensor([2], dtype=torch.int32, device=DEV), act="relu")
    assert dz[0, 3] == math.inf and dz[1, 4] == math.inf and bool(torch.isnan(dz[1, 9]))
    assert db[0, 3] == math.inf and db[0, 4] == math.inf and bool(torch.isnan(db[0, 9]))
    rest = torch.ones_like(z, dtype=torch.bool)
    rest[0, 3] = rest[1, 4] = rest[1, 9] = False
    assert not bool(dz[rest].any())
