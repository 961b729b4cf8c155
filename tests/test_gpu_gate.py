"""The gate of the norm block over its whole range (CUDA path through the C ABI).

With U = 2^-24 the logistic function is off by (2 |x| + 9) U, relative, down to
x = -87.3 and 0 below, where it is less than 2^-126; its norm of a row of ones is
1 within 4 U, and three products round (4 U more).  SiLU's slope sums two terms
of at most (1 + |x|) times that.
"""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import assert_within, host, lib
from tests.layer_oracle import U, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def agb():
    return lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("H", [1024, 1023])
def test_gate_and_slope(agb, H, act, dtype):
    x = torch.cat([torch.linspace(-104, 104, 7 * H), torch.linspace(-1e-3, 1e-3, H - 4), torch.tensor([0.0, -1e30, 1e30, -87.25])])
    G = x.view(8, H).to(dtype).to(DEV)
    B = torch.ones_like(G)
    X, _ = agb.ag_resnorm_fwd(None, B, G, act=act, eps=0.0, next_norm=False)
    d = agb.ag_resnorm_backward(X, B, G, B, None, act=act, eps=0.0)
    torch.cuda.synchronize()
    g = host(G).astype(np.float64)
    e = np.exp(-np.abs(g))
    up, down = 1 / (1 + e), e / (1 + e)
    s, t = np.where(g >= 0, up, down), np.where(g >= 0, down, up)      # the function of x and of -x
    size = np.minimum(np.abs(g), 200.0)                                # (below, both sides are 0 or 1)
    rel = (2 * size + 17) * U
    silu = act == "silu"
    want = g * s if silu else s
    assert_within(X, want, rel * np.abs(want) + TINY * (1 + size) + half_step(dtype) * np.abs(want), 1.0, "gate")
    # 1 - s is taken from the rounded s: U besides
    slope = s + g * s * t if silu else s * t
    terms = s + np.abs(g * s) * (t + U) if silu else s * (t + U)
    err = (rel + 4 * U) * terms + (U + rel * s) * s * (size + 1 if silu else 1)
    assert_within(d["G"], slope, err + TINY * (1 + size) + half_step(dtype) * np.abs(slope), 1.0, "slope")
