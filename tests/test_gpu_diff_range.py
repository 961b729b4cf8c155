"""Differential attention over the range of its inputs (CUDA path through the C
ABI): rising scores with values near the type's largest."""
import numpy as np
import pytest
import torch

import workloads
from tests.gpu_helpers import lib
from tests.test_gpu_diff_weights import check

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def agb():
    return lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("step", [0.5, 4.0, 5.5, 27.0])
@pytest.mark.parametrize("n", [2, 12, 200])
def test_rising_scores_with_large_values(agb, dtype, step, n):
    # scores that rise by `step` an edge up to 60, values of 1e32: n 2^8 times them stays below the largest number
    N, heads, d = n + 1, 2, 4
    Q, K, V, G = (workloads.features(N, 2 * heads * d, torch.float32, k, DEV) for k in range(4))
    first = torch.arange(0, 2 * heads * d, d, device=DEV)
    Q[:] = 0
    Q[:, first] = 1.0
    K[:, first] = (torch.arange(N, device=DEV) * step).clamp(max=60.0)[:, None].expand(-1, first.numel())
    V, G = V * 1e32, G * 1e-30
    lam = torch.tensor([0.3, 0.7], device=DEV)
    check(agb, np.arange(n), np.full(n, n), N, *(x.to(dtype) for x in (Q, K, V, G)), lam, 1.0)
