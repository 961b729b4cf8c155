"""Row-wise outputs that lie on inputs (CUDA path through the C ABI)."""
import pytest
import torch

import workloads
from tests.gpu_helpers import lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def agb():
    return lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("N,heads,D,rot", [(1, 1, 8, 8), (333, 4, 16, 8), (40, 3, 7, 6), (9, 1, 4200, 4096)])
def test_rotary_outputs_on_the_other_matrix(agb, N, heads, D, rot, interleaved, dtype):
    Q, K = (workloads.features(N, heads * D, dtype, k, DEV) for k in range(2))
    pos, freq = torch.arange(N, device=DEV) * 77, agb.ag_rotary_freqs(rot)[0].to(DEV)
    want = agb.ag_rotary(Q, K, pos, freq, heads, interleaved=interleaved)
    a, b = Q.clone(), K.clone()
    agb.ag_rotary(a, b, pos, freq, heads, interleaved=interleaved, Qo=b, Ko=a)
    torch.cuda.synchronize()
    assert torch.equal(b, want[0]) and torch.equal(a, want[1])


def test_a_row_on_its_own_vector_is_refused(agb):
    # one row is as long as a vector, which the kernel may read again after it has written the row
    B, g = torch.randn(1, 4096, device=DEV), torch.ones(4096, device=DEV)
    for kw in (dict(X=g.view(1, -1)), dict(Z=g.view(1, -1))):
        for name in ("gamma1", "beta1", "scale", "gamma2", "beta2"):
            with pytest.raises(agb.AggraphError, match="overlaps"):
                agb.ag_resnorm_fwd(None, B, **{name: g}, **kw)
    X = B.clone()
    assert agb.ag_resnorm_fwd(None, X, gamma1=g, X=X)[0] is X
    torch.cuda.synchronize()
