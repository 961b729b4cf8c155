"""Differential attention where an edge's weight and its values are far apart
(CUDA path through the C ABI), against 64 bits with bounds that weigh the edges
(attention_bounds)."""
import numpy as np
import pytest
import torch

import workloads
from tests import attention_bounds as ab
from tests.gpu_helpers import assert_within, bits, host, lib

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def agb():
    return lib()


def check(agb, src, dst, N, Q, K, V, G, lam, scale, drop=None, u=None):
    """Forward and backward against `bounds`, twice with the same bits; returns the graph."""
    drop = drop or {}
    s, t = (torch.as_tensor(np.asarray(x), dtype=torch.int64).to(DEV) for x in (src, dst))
    g = agb.ag_graph_lower(s.int(), t.int(), N)
    run = lambda: (lambda Y, lse: (Y, lse) + agb.ag_diff_attn_backward(g, Q, K, V, lam, scale, lse, G, **drop))(
        *agb.ag_diff_attn_fwd(g, Q, K, V, lam, scale, **drop))
    got, again = run(), run()
    torch.cuda.synchronize()
    args = (s, t, N, *(x.double() for x in (Q, K, V)), lam.double(), float(np.float32(scale)))
    u = None if u is None else torch.as_tensor(u).to(DEV)
    ref = ab.reference(*args, u, G.double())
    bound = ab.bounds(*args, u, ref, Q.dtype, G.double())
    for name, x, y in zip(("Y", "lse", "dQ", "dK", "dV", "dlam"), got, again):
        assert torch.equal(bits(x), bits(y)), name
        r, b = (m[name].reshape(x.shape) for m in (ref, bound))
        fin = torch.isfinite(r)
        assert torch.equal(torch.isfinite(x), fin), name
        assert_within(x[fin], host(r[fin]), host(b[fin]), 1.0, name)
    return g


def _uneven(heads, d, dtype, big, seed):
    """Rows that open with edges of negligible weight and large values: nodes
    0 .. 4 have scores -6 (j + 1) and values of size big^((j + 1) / 5), the others
    scores in [-1, 1].  Rows of 6, 40 and 64 edges, and of 700 and 5,000, which
    tiles cut (with such edges in their midst too)."""
    rng = np.random.default_rng(seed)
    N, light = 300, np.arange(5)
    dst, src = [], []
    for row, n in enumerate([6, 40, 64, 64, 700, 5000, 6, 7, 8, 9, 33, 34, 35]):
        e = rng.integers(5, N, n)
        e[:5 if row % 2 else 1] = light[::-1][:5 if row % 2 else 1]
        if n > 100:
            e[rng.integers(40, n, 6)] = rng.integers(0, 5, 6)
        src.append(e)
        dst.append(np.full(n, 20 + 3 * row))
    src, dst = np.concatenate(src), np.concatenate(dst)
    H = 2 * heads * d
    Q, K, V, G = (workloads.features(N, H, torch.float32, seed * 10 + k, DEV) for k in range(4))
    first = torch.arange(0, H, d, device=DEV)                      # a map's first column
    Q[:] = 0
    Q[:, first] = 1.0
    K[:, first] = torch.rand(N, 2 * heads, generator=torch.Generator().manual_seed(seed)).to(DEV) * 2 - 1
    for j in range(5):
        K[j, first] = -6.0 * (j + 1)
        V[j] *= big ** ((j + 1) / 5)
    lam = torch.linspace(0.3, 0.7, heads, device=DEV)
    return src, dst, N, *(x.to(dtype) for x in (Q, K, V, G)), lam


@pytest.mark.parametrize("big", [1.0, 1e3, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("heads,d,dtype", [(1, 4, torch.float32), (2, 16, torch.float32), (1, 3, torch.float32),
                                           (4, 64, torch.float32), (4, 16, torch.bfloat16), (2, 5, torch.bfloat16)])
def test_large_values_on_edges_without_weight(agb, heads, d, dtype, big):
    check(agb, *_uneven(heads, d, dtype, big, 3), 1.0)


@pytest.mark.parametrize("n", [1, 2, 3, 31, 33, 4000])
def test_equal_weights_and_one_large_value(agb, n):
    # the first of n edges of one weight holds all of the value
    V = workloads.features(n + 1, 8, torch.float32, 2, DEV)
    V[0] *= 1e4
    K, G = (workloads.features(n + 1, 8, torch.float32, k, DEV) for k in (1, 3))
    check(agb, np.arange(n), np.full(n, n), n + 1, torch.zeros_like(K), K, V, G, torch.full((1,), 0.5, device=DEV), 1.0)


@pytest.mark.parametrize("offset", [10.0, 1e3])
@pytest.mark.parametrize("n", [2, 5, 40, 3000])
def test_values_that_lie_close_together(agb, n, offset):
    # every da of a row is offset sum(dY) and a little: what cancels in dQ is as large as D itself
    N = 300
    rng = np.random.default_rng(n)
    Q, K, V, G = (workloads.features(N, 32, torch.float32, k, DEV) for k in range(4))
    check(agb, rng.integers(0, N, n), np.full(n, 7), N, Q, K, V + offset, G, torch.tensor([0.3, 0.7], device=DEV), 0.35)


def test_one_edge_rows_have_no_gradient_of_scores(agb):
    # a softmax of one edge is 1 whatever its score: dQ is exactly 0
    N = 500
    src, dst = (torch.as_tensor(x).int().to(DEV) for x in (np.random.default_rng(0).integers(0, N, N), np.arange(N)))
    g = agb.ag_graph_lower(src, dst, N)
    Q, K, V, G = (workloads.features(N, 32, torch.float32, k, DEV) for k in range(4))
    lam = torch.full((2,), 0.5, device=DEV)
    _, lse = agb.ag_diff_attn_fwd(g, Q, K, V, lam, 0.3)
    dQ = agb.ag_diff_attn_backward(g, Q, K, V, lam, 0.3, lse, G)[0]
    torch.cuda.synchronize()
    assert not dQ.any()
