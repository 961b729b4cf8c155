"""Infinities and NaN where dropout has dropped: they reach no output that the
kept ones do not (CUDA path through the C ABI)."""
import numpy as np
import pytest
import torch

import workloads
from tests import layer_oracle as lo
from tests.gpu_helpers import host, lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
VALUES = [float("nan"), float("inf"), -float("inf")]


@pytest.fixture(scope="module")
def agb():
    return lib()


def _graph(agb, heads, seed, hub=0):
    """A graph of few edges a row, its dropout, and per edge whether no head keeps it."""
    rng = np.random.default_rng(seed)
    N, E = 400, 700
    src = np.concatenate([rng.integers(0, N, E), rng.integers(0, N, hub)])
    dst = np.concatenate([rng.integers(0, N, E), np.full(hub, 7)])
    g = agb.ag_graph_lower(*(torch.as_tensor(x.astype(np.int32)).to(DEV) for x in (src, dst)), N)
    drop = dict(p=0.7, seed=seed, offset=2)
    gone = ~lo.keep_mask(len(src) * heads, 0.7, seed, 2).reshape(-1, heads).any(1)
    return src, dst, N, g, drop, gone


def _all_gone(index, gone, N):
    """Nodes of at least one edge, all of whose edges are dropped."""
    n = np.bincount(index, minlength=N)
    return np.flatnonzero((n > 0) & (np.bincount(index, weights=gone, minlength=N) == n))


CASES = [(1, 4, torch.float32), (2, 8, torch.float32), (1, 3, torch.float32), (2, 16, torch.bfloat16), (1, 5, torch.bfloat16),
         (2, 33, torch.float32)]


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("heads,d,dtype", CASES)
def test_values_of_dropped_edges(agb, heads, d, dtype, value):
    # V rows whose every edge is dropped: forward and backward as with zeros there
    src, dst, N, g, drop, gone = _graph(agb, heads, 3, hub=600)
    nodes = _all_gone(src, gone, N)
    assert len(nodes) > 10
    Q, K, V, G = (workloads.features(N, 2 * heads * d, dtype, k, DEV) for k in range(4))
    lam = torch.linspace(0.3, 0.7, heads, device=DEV)
    outs = []
    for fill in (0.0, value):
        V[nodes] = fill
        Y, lse = agb.ag_diff_attn_fwd(g, Q, K, V, lam, 0.4, **drop)
        outs.append((Y, lse) + agb.ag_diff_attn_backward(g, Q, K, V, lam, 0.4, lse, G, **drop))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("heads,d,dtype", CASES)
def test_output_gradients_of_dropped_edges(agb, heads, d, dtype, value):
    src, dst, N, g, drop, gone = _graph(agb, heads, 4, hub=600)
    Q, K, V, G = (workloads.features(N, 2 * heads * d, dtype, k, DEV) for k in range(4))
    lam = torch.linspace(0.3, 0.7, heads, device=DEV)
    _, lse = agb.ag_diff_attn_fwd(g, Q, K, V, lam, 0.4, **drop)
    back = lambda: agb.ag_diff_attn_backward(g, Q, K, V, lam, 0.4, lse, G, **drop)
    # dY rows whose every edge is dropped: every gradient as with zeros there
    rows = _all_gone(dst, gone, N)
    assert len(rows) > 10
    G[rows] = 0.0
    want = back()
    G[rows] = value
    got = back()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # rows of kept and dropped edges, the hub among them: dV of the sources whose edges there are dropped
    G[rows] = 0.0
    mixed = np.append(np.setdiff1d(np.unique(dst), rows)[::5], 7)
    reached = np.unique(src[np.isin(dst, mixed) & ~gone])
    clean = np.setdiff1d(np.unique(src[np.isin(dst, mixed) & gone]), reached)
    assert len(clean) > 20
    G[mixed] = 0.0
    want = back()
    G[mixed] = value
    got = back()
    torch.cuda.synchronize()
    assert torch.equal(want[2][clean], got[2][clean])
    assert not bool(torch.isfinite(got[2][reached].float()).all())


@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("H,dtype", [(16, torch.float32), (33, torch.float32), (256, torch.float32), (2048, torch.float32),
                                     (64, torch.bfloat16), (100, torch.bfloat16), (2050, torch.bfloat16), (8192, torch.bfloat16)])
def test_gates_of_dropped_elements(agb, H, dtype, act, value):
    # a gate that is infinite or NaN where its element is dropped: every output and gradient as with zeros there
    N = 37
    R, B, G, dX, dZ = (workloads.features(N, H, dtype, k, DEV) for k in range(5))
    gen = torch.Generator().manual_seed(1)
    v = {k: (0.5 + torch.rand(H, generator=gen)).to(DEV) for k in ("gamma1", "beta1", "scale", "gamma2", "beta2")}
    kw = dict(norm="layer", act=act, p=0.3, seed=8, offset=1, **v)
    gone = torch.as_tensor(~lo.keep_mask(N * H, 0.3, 8, 1).reshape(N, H)).to(DEV)
    outs = []
    for fill in (0.0, value):
        G = torch.where(gone, torch.tensor(fill, dtype=dtype, device=DEV), G)
        X, Z = agb.ag_resnorm_fwd(R, B, G, **kw)
        d = agb.ag_resnorm_backward(X, B, G, dX, dZ, **kw)
        outs.append([X, Z] + [d[k] for k in sorted(d)])
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert bool(torch.isfinite(a.float()).all()) and torch.equal(a, b)
