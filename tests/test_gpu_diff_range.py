"""Differential attention over the range of its inputs (CUDA path through the C
ABI): rising scores with values near the type's largest, large scores through
the backward pass, infinities, and the longest tiles."""
import numpy as np
import pytest
import torch

import workloads
from tests import attention_bounds as ab
from tests import layer_oracle as lo
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("factor,scale", [(64.0, 8.0), (0.0, 1.0), (8.0, 1.0)])
def test_large_and_equal_scores_through_the_backward_pass(agb, dtype, factor, scale):
    # scores of several thousand, of several hundred, and rows of equal scores; with rows of one edge
    rng = np.random.default_rng(4)
    N, E = 300, 2500
    src, dst = rng.integers(0, N, E + 60), np.concatenate([rng.integers(0, 200, E), np.arange(220, 280)])
    Q, K, V, G = (workloads.features(N, 32, dtype, k, DEV) for k in range(4))
    check(agb, src, dst, N, (Q.float() * factor).to(dtype), K, V, G, torch.tensor([0.3, 0.7], device=DEV), scale)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_key(agb, sign):
    # edges 0 -> 5, 1 -> 5, 2 -> 6 with K[1, 0] infinite: a score of +inf makes map 1 of row 5 NaN,
    # one of -inf has weight 0 there; row 6 keeps its bits
    g = agb.ag_graph_lower(*(torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1, 2], [5, 5, 6])), 8)
    Q, K, V, G = (workloads.features(8, 8, torch.float32, k, DEV) for k in range(4))
    lam = torch.tensor([0.5], device=DEV)
    Q[5, 0] = sign
    clean, _ = agb.ag_diff_attn_fwd(g, Q, K, V, lam, 0.5)
    bad, far = K.clone(), K.clone()
    bad[1, 0], far[1, 0] = float("inf"), 1e6                  # a score of -5e5 has weight 0 too
    Y, lse = agb.ag_diff_attn_fwd(g, Q, bad, V, lam, 0.5)
    torch.cuda.synchronize()
    rest = [r for r in range(8) if r != 5]
    assert torch.equal(Y[rest], clean[rest])
    if sign > 0:
        assert bool(torch.isnan(Y[5]).all())
        return
    args = (torch.tensor([0, 1, 2], device=DEV), torch.tensor([5, 5, 6], device=DEV), 8, Q.double(), far.double(), V.double(),
            lam.double(), 0.5)
    ref = ab.reference(*args)
    assert float(ref["a"][1, 0, 0]) == 0.0
    # weights of 1 and 0, and a second map of 4 products: 64 U of the terms |V|
    assert bool(((Y[5].double() - ref["Y"][5]).abs() <= 64 * ab.U * (V[0].abs() + V[1].abs())).all())
    assert abs(float(lse[5, 0, 0]) - float(ref["lse"][5, 0, 0])) <= 64 * ab.U


@pytest.mark.parametrize("E,tile,p", [(2_200_000, 512, 0.1), (4_300_000, 1024, 0.0)])
def test_the_longest_joined_tiles(agb, E, tile, p):
    # one lane group per warp (4 heads of 8 lanes), so that the walks join tiles of the schedule up to `tile`
    # positions while 4,144 of them are left; hubs on both sides that are cut into many of them
    rng = np.random.default_rng(31)
    N = 70_000
    src, dst = rng.integers(0, N, E), rng.integers(0, N - 50, E)
    dst[rng.permutation(E)[:30_000]] = 11
    src[rng.permutation(E)[:40_000]] = N - 1
    Q, K, V, G = (workloads.features(N, 8, torch.float32, k, DEV) for k in range(4))
    drop = dict(p=p, seed=5, offset=1)
    u = lo.drop_factors(4 * E, p, 5, 1).reshape(E, 4) if p else None
    g = check(agb, src, dst, N, Q, K, V, G, torch.linspace(0.2, 0.8, 4, device=DEV), 1.0, drop, u)
    assert 4144 * tile <= g.stats["tiles"] * g.stats["tile_edges"] and tile > g.stats["tile_edges"]
    assert g.stats["max_degree_f"] > 20 * tile


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,d", [(64, 1), (65, 3), (100, 4), (130, 8), (256, 1), (256, 6), (200, 16)])
def test_many_heads(agb, heads, d, dtype):
    # more heads than a block of the walk has threads, and up to the most there may be; rows cut by tiles
    rng = np.random.default_rng(heads)
    N, E, p = 150, 900, 0.2
    src, dst = rng.integers(0, N, E + 200), np.concatenate([rng.integers(0, N - 9, E), np.full(200, 5)])
    Q, K, V, G = (workloads.features(N, 2 * heads * d, dtype, k, DEV) for k in range(4))
    drop = dict(p=p, seed=11, offset=4)
    check(agb, src, dst, N, Q, K, V, G, torch.linspace(0.1, 0.9, heads, device=DEV), d ** -0.5, drop,
          lo.drop_factors((E + 200) * heads, p, 11, 4).reshape(-1, heads))


@pytest.mark.parametrize("scale,lam", [(-0.5, 0.5), (0.0, 0.5), (0.3, 0.0), (0.3, -1.5), (0.3, 4.0)])
def test_signs_of_the_scale_and_of_lambda(agb, scale, lam):
    rng = np.random.default_rng(3)
    N, E = 200, 2000
    src, dst = rng.integers(0, N, E), rng.integers(0, N // 2, E)
    Q, K, V, G = (workloads.features(N, 48, torch.float32, k, DEV) for k in range(4))
    check(agb, src, dst, N, Q, K, V, G, torch.full((3,), lam, device=DEV), scale)


@pytest.mark.parametrize("heads,d,dtype", [(1, 4, torch.float32), (2, 8, torch.float32), (4, 16, torch.bfloat16), (3, 5, torch.bfloat16)])
def test_rows_do_not_depend_on_other_rows(agb, heads, d, dtype):
    # rows of rising scores of 100, and of infinite ones, beside rows of small scores: these keep their bits
    rng = np.random.default_rng(6)
    N, E = 40_000, 400_000
    src, dst = (torch.as_tensor(rng.integers(0, N, E).astype(np.int32)).to(DEV) for _ in range(2))
    g = agb.ag_graph_lower(src, dst, N)
    Q, K, V = (workloads.features(N, 2 * heads * d, dtype, k, DEV) for k in range(3))
    lam = torch.linspace(0.3, 0.7, heads, device=DEV)
    want = agb.ag_diff_attn_fwd(g, Q, K, V, lam, d ** -0.5)
    rest = torch.arange(N, device=DEV) % 3 != 0
    for factor in (50.0, float("inf")):
        got = agb.ag_diff_attn_fwd(g, torch.where(rest[:, None], Q, Q * factor), K, V, lam, d ** -0.5)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[rest], b[rest])
