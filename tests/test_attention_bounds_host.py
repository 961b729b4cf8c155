"""The weighted bounds' 64-bit reference against the layer oracle (CPU), and a
mistake of the kind they are for, planted in an fp32 copy of the arithmetic."""
import numpy as np
import pytest
import torch

from tests import attention_bounds as ab
from tests import layer_oracle as lo


def _case(seed, N=40, E=200, h=2, d=3):
    rng = np.random.default_rng(seed)
    src, dst = rng.integers(0, N, E), rng.integers(0, N - 3, E)
    x = [rng.standard_normal((N, 2 * h * d)) for _ in range(4)]
    return src, dst, N, x, rng.uniform(0.2, 0.8, h), lo.drop_factors(E * h, 0.3, 9, 1).reshape(E, h)


def test_reference_is_the_oracle():
    src, dst, N, x, lam, u = _case(0)
    want = lo.diff_attention(src, dst, N, *x[:3], lam, 0.6, u, x[3])
    t = torch.as_tensor
    got = ab.reference(t(src), t(dst), N, *(t(m) for m in x[:3]), t(lam), 0.6, t(u), t(x[3]))
    for name in ("Y", "lse", "dQ", "dK", "dV", "dlam"):
        np.testing.assert_allclose(got[name].numpy(), want[name], rtol=1e-12, atol=1e-12)
    for dtype, at_most in ((torch.float32, 2e-4), (torch.bfloat16, 0.02)):
        b = ab.bounds(t(src), t(dst), N, *(t(m) for m in x[:3]), t(lam), 0.6, t(u), got, dtype, t(x[3]))
        for name in ("Y", "dQ", "dK", "dV", "dlam"):
            assert b[name].shape == got[name].shape and bool((b[name] >= 0).all())
            assert float(b[name].max()) < at_most * float(got[name].abs().max()), name


@pytest.mark.parametrize("big", [1e4, 1e6])
def test_bound_of_dq_shows_a_reference_without_weight(big):
    # one row, its first edge of weight e^-25 with da = big: sums about that da in fp32 leave
    # the bound, sums about 0 stay inside
    n, d = 64, 4
    rng = np.random.default_rng(1)
    K, V = rng.standard_normal((n, 2 * d)), rng.standard_normal((n, 2 * d))
    K[:, 0] = K[:, d] = rng.uniform(-1, 1, n)
    K[0, 0] = K[0, d] = -25.0
    V[0] = big
    Q, dY = np.zeros((n, 2 * d)), rng.standard_normal((n, 2 * d))
    Q[:, 0] = Q[:, d] = 1.0
    f = lambda m: torch.as_tensor(m.astype(np.float32))
    K, V, Q, dY = f(K), f(V), f(Q), f(dY)
    src, dst = torch.arange(n), torch.zeros(n, dtype=torch.int64)
    lam = torch.tensor([0.5], dtype=torch.float64)
    args = (src, dst, n, Q.double(), K.double(), V.double(), lam, 1.0)
    ref = ab.reference(*args, None, dY.double())
    bound = ab.bounds(*args, None, ref, torch.float32, dY.double())["dQ"][0, :d]
    a = torch.softmax(K[:, 0], 0)
    da = (V * dY[0]).sum(1)

    def sums(c):
        A, B, D = torch.zeros(d), torch.zeros(d), torch.zeros(())
        for e in range(n):
            A, B, D = A + a[e] * (da[e] - c) * K[e, :d], B + a[e] * K[e, :d], D + a[e] * (da[e] - c)
        return ((A - D * B).double() - ref["dQ"][0, :d]).abs()
    assert bool((sums(da[0]) > bound).any()) and bool((sums(torch.zeros(())) <= bound).all())
