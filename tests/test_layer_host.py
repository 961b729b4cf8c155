"""The differential attention layer on the CPU: the oracle against published
vectors, differences and plain loops; the frequency table; every refusal that
the library's entry points answer without a GPU."""
import ctypes

import numpy as np
import pytest
import torch

from tests import layer_oracle as lo


@pytest.fixture(scope="module")
def agb():
    from __graft_entry__ import build_library
    build_library()
    import gnn_sparse_aggregation_b200 as m
    return m


@pytest.mark.parametrize("counter,key,want", [
    # the generator's published known-answer vectors
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_oracle_generator_known_answers(counter, key, want):
    got = lo.philox(np.array([counter], np.uint64), np.array([key], np.uint64))[0]
    assert tuple(int(x) for x in got) == want


def test_oracle_mask_keeps_the_asked_share():
    # 2^18 elements: the share's standard deviation is at most 2^-10; five of them
    for p in (0.1, 0.5, 0.9):
        kept = lo.keep_mask(1 << 18, p, 1234567890123, 5)
        assert abs(kept.mean() - (1 - p)) < 5 * 2.0 ** -10
    assert lo.keep_mask(100, 0.3, 1, 2).tolist() == lo.keep_mask(60, 0.3, 1, 2).tolist() + lo.keep_mask(40, 0.3, 1, 2, 60).tolist()


def _small_graph(rng, N=7, E=25):
    return rng.integers(0, N, E), rng.integers(0, N - 1, E), N   # row N - 1 has no edges


def test_oracle_attention_against_a_plain_loop():
    rng = np.random.default_rng(0)
    src, dst, N = _small_graph(rng)
    h, d = 2, 3
    Q, K, V = (rng.standard_normal((N, 2 * h * d)) for _ in range(3))
    lam, scale = rng.uniform(0.2, 0.8, h), 0.7
    u = lo.drop_factors(len(src) * h, 0.3, 9, 1).reshape(-1, h)
    got = lo.diff_attention(src, dst, N, Q, K, V, lam, scale, u)
    for r in range(N):
        edges = [e for e in range(len(src)) if dst[e] == r]
        for j in range(h):
            y = np.zeros(2 * d)
            maps = []
            for m in range(2):
                c = slice((2 * j + m) * d, (2 * j + m + 1) * d)
                s = np.array([scale * Q[r, c] @ K[src[e], c] for e in edges])
                maps.append(np.exp(s) / np.exp(s).sum() if edges else s)
                if edges:
                    assert abs(got["lse"][r, j, m] - np.log(np.exp(s).sum())) < 1e-12
                else:
                    assert got["lse"][r, j, m] == -np.inf
            for i, e in enumerate(edges):
                y += u[e, j] * (maps[0][i] - lam[j] * maps[1][i]) * V[src[e], 2 * d * j: 2 * d * (j + 1)]
            np.testing.assert_allclose(got["Y"][r, 2 * d * j: 2 * d * (j + 1)], y, atol=1e-12)


def test_oracle_attention_gradients_against_differences():
    rng = np.random.default_rng(1)
    src, dst, N = _small_graph(rng)
    h, d = 2, 2
    x = {k: rng.standard_normal((N, 2 * h * d)) for k in ("Q", "K", "V")}
    x["lam"] = rng.uniform(0.2, 0.8, h)
    u = lo.drop_factors(len(src) * h, 0.3, 5, 0).reshape(-1, h)
    G = rng.standard_normal((N, 2 * h * d))
    loss = lambda y: (lo.diff_attention(src, dst, N, y["Q"], y["K"], y["V"], y["lam"], 0.6, u)["Y"] * G).sum()
    ref = lo.diff_attention(src, dst, N, x["Q"], x["K"], x["V"], x["lam"], 0.6, u, G)
    # central differences at step e: e^2 times a third derivative of order 10, and 2^-52 |loss| / e
    e = 1e-5
    for name in x:
        grad = ref["d" + name]
        for i in np.ndindex(x[name].shape):
            y = {k: t.copy() for k, t in x.items()}
            y[name][i] += e
            up = loss(y)
            y[name][i] -= 2 * e
            assert abs((up - loss(y)) / (2 * e) - grad[i]) < 1e-7, (name, i)


def test_frequency_table(agb):
    f, factor = agb.ag_rotary_freqs(8)
    np.testing.assert_allclose(f.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    assert factor == 1.0
    lin, _ = agb.ag_rotary_freqs(8, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin.numpy(), f.numpy() / 4, rtol=1e-15)
    ntk, _ = agb.ag_rotary_freqs(8, scaling="ntk", factor=4.0)
    # the fastest pair stays, the slowest is slowed down by exactly the factor
    np.testing.assert_allclose(ntk.numpy()[[0, -1]], [1.0, 0.001 / 4], rtol=1e-12)
    yarn, factor = agb.ag_rotary_freqs(64, scaling="yarn", factor=8.0, original=4096.0)
    base, _ = agb.ag_rotary_freqs(64)
    ratio = (yarn / base).numpy()
    turns = 4096 * base.numpy() / (2 * np.pi)
    assert np.all(ratio[turns > 2 * 32] == 1.0) and np.allclose(ratio[turns < 0.5], 1 / 8, rtol=1e-15)
    assert np.all(np.diff(ratio) <= 1e-15) and abs(factor - (0.1 * np.log(8.0) + 1)) < 1e-15


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=8192), dict(rot=8, base=-1.0),
                                dict(rot=8, scaling="linear", factor=0.5), dict(rot=8, scaling="ntk", factor=float("nan")),
                                dict(rot=8, scaling="yarn", factor=2.0), dict(rot=8, scaling="other"),
                                dict(rot=8, scaling="yarn", factor=2.0, original=100.0, beta_fast=1.0, beta_slow=2.0)])
def test_frequency_table_refusals(agb, kw):
    with pytest.raises(agb.AggraphError):
        agb.ag_rotary_freqs(**kw)


INVALID, SHAPE, DTYPE, WORKSPACE = 1, 2, 3, 7


def test_dropout_refusals_without_gpu(agb):
    f, p = agb.lib.ag_dropout, ctypes.c_void_p(256)
    assert f(p, p, -1, 0.1, 0, 0, 0, None) == SHAPE
    assert f(p, p, 1 << 40, 0.1, 0, 0, 0, None) == SHAPE
    assert f(p, p, 4, 0.1, 0, 0, 7, None) == DTYPE
    for bad in (-0.1, 1.0, float("nan"), float("inf")):
        assert f(p, p, 4, bad, 0, 0, 0, None) == INVALID
    assert f(None, p, 4, 0.1, 0, 0, 0, None) == INVALID and f(p, None, 4, 0.1, 0, 0, 0, None) == INVALID
    assert f(ctypes.c_void_p(258), p, 4, 0.1, 0, 0, 0, None) == INVALID
    assert f(None, None, 0, 0.1, 0, 0, 0, None) == 0                      # nothing to do


def test_rotary_refusals_without_gpu(agb):
    p = ctypes.c_void_p(256)

    def call(N=4, H=16, heads=2, rot=8, inter=0, factor=1.0, dtype=0, q=p, qo=p, k=None, ko=None, pos=p, freq=p):
        return agb.lib.ag_rotary(q, k, pos, freq, qo, ko, N, H, heads, rot, inter, factor, 0, dtype, None)
    for kw in (dict(N=-1), dict(N=1 << 31), dict(H=0), dict(H=(1 << 20) + 1), dict(heads=0), dict(heads=3), dict(heads=17),
               dict(rot=0), dict(rot=7), dict(rot=10), dict(rot=-2), dict(H=1 << 14, heads=1, rot=8192)):
        assert call(**kw) == SHAPE, kw
    assert call(dtype=2) == DTYPE
    for kw in (dict(factor=float("nan")), dict(q=None), dict(qo=None), dict(pos=None), dict(freq=None), dict(k=p),
               dict(pos=ctypes.c_void_p(260)), dict(q=ctypes.c_void_p(257), dtype=1)):
        assert call(**kw) == INVALID, kw
    assert call(N=0) == 0


def test_diff_attention_refusals_without_gpu(agb):
    lib = agb.lib
    assert lib.ag_diff_attn_fwd(None, *[None] * 4, 1.0, 0.0, 0, 0, None, None, 16, 2, 0, None, 0, None) == INVALID
    assert lib.ag_diff_attn_backward(None, *[None] * 4, 1.0, 0.0, 0, 0, *[None] * 6, 16, 2, 0, None, 0, None) == INVALID
    assert lib.ag_diff_attn_scratch_bytes(None, 16, 2) == 0


def test_resnorm_refusals_without_gpu(agb):
    lib, p = agb.lib, 256
    op = lambda **kw: ctypes.byref(agb.ResNorm(**{**dict(eps=1e-5), **kw}))

    def fwd(o=None, R=p, B=p, G=p, X=p, Z=p, N=4, H=8, dtype=0):
        return lib.ag_resnorm_fwd(op() if o is None else o, R, B, G, X, Z, N, H, dtype, None)
    assert lib.ag_resnorm_fwd(None, p, p, p, p, p, 4, 8, 0, None) == INVALID
    for kw in (dict(N=-1), dict(N=1 << 31), dict(H=0), dict(H=8193)):
        assert fwd(**kw) == SHAPE, kw
    assert fwd(dtype=5) == DTYPE
    for o in (dict(norm=2), dict(norm=-1), dict(act=2), dict(eps=-1.0), dict(eps=float("nan")), dict(p=1.0), dict(p=-0.5),
              dict(gamma1=p + 1)):
        assert fwd(o=op(**o)) == INVALID, o
    for kw in (dict(B=None), dict(B=None, G=None), dict(B=None, G=None, X=None, R=None), dict(X=None),
               dict(X=None, Z=None), dict(R=p + 2)):
        assert fwd(**kw) == INVALID, kw
    assert fwd(N=0) == 0

    def bwd(X=p, B=p, G=p, dX=p, dZ=p, dR=p, dB=p, dG=p, sums=(None,) * 5, scratch=None, size=0, N=4, H=8, dtype=0, o=None):
        return lib.ag_resnorm_backward(op() if o is None else o, X, B, G, dX, dZ, dR, dB, dG, *sums, N, H, dtype, scratch,
                                       size, None)
    for kw in (dict(N=-1), dict(H=8193)):
        assert bwd(**kw) == SHAPE, kw
    assert bwd(dtype=-1) == DTYPE
    for kw in (dict(o=op(p=2.0)), dict(B=None), dict(B=None, G=None, dB=None), dict(G=None), dict(dX=None, dZ=None),
               dict(dZ=None, sums=(None, None, None, p, None)), dict(X=None), dict(dB=None), dict(dR=p + 1),
               dict(B=None, G=None, dB=None, dG=None, sums=(p, None, None, None, None))):
        assert bwd(**kw) == INVALID, kw
    need = lib.ag_resnorm_scratch_bytes(4, 8)
    assert need > 0 and lib.ag_resnorm_scratch_bytes(4, 8193) == 0 and lib.ag_resnorm_scratch_bytes(-1, 8) == 0
    sums = (p,) * 5
    assert bwd(sums=sums) == WORKSPACE
    assert bwd(sums=sums, scratch=p, size=need - 1) == WORKSPACE
    assert bwd(sums=sums, scratch=p + 8, size=need) == WORKSPACE


def test_binding_refuses_cpu_tensors_and_bad_words(agb):
    X = torch.zeros(4, 8)
    for call in (lambda: agb.ag_dropout(X, 0.1, 1), lambda: agb.ag_rotary(X, None, X, X, 1),
                 lambda: agb.ag_resnorm_fwd(X, None), lambda: agb.ag_resnorm_backward(X, None, None, X, None),
                 lambda: agb.ag_resnorm_fwd(None, None)):
        with pytest.raises(agb.AggraphError):
            call()
