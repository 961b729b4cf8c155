"""Dropout, rotary positions and the norm / gate / residual block (CUDA path
through the C ABI) against the 64-bit oracle.

Bounds, with U = 2^-24 and `half` half a step of the output's type:
  dropout   the factor and the product round once each, then the type:
            (3 U + half) |y|; dropped elements are exactly 0.
  rotary    an angle reduced in fp64 is rounded to fp32 below pi (pi U, and
            2^-50 turns per turn), sincospi is off by 2 steps, the factor, two
            products and a sum round: 16 U factor (|x0| + |x1|) + half |y|.
  resnorm   every output is a short chain of sums whose terms are taken here in
            absolute value (a normalised value as r (|x| + mean |x|), its size
            before the mean cancels).  A chain has at most 2 row sums of depth
            20, and 40 further roundings: 128 U of the absolute sum.  Column
            sums add at most 400 steps over rows, groups and blocks.
"""
import numpy as np
import pytest
import torch

import workloads
from tests import layer_oracle as lo
from tests.gpu_helpers import assert_within, bits, host, lib
from tests.layer_oracle import U, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOTH = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def agb():
    return lib()


def _shifted(t, shift):
    big = torch.zeros(t.numel() + shift, dtype=t.dtype, device=t.device)
    big[shift:].copy_(t.reshape(-1))
    return big[shift:].view(t.shape)


# ------------------------------------------------------------------- dropout

@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 31, 255, 1023, 1025, 100003])
def test_dropout_lengths(agb, n, dtype):
    for shift in (0, 1, 3):
        X = _shifted(workloads.features(1, n, dtype, n, DEV)[0], shift)
        p, seed, offset = 0.3, (1 << 64) - n, (1 << 40) + n
        Y = agb.ag_dropout(X, p, seed, offset)
        torch.cuda.synchronize()
        f = lo.drop_factors(n, p, seed, offset)
        ref = host(X).astype(np.float64) * f
        assert_within(Y, ref, np.abs(ref) * (3 * U + half_step(dtype)), 1.0, f"n {n} shift {shift}")


def test_dropout_matrix_in_place_probabilities_and_masked_values(agb):
    X = workloads.features(333, 40, torch.float32, 5, DEV)
    Y = agb.ag_dropout(X, 0.5, 11)
    keep = torch.as_tensor(lo.keep_mask(X.numel(), 0.5, 11, 0).reshape(X.shape)).to(DEV)
    assert torch.equal(Y != 0, keep)
    for value in (float("nan"), float("inf")):                # what is dropped does not matter
        assert torch.equal(agb.ag_dropout(torch.where(keep, X, torch.tensor(value, device=DEV)), 0.5, 11), Y)
    Z = X.clone()
    assert agb.ag_dropout(Z, 0.5, 11, out=Z) is Z and torch.equal(Z, Y)
    assert torch.equal(agb.ag_dropout(X, 0.0, 11), X)
    assert torch.equal(agb.ag_dropout(X, 1e-12, 11), X)       # round(p 2^32) = 0 keeps all; 1 / (1 - p) = 1 in fp32
    assert not torch.equal(agb.ag_dropout(X, 0.5, 12), Y) and not torch.equal(agb.ag_dropout(X, 0.5, 11, 1), Y)
    near = agb.ag_dropout(X, 1.0 - 2.0 ** -40, 11)            # threshold 2^32 - 1: hardly an element is kept
    assert int((near != 0).sum()) <= 1
    assert agb.ag_dropout(X[:0], 0.5, 11).shape == (0, 40)
    # one gradient: the same call
    torch.testing.assert_close(agb.ag_dropout(torch.ones_like(X), 0.5, 11), keep.float() * 2, rtol=0, atol=0)


def test_dropped_edges_reach_the_aggregation(agb):
    # the weights of dropped edges are 0 and the others' sums are scaled: Y = A_(drop w) X
    import oracle
    wl = workloads.make("uniform", seed=3, device=DEV)
    g = agb.ag_graph_lower(wl.src, wl.dst, wl.N)
    w = agb.ag_dropout(wl.w, 0.4, 21, 3)
    Y = agb.ag_spmm_fwd(g, w, wl.X)
    torch.cuda.synchronize()
    f = lo.drop_factors(wl.E, 0.4, 21, 3)
    ref, bound = oracle.fwd(host(wl.src), host(wl.dst), wl.N, (host(wl.w) * f).astype(np.float32), host(wl.X), with_bound=True)
    assert_within(Y, ref, bound, 1e-5 + 4 * U, "dropped edges")


# ------------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,D,rot", [(1, 2, 2), (3, 2, 2), (2, 6, 2), (2, 6, 4), (1, 7, 6), (2, 8, 8), (4, 16, 8), (2, 16, 16),
                                         (3, 20, 10), (8, 16, 4), (2, 24, 12), (16, 64, 32), (1, 128, 128), (5, 100, 50),
                                         (1, 300, 300), (1, 5000, 4096)])
def test_rotary_sizes(agb, heads, D, rot, interleaved, dtype):
    N = 9 if D > 1000 else 157
    rng = np.random.default_rng(heads * D + rot)
    pos = rng.integers(-(1 << 20), 1 << 31, N)
    pos[:3] = (0, 1, -1)
    freq, _ = agb.ag_rotary_freqs(rot, scaling="linear", factor=2.0)
    for shift, inverse, factor in ((0, False, 1.0), (0, True, 1.25), (1, False, 1.25)):
        Q, K = (_shifted(workloads.features(N, heads * D, dtype, s, DEV), shift) for s in (1, 2))
        out = agb.ag_rotary(Q, K, torch.as_tensor(pos).to(DEV), freq.to(DEV), heads, interleaved=interleaved,
                            factor=factor, inverse=inverse)
        alone, none = agb.ag_rotary(Q, None, torch.as_tensor(pos).to(DEV), freq.to(DEV), heads, interleaved=interleaved,
                                    factor=factor, inverse=inverse)
        torch.cuda.synchronize()
        assert none is None and torch.equal(bits(alone), bits(out[0]))
        turns = np.abs(pos[:, None] * freq.numpy()) * 2.0 ** -50
        err = np.zeros((N, heads, D))
        for X, got in zip((Q, K), out):
            x = host(X).astype(np.float64)
            ref = lo.rotary(x, pos, freq.numpy(), heads, interleaved, factor, inverse)
            a = np.abs(x).reshape(N, heads, D)
            i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
            err[...] = 0.0
            err[..., i0] = err[..., i1] = factor * (a[..., i0] + a[..., i1]) * (16 * U + turns[:, None])
            assert_within(got, ref, err.reshape(N, -1) + half_step(dtype) * np.abs(ref), 1.0, f"shift {shift} inv {inverse}")
            rest = host(X).reshape(N, heads, D)[..., rot:]
            assert np.array_equal(host(got).reshape(N, heads, D)[..., rot:], rest)   # copied


def test_rotary_in_place_lengths_and_inverse(agb):
    freq = agb.ag_rotary_freqs(8)[0].to(DEV)
    for N in (0, 1, 2, 147, 149, 5000):
        X = workloads.features(max(N, 1), 32, torch.float32, 3, DEV)[:N].contiguous()
        pos = torch.arange(N, device=DEV) * 1001
        Y, _ = agb.ag_rotary(X, None, pos, freq, 2)
        Z = X.clone()
        W = X.clone()
        agb.ag_rotary(Z, W, pos, freq, 2, Qo=Z, Ko=W)
        assert torch.equal(Z, Y) and torch.equal(W, Y)
        back, _ = agb.ag_rotary(Y, None, pos, freq, 2, inverse=True)
        assert N == 0 or (back - X).abs().max() <= 2 * 16 * U * 2 * X.abs().max()   # two rotations' bounds


def test_rotary_scores_depend_on_differences_alone(agb):
    # <rot(q, a), rot(k, b)> for equal a - b, from far positions: 2 rotations, 16 U each of |q| |k|, and the dot's own sums
    q, k = (workloads.features(1, 64, torch.float32, s, DEV) for s in (1, 2))
    freq = agb.ag_rotary_freqs(64)[0].to(DEV)
    vals = []
    for base in (0, 1000, 1 << 20, 1 << 30):
        pos = torch.tensor([base + 17, base], device=DEV)
        out, _ = agb.ag_rotary(torch.cat([q, k]), None, pos, freq, 1)
        vals.append(float((out[0].double() * out[1].double()).sum()))
    # (angles at 2^30 are off by 2^30 2^-50 turns, far below)
    bound = 4 * 32 * U * float(q.norm() * k.norm()) * 2
    assert max(vals) - min(vals) <= bound


# ------------------------------------------------------------------- norm, gate and residual

def _resnorm_case(N, H, dtype, seed, shift=0):
    names = ("R", "B", "G", "X", "dX", "dZ")
    m = {k: _shifted(workloads.features(N, H, dtype, seed * 100 + i, DEV), shift) for i, k in enumerate(names)}
    gen = torch.Generator().manual_seed(seed)
    v = {k: (lo_ + (hi - lo_) * torch.rand(H, generator=gen)).to(DEV)
         for k, (lo_, hi) in dict(gamma1=(0.5, 1.5), beta1=(-0.5, 0.5), scale=(0.1, 1.0), gamma2=(0.5, 1.5), beta2=(-0.5, 0.5)).items()}
    return m, v


def _abs_norm(x, layer, eps):
    """(normalised size before cancellation, reciprocal deviation) per element, fp64."""
    c = x - x.mean(1, keepdim=True) if layer else x
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    return r * (x.abs() + x.abs().mean(1, keepdim=True)), r


def _check_resnorm(agb, N, H, dtype, norm, act, p, use=("R", "G", "Z"), vectors=True, seed=5, shift=0, dX=True, dZ=True,
                   B=True):
    m, v = _resnorm_case(N, H, dtype, seed, shift)
    if not vectors:
        v = {k: None for k in v}
    if not B:
        v.update(gamma1=None, beta1=None, scale=None)
    layer, silu, eps = norm == "layer", act == "silu", 1e-5
    R = m["R"] if "R" in use else None
    G = m["G"] if "G" in use else None
    Bt = m["B"] if B else None
    kw = dict(eps=eps, norm=norm, act=act, p=p, seed=seed, offset=7, **v)
    X, Z = agb.ag_resnorm_fwd(R, Bt, G, next_norm="Z" in use, **kw)
    d = lambda t: None if t is None else t.double().cpu()
    eps64 = float(np.float32(eps))
    u = torch.as_tensor(lo.drop_factors(N * H, p, seed, 7)).view(N, H) if p else None
    v64 = {k: d(t) for k, t in v.items()}
    rX, rZ = lo.resnorm(d(R), d(Bt), d(G), v64, eps64, layer, silu, u)
    one = lambda k: 1.0 if v64[k] is None else v64[k].abs()
    nil = lambda k: 0.0 if v64[k] is None else v64[k].abs()
    half = half_step(dtype)
    aX = torch.zeros(N, H, dtype=torch.float64) if R is None else d(R).abs()
    if B:
        n1, r1 = _abs_norm(d(Bt), layer, eps64)
        g = d(G)
        sig = None if G is None else torch.sigmoid(g)
        act_a = 1.0 if G is None else (g.abs() * sig if silu else sig)
        slope_a = None if G is None else (sig + g.abs() if silu else sig)
        uu = 1.0 if u is None else u
        u1 = n1 * one("gamma1") + nil("beta1")
        aX = aX + one("scale") * uu * act_a * u1
        assert_within(X, rX.numpy(), (128 * U * aX + half * rX.abs()).numpy(), 1.0, "X")
    else:
        assert X is R
    if "Z" in use:
        n2, r2 = _abs_norm(rX, layer, eps64)
        through = r2 * (aX + aX.mean(1, keepdim=True) + n2 * (n2 * aX).mean(1, keepdim=True)) * one("gamma2")
        assert_within(Z, rZ.numpy(), (128 * U * (n2 * one("gamma2") + nil("beta2") + through) + half * rZ.abs()).numpy(), 1.0, "Z")
    else:
        assert Z is None
    # gradients, from the stored sum m["X"]
    gX, gZ = (m["dX"] if dX else None), (m["dZ"] if dZ else None)
    if not dZ:
        v.update(gamma2=None, beta2=None)
        kw.update(gamma2=None, beta2=None)
    got = agb.ag_resnorm_backward(m["X"], Bt, G, gX, gZ, **kw)
    torch.cuda.synchronize()
    v64 = {k: d(t) for k, t in v.items()}
    ref = lo.resnorm(None, d(Bt), d(G), v64, eps64, layer, silu, u, d(gX), d(gZ), d(m["X"]))
    assert set(got) == set(ref)
    aR = torch.zeros(N, H, dtype=torch.float64) if gX is None else d(gX).abs()
    cols = {}
    mean = lambda t: t.mean(1, keepdim=True)
    if dZ:
        n2, r2 = _abs_norm(d(m["X"]), layer, eps64)
        y = d(gZ).abs() * one("gamma2")
        aR = aR + r2 * (y + n2 * mean(y * n2) + mean(y))
        cols["gamma2"], cols["beta2"] = d(gZ).abs() * n2, d(gZ).abs()
    bound = {"R": aR}
    if B:
        dd = aR * uu
        if G is not None:
            bound["G"] = dd * one("scale") * u1 * slope_a
        du = dd * one("scale") * act_a
        yb = du * one("gamma1")
        bound["B"] = r1 * (yb + n1 * mean(yb * n1) + mean(yb))
        cols.update(gamma1=du * n1, beta1=du, scale=dd * act_a * u1)
    for k in ref:
        if k in bound:
            assert_within(got[k], ref[k].numpy(), (128 * U * bound[k] + half * ref[k].abs()).numpy(), 1.0, f"d{k}")
        else:
            assert_within(got[k], ref[k].numpy(), ((528 * U) * cols[k].sum(0) + U * ref[k].abs()).numpy(), 1.0, f"d{k}")
    again = agb.ag_resnorm_backward(m["X"], Bt, G, gX, gZ, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(again[k]), bits(got[k])) for k in got)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("H", [1, 2, 3, 4, 8, 16, 33, 40, 64, 100, 128, 200, 256, 257, 500, 512, 1000, 1024, 1025, 2048, 4096,
                               4100, 8191, 8192])
def test_resnorm_widths(agb, H, dtype):
    # (a mean over one or two columns leaves nothing or a sign of LAYER's deviations: RMS there)
    norm = "layer" if H % 3 != 1 and H > 4 else "rms"
    _check_resnorm(agb, 37 if H > 1000 else 333, H, dtype, norm, "silu" if H % 2 else "sigmoid", 0.1 if H % 4 else 0.0)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 255, 4999])
def test_resnorm_lengths(agb, N):
    _check_resnorm(agb, N, 64, torch.float32, "layer", "silu", 0.2)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_resnorm_forms(agb, norm, act, p):
    _check_resnorm(agb, 100, 48, torch.float32, norm, act, p)
    _check_resnorm(agb, 100, 48, torch.bfloat16, norm, act, p, vectors=False)


@pytest.mark.parametrize("use,kw", [(("R", "Z"), {}), (("G", "Z"), {}), (("Z",), {}), (("R", "G"), dict(dZ=False)),
                                    (("R", "Z"), dict(B=False)), (("R", "Z"), dict(B=False, dX=False)),
                                    (("G",), dict(dZ=False)), (("R", "G", "Z"), dict(dX=False))])
def test_resnorm_parts_left_out(agb, use, kw):
    _check_resnorm(agb, 130, 40, torch.float32, "layer", "sigmoid", 0.1 if kw.get("B", True) else 0.0, use=use, **kw)


@pytest.mark.parametrize("dtype,H,shift", [(torch.float32, 64, 1), (torch.bfloat16, 64, 1), (torch.bfloat16, 64, 4),
                                           (torch.bfloat16, 2048, 3)])
def test_resnorm_addresses_without_a_wide_vector(agb, dtype, H, shift):
    _check_resnorm(agb, 50, H, dtype, "rms", "silu", 0.3, shift=shift)


def test_resnorm_is_the_norm_of_every_head(agb):
    # [N, H] as [N * heads, D]: the per-head norm behind the attention, against each head by itself
    X = workloads.features(50, 96, torch.float32, 4, DEV)
    g = torch.rand(32, device=DEV) + 0.5
    _, Z = agb.ag_resnorm_fwd(X.view(150, 32), None, gamma2=g)
    for h in range(3):
        _, one = agb.ag_resnorm_fwd(X[:, 32 * h:32 * h + 32].contiguous(), None, gamma2=g)
        assert torch.equal(Z.view(50, 96)[:, 32 * h:32 * h + 32], one)


def test_resnorm_offset_rows_constant_rows_and_no_rows(agb):
    # rows far from zero (the mean cancels), constant rows (deviation 0: eps alone), no rows at all
    X = workloads.features(60, 64, torch.float32, 9, DEV) + 100.0
    X[3] = 5.0
    _, Z = agb.ag_resnorm_fwd(X, None, norm="layer", eps=1e-5)
    x = X.double().cpu()
    c = x - x.mean(1, keepdim=True)
    r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + float(np.float32(1e-5)))
    # the mean of values near 100 is off by 20 U * 100, which moves the deviation too
    err = r * (22 * U * x.abs().max()) * (1 + (c * r).abs()) + 32 * U * (c * r).abs()
    assert_within(Z, (c * r).numpy(), err.numpy(), 1.0, "offset rows")
    E = X[:0].contiguous()
    g = torch.ones(64, device=DEV)
    assert agb.ag_resnorm_fwd(E, E, gamma1=g)[1].shape == (0, 64)
    d = agb.ag_resnorm_backward(E, E, None, E, E, gamma1=g, gamma2=g)
    torch.cuda.synchronize()
    assert not d["gamma1"].any() and not d["gamma2"].any()


def test_resnorm_eps_zero_and_rows_behind_the_last(agb):
    # 7 rows fill no block: what stands in for further rows must not reach the column sums
    N, H = 7, 32
    m, v = _resnorm_case(N, H, torch.float32, 12)
    d = agb.ag_resnorm_backward(m["X"], m["B"], m["G"], m["dX"], m["dZ"], eps=0.0, **v)
    e = agb.ag_resnorm_backward(m["X"], m["B"], m["G"], m["dX"], m["dZ"], eps=1e-12, **v)
    torch.cuda.synchronize()
    for k in d:   # variances near 1: 1e-12 more changes a deviation by 5e-13, below a rounding
        assert torch.isfinite(d[k]).all() and (d[k] - e[k]).abs().max() <= 64 * U * e[k].abs().max(), k


def test_rowwise_streams_and_capture(agb):
    N, H = 700, 96
    m, v = _resnorm_case(N, H, torch.bfloat16, 3)
    pos, freq = torch.arange(N, device=DEV), agb.ag_rotary_freqs(8)[0].to(DEV)

    def step(stream=None):
        X, Z = agb.ag_resnorm_fwd(m["R"], m["B"], m["G"], p=0.1, seed=4, stream=stream, **v)
        q, k = agb.ag_rotary(Z, X, pos, freq, 6, stream=stream)
        y = agb.ag_dropout(q, 0.2, 9, stream=stream)
        d = agb.ag_resnorm_backward(X, m["B"], m["G"], k, y, p=0.1, seed=4, stream=stream, **v)
        return [X, Z, q, k, y] + [d[n] for n in sorted(d)]
    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [step(s) for _ in range(4)]
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        out = step()
    for t in out:
        t.zero_()
    cg.replay()
    torch.cuda.synchronize()
    for o in got + [out]:
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(o, want))


def test_rowwise_beyond_32_bit_offsets(agb):
    # 2^31 + 24 elements of bf16: the last block's counters pass 2^29, offsets 2^32 bytes
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    n = (1 << 31) + 24
    X = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    Y = agb.ag_dropout(X, 0.5, 5, 6)
    for first in (0, (1 << 31) - 512, n - 1000):
        some = host(Y[first:first + 1000])      # (fewer at the end)
        assert np.array_equal(some != 0, lo.keep_mask(len(some), 0.5, 5, 6, first=first)), first
    # the same rows at the end of a matrix and by themselves (the mask goes by the index: without dropout)
    N, H = n // 8, 8
    tail = workloads.features(64, H, torch.bfloat16, 3, DEV)
    M = X.view(N, H)
    M[-64:] = tail
    _, Z = agb.ag_resnorm_fwd(M, None, norm="layer", Z=Y.view(N, H))
    assert torch.equal(Z[-64:], agb.ag_resnorm_fwd(tail, None, norm="layer")[1])
    freq = agb.ag_rotary_freqs(4)[0].to(DEV)
    pos = torch.arange(N, device=DEV)
    agb.ag_rotary(M, None, pos, freq, 2, Qo=M)
    assert torch.equal(M[-64:], agb.ag_rotary(tail, None, pos[-64:].contiguous(), freq, 2)[0])


def test_outputs_in_place_and_overlaps(agb):
    N, H = 60, 32
    m, v = _resnorm_case(N, H, torch.float32, 21)
    want = agb.ag_resnorm_fwd(m["R"], m["B"], m["G"], p=0.1, **v)
    R, B = m["R"].clone(), m["B"].clone()
    got = agb.ag_resnorm_fwd(R, B, m["G"], p=0.1, X=R, Z=B, **v)
    assert got[0] is R and got[1] is B and all(torch.equal(a, b) for a, b in zip(got, want))
    big = torch.zeros(3 * N * H, device=DEV)
    A, part = big[:N * H].view(N, H), big[H:H + N * H].view(N, H)
    f, pos = torch.ones(4, dtype=torch.float64, device=DEV), torch.arange(N, device=DEV)
    for call in (lambda: agb.ag_dropout(A, 0.1, 1, out=part), lambda: agb.ag_rotary(A, None, pos, f, 2, Qo=part),
                 lambda: agb.ag_rotary(A, m["R"], pos, f, 2, Qo=m["B"], Ko=m["B"]),
                 lambda: agb.ag_resnorm_fwd(A, m["B"], X=part), lambda: agb.ag_resnorm_fwd(A, m["B"], X=m["R"], Z=m["R"])):
        with pytest.raises(agb.AggraphError, match="overlaps"):
            call()


def test_rowwise_refusals(agb):
    X = torch.randn(8, 16, device=DEV)
    f = torch.ones(4, dtype=torch.float64, device=DEV)
    pos = torch.arange(8, device=DEV)
    g = torch.ones(16, device=DEV)
    bad = [lambda: agb.ag_dropout(X.double(), 0.1, 1), lambda: agb.ag_dropout(X.t(), 0.1, 1),
           lambda: agb.ag_dropout(X, 0.1, 1, out=X.bfloat16()), lambda: agb.ag_dropout(X, 0.1, 1 << 64),
           lambda: agb.ag_rotary(X, None, pos.int(), f, 2), lambda: agb.ag_rotary(X, None, pos, f.float(), 2),
           lambda: agb.ag_rotary(X, None, pos[:-1], f, 2), lambda: agb.ag_rotary(X, X[:4], pos, f, 2),
           lambda: agb.ag_rotary(X, None, pos, f, 3), lambda: agb.ag_rotary(X, None, pos, f, 4),
           lambda: agb.ag_rotary(X, None, pos, f[:0], 2), lambda: agb.ag_rotary(X, None, pos, f, 2, Ko=X),
           lambda: agb.ag_rotary(X[0], None, pos, f, 2), lambda: agb.ag_rotary(X, None, pos.cpu(), f, 2),
           lambda: agb.ag_resnorm_fwd(X, X, X.bfloat16()), lambda: agb.ag_resnorm_fwd(X, X[:4]),
           lambda: agb.ag_resnorm_fwd(X, X, gamma1=g[:8]), lambda: agb.ag_resnorm_fwd(X, X, gamma1=g.double()),
           lambda: agb.ag_resnorm_fwd(X, X, norm="batch"), lambda: agb.ag_resnorm_fwd(X, X, act="relu"),
           lambda: agb.ag_resnorm_fwd(X, X, eps=-1.0), lambda: agb.ag_resnorm_fwd(X, None, G=X),
           lambda: agb.ag_resnorm_fwd(X, None, X=X), lambda: agb.ag_resnorm_fwd(X, X, next_norm=False, Z=X),
           lambda: agb.ag_resnorm_fwd(X, None, next_norm=False), lambda: agb.ag_resnorm_fwd(X, X, p=1.5),
           lambda: agb.ag_resnorm_backward(X, None, None, X, X, gamma1=g),
           lambda: agb.ag_resnorm_backward(X, X, None, X, None, gamma2=g),
           lambda: agb.ag_resnorm_backward(X, X, None, None, None), lambda: agb.ag_resnorm_backward(None, X, None, X, X)]
    for i, call in enumerate(bad):
        with pytest.raises(agb.AggraphError):
            call()
            pytest.fail(f"refusal {i} did not come")
    host_x = torch.zeros(16)
    import ctypes
    P = lambda t: ctypes.c_void_p(t.data_ptr())
    assert agb.lib.ag_dropout(P(host_x), P(X), 16, 0.1, 0, 0, 0, None) == 4      # host memory
