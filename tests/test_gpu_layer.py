"""A whole differential attention layer, forward and backward, through the
library's calls in the order a training program makes them: norm, projections,
rotary positions, attention with dropout, the norm of every head, output
projection, gated residual with the next norm; against autograd in 64 bits.

Tolerance: every call's results are within 128 U (U = 2^-24) of its terms (the
bound of the row-wise tests, above the attention's at these sizes).  The 64-bit
layer is run with each intermediate changed by that much, relative, with
random signs; the largest change over four draws, times 8 (for the changes of
a worst case against a random one), bounds the error of each output.
"""
import numpy as np
import pytest
import torch

import workloads
from tests import layer_oracle as lo
from tests.gpu_helpers import host, lib
from tests.layer_oracle import U

pytestmark = pytest.mark.gpu
DEV = "cuda"
HEADS, D = 4, 8
H = 2 * HEADS * D
EPS = 1e-5
PA, PR, SEED = 0.1, 0.2, 77


def _inputs(N, seed):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen)
    t = dict(X0=rnd(N, H), G1=rnd(N, H), G2=rnd(N, H))
    t.update({k: rnd(H, H) / H ** 0.5 for k in ("Wq", "Wk", "Wv", "Wo", "Wg")})
    t.update({k: 0.5 + torch.rand(H, generator=gen) for k in ("g0", "g1", "g2", "sc")}, gh=0.5 + torch.rand(2 * D, generator=gen),
             lam=0.2 + 0.6 * torch.rand(HEADS, generator=gen))
    return t


GRADS = ("X0", "Wq", "Wk", "Wv", "Wo", "Wg", "g0", "g1", "g2", "sc", "gh", "lam")


def _oracle(t, src, dst, pos, freq, factor, noise=0.0, seed=0):
    """fp64 autograd; every intermediate is changed by `noise`, relative."""
    gen = torch.Generator().manual_seed(seed)
    v = {k: x.double().requires_grad_(k in GRADS) for k, x in t.items()}

    def near(x):
        return x if not noise else x * (1 + noise * (torch.randint(0, 2, x.shape, generator=gen) * 2 - 1))

    rms = lambda x, g: near(x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * g)
    N, E = v["X0"].shape[0], len(src)
    z0 = rms(v["X0"], v["g0"])
    q, k, w = (near(z0 @ v[n]) for n in ("Wq", "Wk", "Wv"))
    a = torch.outer(pos.double(), freq)
    c, s = (factor * torch.cos(a))[:, None], (factor * torch.sin(a))[:, None]

    def turn(x):
        x = x.view(N, 2 * HEADS, D)
        r = freq.numel()
        x0, x1, rest = x[..., :r], x[..., r:2 * r], x[..., 2 * r:]
        return near(torch.cat([x0 * c - x1 * s, x1 * c + x0 * s, rest], -1)).view(N, HEADS, 2, D)
    q, k = turn(q), turn(k)
    e = torch.exp((q[dst] * k[src]).sum(-1) * D ** -0.5)
    p = near(e / torch.zeros(N, HEADS, 2, dtype=torch.float64).index_add(0, dst, e)[dst])
    m = torch.as_tensor(lo.drop_factors(E * HEADS, PA, SEED, 1)).view(E, HEADS)
    y = torch.zeros(N, HEADS, 2 * D, dtype=torch.float64).index_add(
        0, dst, (m * (p[..., 0] - v["lam"] * p[..., 1]))[..., None] * w.view(N, HEADS, 2 * D)[src])
    y = rms(near(y), v["gh"]).reshape(N, H)
    o = near(y @ v["Wo"])
    gate = near(torch.sigmoid(near(z0 @ v["Wg"])))
    mr = torch.as_tensor(lo.drop_factors(N * H, PR, SEED, 2)).view(N, H)
    x1 = near(v["X0"] + v["sc"] * mr * gate * rms(o, v["g1"]))
    z1 = rms(x1, v["g2"])
    loss = (x1 * v["G1"]).sum() + (z1 * v["G2"]).sum()
    grads = torch.autograd.grad(loss, [v[k] for k in GRADS])
    return [x1.detach(), z1.detach()] + [near(x) for x in grads]


def _layer(agb, g, t, pos, freq, factor):
    N = t["X0"].shape[0]
    _, z0 = agb.ag_resnorm_fwd(t["X0"], None, gamma2=t["g0"], eps=EPS)
    q, k, w, gate = (z0 @ t[n] for n in ("Wq", "Wk", "Wv", "Wg"))
    q, k = agb.ag_rotary(q, k, pos, freq, 2 * HEADS, factor=factor)
    att = dict(p=PA, seed=SEED, offset=1)
    y, lse = agb.ag_diff_attn_fwd(g, q, k, w, t["lam"], D ** -0.5, **att)
    _, yh = agb.ag_resnorm_fwd(y.view(N * HEADS, 2 * D), None, gamma2=t["gh"], eps=EPS)
    yh = yh.view(N, H)
    o = yh @ t["Wo"]
    res = dict(gamma1=t["g1"], scale=t["sc"], gamma2=t["g2"], eps=EPS, p=PR, seed=SEED, offset=2)
    x1, z1 = agb.ag_resnorm_fwd(t["X0"], o, gate, **res)
    # backward
    d = agb.ag_resnorm_backward(x1, o, gate, t["G1"], t["G2"], **res)
    out = dict(g1=d["gamma1"], sc=d["scale"], g2=d["gamma2"], Wo=yh.t() @ d["B"], Wg=z0.t() @ d["G"])
    dyh = (d["B"] @ t["Wo"].t()).view(N * HEADS, 2 * D)
    dh = agb.ag_resnorm_backward(y.view(N * HEADS, 2 * D), None, None, None, dyh, gamma2=t["gh"], eps=EPS)
    out["gh"] = dh["gamma2"]
    dq, dk, dw, out["lam"] = agb.ag_diff_attn_backward(g, q, k, w, t["lam"], D ** -0.5, lse, dh["R"].view(N, H), **att)
    dq, dk = agb.ag_rotary(dq, dk, pos, freq, 2 * HEADS, factor=factor, inverse=True, Qo=dq, Ko=dk)
    dz0 = dq @ t["Wq"].t() + dk @ t["Wk"].t() + dw @ t["Wv"].t() + d["G"] @ t["Wg"].t()
    out.update(Wq=z0.t() @ dq, Wk=z0.t() @ dk, Wv=z0.t() @ dw)
    d0 = agb.ag_resnorm_backward(t["X0"], None, None, d["R"], dz0, gamma2=t["g0"], eps=EPS)
    out.update(X0=d0["R"], g0=d0["gamma2"])
    return [x1, z1] + [out[k] for k in GRADS]


def _graph(agb, N=150, E=1200):
    rng = np.random.default_rng(3)
    # every row has at least two edges: the head norm of an empty row's zeros has a gradient of order 1 / sqrt(eps)
    src = np.concatenate([np.arange(N), rng.integers(0, N, E)])
    dst = np.concatenate([np.arange(N), rng.permutation(np.arange(E) % N)])
    g = agb.ag_graph_lower(*(torch.as_tensor(x.astype(np.int32)).to(DEV) for x in (src, dst)), N)
    return g, torch.as_tensor(src), torch.as_tensor(dst), N


def test_layer_matches_autograd_and_its_captured_form():
    agb = lib()
    assert not torch.backends.cuda.matmul.allow_tf32
    g, src, dst, N = _graph(agb)
    t = _inputs(N, 5)
    pos = torch.as_tensor(np.random.default_rng(8).integers(0, 1 << 20, N))
    freq, factor = agb.ag_rotary_freqs(4, scaling="yarn", factor=4.0, original=1024.0)
    factor = float(np.float32(factor))
    dev = {k: x.to(DEV) for k, x in t.items()}
    args = (dev, pos.to(DEV), freq.to(DEV), factor)
    got = _layer(agb, g, *args)
    torch.cuda.synchronize()
    ref = _oracle(t, src, dst, pos, freq, factor)
    moved = [_oracle(t, src, dst, pos, freq, factor, 128 * U, s) for s in range(4)]
    for name, a, r, *others in zip(("X1", "Z1") + GRADS, got, ref, *moved):
        limit = 8 * max(float((o - r).abs().max()) for o in others)
        err = float((a.double().cpu() - r).abs().max())
        assert err <= limit, (name, err, limit)
        assert limit <= 0.02 * float(r.abs().max()), name      # the bound says something
    # the same step captured and replayed on new inputs of the same buffers
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(agb, g, *args)
    fresh = _inputs(N, 6)
    for k, x in fresh.items():
        dev[k].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    replayed = [x.clone() for x in out]
    eager = _layer(agb, g, *args)
    torch.cuda.synchronize()
    # (the library calls' bits are fixed; the projections between them may take another cuBLAS kernel under capture)
    for name, a, b in zip(("X1", "Z1") + GRADS, replayed, eager):
        assert float((a - b).abs().max()) <= 1e-3 * float(b.abs().max()), name


def test_calls_in_a_row_share_memory_without_a_wait():
    # outputs and scratch of one call are the next one's memory, each call's
    # launches start as the one before runs out: eager and in one captured graph
    # every call gives what it gives alone
    agb = lib()
    rng = np.random.default_rng(4)
    N = 2000
    src, dst = rng.integers(0, N, 30000), rng.integers(0, N, 30000)
    dst[:5000], src[-4000:] = 17, 3       # rows of many tiles on both sides
    g = agb.ag_graph_lower(*(torch.as_tensor(x.astype(np.int32)).to(DEV) for x in (src, dst)), N)
    gen = torch.Generator().manual_seed(9)
    sets = [[torch.randn(N, H, generator=gen).to(DEV) for _ in range(4)] for _ in range(2)]
    lam = torch.full((HEADS,), 0.4, device=DEV)
    ones = torch.ones(H, device=DEV)

    def step(q, k, v, dy):
        y, lse = agb.ag_diff_attn_fwd(g, q, k, v, lam, 0.3, p=PA, seed=SEED)
        dq, dk, dv, dlam = agb.ag_diff_attn_backward(g, q, k, v, lam, 0.3, lse, dy, p=PA, seed=SEED)
        back = agb.ag_resnorm_backward(v, y, k, dy, dq, gamma1=ones, scale=ones, gamma2=ones)
        return [y, dq, dk, dv, dlam, *back.values()]

    want = []
    for s in sets:
        want.append([x.clone() for x in step(*s)])
        torch.cuda.synchronize()
    got = [[x.clone() for x in step(*sets[i % 2])] for i in range(20)]
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2], strict=True)), i
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        kept = [[x.clone() for x in step(*sets[i % 2])] for i in range(6)]
    for _ in range(5):
        cg.replay()
    torch.cuda.synchronize()
    for i, r in enumerate(kept):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2], strict=True)), i
