"""The operators of a differential graph-attention layer, as they are measured.

Four operators that a layer of this kind chains, on the [N, H] feature matrices
of a graph with E edges:

  rotary   rotary positions on queries and keys (half and interleaved layouts,
           part of a head, frequencies scaled for long ranges), and the inverse
           rotation that its gradient is
  diff     differential edge-softmax attention, with dropout of the maps:
           Y = sum over edges of (alpha1 - lambda alpha2) V, and its gradients
  resnorm  a norm after a block, its gate, dropout and residual scale, the
           residual sum, and the norm before the next block, with gradients
  dropout  dropout from a counter-based generator on features or edge weights

`run` computes an operator in its plain form (elementary torch operations), or
calls the library's entry points where `own` is true.  `exact` computes the
same from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
U32 = 0xFFFFFFFF


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one small sampled subgraph, scored as it arrives: latency counts
        dict(name="diff fwd uniform fp32", op="diff", graph="uniform", N=1024, E=8192, H=16, heads=1, dtype="fp32",
             p=0.0, train=False),
        # a training step's attention on a community graph
        dict(name="diff train blocks fp32", op="diff", graph="blocks", N=20000, E=564011, H=64, heads=2,
             dtype="fp32", p=0.0, train=True),
        # wide rows of a two-hop minibatch (15, then 10 neighbours), trained with dropout
        dict(name="diff train twohop fp32", op="diff", graph="twohop", N=169984, E=168960, H=256, heads=4,
             dtype="fp32", p=0.1, train=True),
        # a ragged head size on a small skewed graph
        dict(name="diff train ragged bf16", op="diff", graph="skewed", N=5003, E=70001, H=72, heads=3, dtype="bf16",
             p=0.2, train=True),
        # the largest: a skewed graph of 4.2 million edges
        dict(name="diff train rmat18 bf16", op="diff", graph="rmat", N=1 << 18, E=16 << 18, H=128, heads=4,
             dtype="bf16", p=0.1, train=True),
        # positions of the nodes of one small subgraph
        dict(name="rotary uniform fp32", op="rotary", N=1024, H=16, heads=2, rot=8, layout="half", scaling="none",
             inverse=False, dtype="fp32"),
        # far positions, part of each head, frequencies scaled
        dict(name="rotary rmat20 bf16", op="rotary", N=1 << 20, H=128, heads=8, rot=8, layout="interleaved",
             scaling="yarn", inverse=False, dtype="bf16"),
        # one small subgraph through the norms, forward only
        dict(name="resnorm fwd uniform fp32", op="resnorm", N=1024, H=16, norm="rms", act="sigmoid", p=0.0,
             dtype="fp32", back=False),
        # norms, gate, dropout and residual over a large graph's nodes
        dict(name="resnorm fwd rmat20 bf16", op="resnorm", N=1 << 20, H=128, norm="layer", act="silu", p=0.1,
             dtype="bf16", back=False),
        # their gradients on a two-hop minibatch's wide rows, from the stored sum
        dict(name="resnorm bwd twohop fp32", op="resnorm", N=156323, H=256, norm="layer", act="sigmoid", p=0.1,
             dtype="fp32", back=True),
        # dropped edges: weights of a skewed graph's million edges
        dict(name="dropout edges fp32", op="dropout", rows=1 << 20, H=1, p=0.3, dtype="fp32"),
        # dropped features of a large graph's nodes
        dict(name="dropout rmat20 bf16", op="dropout", rows=1 << 20, H=128, p=0.1, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["diff", "diff", "diff", "rotary", "resnorm", "resnorm", "dropout"])
    dtype = rng.choice(["fp32", "bf16"])
    if op == "diff":
        heads = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([3, 4, 8, 12, 16, 20, 32, 64])
        H = 2 * heads * d
        E = _log_int(rng, 2000, min(16 << 18, (16 << 18) * 128 // H))
        N = max(2, int(E / math.exp(rng.uniform(math.log(1.5), math.log(40)))))
        graph = rng.choice(["uniform", "blocks", "skewed"])
        if graph == "blocks":
            N = max(20, N // 20 * 20)
        return dict(op=op, graph=graph, N=N, E=E, H=H, heads=heads, dtype=dtype, p=rng.choice([0.0, 0.1, 0.5]),
                    train=rng.random() < 0.7)
    if op == "rotary":
        heads = rng.choice([2, 4, 8, 16])
        D = rng.choice([6, 8, 16, 20, 32, 64, 128])
        H = heads * D
        rot = rng.choice([D, 2 * max(1, D // 4)])
        N = _log_int(rng, 500, min(1 << 20, (1 << 27) // H))
        return dict(op=op, N=N, H=H, heads=heads, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), inverse=rng.random() < 0.5, dtype=dtype)
    if op == "resnorm":
        H = rng.choice([16, 33, 64, 100, 128, 200, 256, 512, 1000, 2048, 4096])
        N = _log_int(rng, 300, min(1 << 20, (1 << 27) // H))
        return dict(op=op, N=N, H=H, norm=rng.choice(["rms", "layer"]), act=rng.choice(["sigmoid", "silu"]),
                    p=rng.choice([0.0, 0.1]), dtype=dtype, back=rng.random() < 0.6)
    H = rng.choice([1, 1, 16, 33, 64, 100, 128, 256])
    rows = _log_int(rng, 2000, min(1 << 22, (1 << 27) // H))
    return dict(op=op, rows=rows, H=H, p=rng.choice([0.05, 0.1, 0.3, 0.5]), dtype=dtype)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _edges(kind, N, E, g):
    """COO endpoints (int32): uniform, 88 % inside one of 20 blocks, skewed
    towards low ids, R-MAT (.57, .19, .19, .05), or a two-hop sample."""
    if kind == "uniform":
        src = torch.randint(0, N, (E,), generator=g, device=DEV)
        dst = torch.randint(0, N, (E,), generator=g, device=DEV)
    elif kind == "blocks":
        size = N // 20
        dst = torch.randint(0, N, (E,), generator=g, device=DEV)
        inside = torch.rand(E, generator=g, device=DEV) < 0.88
        near = dst // size * size + torch.randint(0, size, (E,), generator=g, device=DEV)
        far = torch.randint(0, N, (E,), generator=g, device=DEV)
        src = torch.where(inside & (near < N), near, far)
    elif kind == "skewed":
        src = (N * torch.rand(E, generator=g, device=DEV).pow(3)).long().clamp_(max=N - 1)
        dst = (N * torch.rand(E, generator=g, device=DEV).pow(3)).long().clamp_(max=N - 1)
    elif kind == "rmat":
        src = torch.zeros(E, dtype=torch.int64, device=DEV)
        dst = torch.zeros(E, dtype=torch.int64, device=DEV)
        for level in range(N.bit_length() - 1):
            u = torch.rand(E, generator=g, device=DEV)
            src += (u >= 0.76).long() << level
            dst += (((u >= 0.57) & (u < 0.76)) | (u >= 0.95)).long() << level
    elif kind == "twohop":
        first = torch.arange(1024, device=DEV).repeat_interleave(15)
        second = 1024 + torch.arange(15 * 1024, device=DEV).repeat_interleave(10)
        dst = torch.cat([first, second])
        src = 1024 + torch.arange(dst.numel(), device=DEV)
        order = torch.randperm(dst.numel(), generator=g, device=DEV)
        src, dst = src[order], dst[order]
    else:
        raise ValueError(kind)
    return src.int(), dst.int()


def _inv_freq(rot, scaling):
    """Frequencies of the rot / 2 pairs: base 10000, and the ways to stretch
    them by 8 beyond 4096 positions (linear; a larger base; a ramp between the
    two by the number of turns, with the factor 0.1 ln 8 + 1 on the outputs)."""
    base, s, orig = 10000.0, 8.0, 4096.0
    if scaling == "ntk" and rot > 2:
        base *= s ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / s for x in f]
    if scaling == "yarn":
        at = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(at(32.0))), min(rot - 1, math.ceil(at(1.0)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        f = [x / s * r + x * (1 - r) for x, r in zip(f, ramp)]
    return f, (0.1 * math.log(s) + 1.0 if scaling == "yarn" else 1.0)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    st = dict(case)
    rnd = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(dt)
    uni = lambda lo, hi, *shape: lo + (hi - lo) * torch.rand(shape, generator=g, device=DEV)
    st["seed"], st["offset"] = int(seed) * 2654435761 % (1 << 62) + 1, int(seed) % 1000
    if case["op"] == "diff":
        N, H = case["N"], case["H"]
        st["src"], st["dst"] = _edges(case["graph"], N, case["E"], g)
        st["Q"], st["K"], st["V"] = rnd(N, H), rnd(N, H), rnd(N, H)
        st["lam"] = uni(0.2, 0.8, case["heads"])
        st["scale"] = (H // (2 * case["heads"])) ** -0.5
        if case["train"]:
            st["dY"] = rnd(N, H)
        if own:  # the lowered topology, which a user keeps for every call on the graph
            import gnn_sparse_aggregation_b200 as ag
            st["g"] = ag.ag_graph_lower(st["src"], st["dst"], N)
    elif case["op"] == "rotary":
        N, H = case["N"], case["H"]
        st["Q"], st["K"] = rnd(N, H), rnd(N, H)
        st["pos"] = torch.randint(0, 1 << 20, (N,), generator=g, device=DEV)
        f, st["factor"] = _inv_freq(case["rot"], case["scaling"])
        st["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    elif case["op"] == "resnorm":
        N, H = case["N"], case["H"]
        st["B"], st["G"] = rnd(N, H), rnd(N, H)
        st["gamma1"], st["gamma2"] = uni(0.5, 1.5, H), uni(0.5, 1.5, H)
        st["beta1"] = uni(-0.5, 0.5, H) if case["norm"] == "layer" else None
        st["beta2"] = uni(-0.5, 0.5, H) if case["norm"] == "layer" else None
        st["rscale"] = uni(0.1, 1.0, H)
        st["eps"] = 1e-5
        if case["back"]:  # the sum that the forward pass stored, and the gradients of both outputs
            st["X"], st["dX"], st["dZ"] = rnd(N, H), rnd(N, H), rnd(N, H)
        else:
            st["R"] = rnd(N, H)
    else:
        st["X"] = rnd(case["rows"], case["H"])
    return st


# ------------------------------------------------------------------- plain forms

def _keep(n, p, seed, offset):
    """Truth values of n elements: element i is kept where word i % 4 of
    Philox4x32-10 (counter (i / 4, offset), key seed) is at least p 2^32."""
    i = torch.arange((n + 3) // 4, dtype=torch.int64, device=DEV)
    c0, c1 = i & U32, i >> 32
    c2, c3 = torch.full_like(i, offset & U32), torch.full_like(i, offset >> 32)
    k0, k1 = seed & U32, (seed >> 32) & U32
    for _ in range(10):
        m0, m1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # products mod 2^64
        c0, c1, c2, c3 = ((m1 >> 32) & U32) ^ c1 ^ k0, m1 & U32, ((m0 >> 32) & U32) ^ c3 ^ k1, m0 & U32
        k0, k1 = (k0 + 0x9E3779B9) & U32, (k1 + 0xBB67AE85) & U32
    word = torch.stack([c0, c1, c2, c3], 1).view(-1)[:n]
    return word >= round(p * 4294967296.0)


def _mask(n, p, seed, offset):
    """1 / (1 - p) where kept, else 0 (None without dropout)."""
    return _keep(n, p, seed, offset).float() * (1.0 / (1.0 - p)) if p > 0 else None


def _rows(index, value, N):
    """Sums of the edges' values by row."""
    return torch.zeros((N,) + value.shape[1:], device=DEV).index_add_(0, index, value)


def _diff_plain(s):
    N, E, h = s["N"], s["E"], s["heads"]
    d = s["H"] // (2 * h)
    dt = s["Q"].dtype
    src, dst = s["src"].long(), s["dst"].long()
    Q, K = (s[k].float().view(N, h, 2, d) for k in ("Q", "K"))
    V = s["V"].float().view(N, h, 2 * d)
    lam = s["lam"]
    score = (Q[dst] * K[src]).sum(3) * s["scale"]                                    # [E, h, 2]
    top = torch.full((N, h, 2), -math.inf, device=DEV)
    top = top.scatter_reduce(0, dst.view(E, 1, 1).expand(E, h, 2), score, "amax")
    e = torch.exp(score - top[dst])
    total = _rows(dst, e, N)
    lse = top + torch.log(total)
    alpha = e / total[dst]
    mask = _mask(E * h, s["p"], s["seed"], s["offset"])
    mask = torch.ones(E, h, device=DEV) if mask is None else mask.view(E, h)
    both = mask * (alpha[:, :, 0] - lam * alpha[:, :, 1])
    Y = _rows(dst, both.unsqueeze(2) * V[src], N).view(N, -1).to(dt)
    if not s["train"]:
        return Y, lse
    dY = s["dY"].float().view(N, h, 2 * d)
    dV = _rows(src, both.unsqueeze(2) * dY[dst], N)
    da = mask * (dY[dst] * V[src]).sum(2)                                            # [E, h]
    row = _rows(dst, alpha * da.unsqueeze(2), N)                                     # [N, h, 2]
    dlam = -row[:, :, 1].double().sum(0).float()
    weight = torch.stack([torch.ones_like(lam), -lam], 1) * s["scale"]               # [h, 2]
    ds = (alpha * (da.unsqueeze(2) - row[dst]) * weight).unsqueeze(3)
    dQ, dK = _rows(dst, ds * K[src], N), _rows(src, ds * Q[dst], N)
    return (Y, lse) + tuple(t.reshape(N, -1).to(dt) for t in (dQ, dK, dV)) + (dlam,)


def _rotate_plain(s, X):
    N, h, rot = s["N"], s["heads"], s["rot"]
    x = X.float().view(N, h, -1)
    angle = s["pos"].double().unsqueeze(1) * s["inv_freq"]
    c = (torch.cos(angle) * s["factor"]).float().unsqueeze(1)
    t = (torch.sin(angle) * (-s["factor"] if s["inverse"] else s["factor"])).float().unsqueeze(1)
    y = x.clone()
    if s["layout"] == "half":
        a, b = x[:, :, : rot // 2], x[:, :, rot // 2: rot]
        y[:, :, : rot // 2], y[:, :, rot // 2: rot] = a * c - b * t, b * c + a * t
    else:
        a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
        y[:, :, 0:rot:2], y[:, :, 1:rot:2] = a * c - b * t, b * c + a * t
    return y.view(N, -1).to(X.dtype)


def _norm_plain(x, s):
    """The normalised rows and the reciprocal deviations."""
    if s["norm"] == "layer":
        x = x - x.mean(1, keepdim=True)
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + s["eps"])
    return x * r, r


def _norm_back(n, r, dn, s):
    """The gradient of _norm_plain for the gradient dn of the normalised rows."""
    dx = dn - n * (dn * n).mean(1, keepdim=True)
    if s["norm"] == "layer":
        dx = dx - dn.mean(1, keepdim=True)
    return dx * r


def _resnorm_plain(s):
    dt = s["B"].dtype
    B, G = s["B"].float(), s["G"].float()
    b1 = 0.0 if s["beta1"] is None else s["beta1"]
    b2 = 0.0 if s["beta2"] is None else s["beta2"]
    n1, r1 = _norm_plain(B, s)
    sig = 1.0 / (1.0 + torch.exp(-G))
    act = sig if s["act"] == "sigmoid" else G * sig
    mask = _mask(B.numel(), s["p"], s["seed"], s["offset"])
    mask = 1.0 if mask is None else mask.view_as(B)
    u1 = n1 * s["gamma1"] + b1
    if not s["back"]:
        X = s["R"].float() + s["rscale"] * (mask * (act * u1))
        n2, _ = _norm_plain(X, s)
        return X.to(dt), (n2 * s["gamma2"] + b2).to(dt)
    dZ = s["dZ"].float()
    n2, r2 = _norm_plain(s["X"].float(), s)
    dR = s["dX"].float() + _norm_back(n2, r2, dZ * s["gamma2"], s)
    dbranch = dR * s["rscale"] * mask
    dact, du1 = dbranch * u1, dbranch * act
    dsig = sig * (1.0 - sig)
    dG = dact * (dsig if s["act"] == "sigmoid" else sig + G * dsig)
    dB = _norm_back(n1, r1, du1 * s["gamma1"], s)
    total = lambda v: v.sum(0, dtype=torch.float64).float()
    grads = (total(du1 * n1), total(dR * mask * act * u1), total(dZ * n2))
    if s["norm"] == "layer":
        grads += (total(du1), total(dZ))
    return (dR.to(dt), dB.to(dt), dG.to(dt)) + grads


def _run_plain(s):
    if s["op"] == "diff":
        return _diff_plain(s)
    if s["op"] == "rotary":
        return _rotate_plain(s, s["Q"]), _rotate_plain(s, s["K"])
    if s["op"] == "resnorm":
        return _resnorm_plain(s)
    X = s["X"]
    return (X.float() * _mask(X.numel(), s["p"], s["seed"], s["offset"]).view_as(X)).to(X.dtype)


def _run_own(s):
    import gnn_sparse_aggregation_b200 as ag
    if s["op"] == "diff":
        drop = dict(p=s["p"], seed=s["seed"], offset=s["offset"])
        Y, lse = ag.ag_diff_attn_fwd(s["g"], s["Q"], s["K"], s["V"], s["lam"], s["scale"], **drop)
        if not s["train"]:
            return Y, lse
        return (Y, lse) + ag.ag_diff_attn_backward(s["g"], s["Q"], s["K"], s["V"], s["lam"], s["scale"], lse,
                                                   s["dY"], **drop)
    if s["op"] == "rotary":
        return ag.ag_rotary(s["Q"], s["K"], s["pos"], s["inv_freq"], s["heads"],
                            interleaved=s["layout"] == "interleaved", factor=s["factor"], inverse=s["inverse"])
    if s["op"] == "resnorm":
        kw = dict(gamma1=s["gamma1"], beta1=s["beta1"], scale=s["rscale"], gamma2=s["gamma2"], beta2=s["beta2"],
                  eps=s["eps"], norm=s["norm"], act=s["act"], p=s["p"], seed=s["seed"], offset=s["offset"])
        if not s["back"]:
            return ag.ag_resnorm_fwd(s["R"], s["B"], s["G"], **kw)
        d = ag.ag_resnorm_backward(s["X"], s["B"], s["G"], s["dX"], s["dZ"], **kw)
        grads = (d["gamma1"], d["scale"], d["gamma2"])
        if s["norm"] == "layer":
            grads += (d["beta1"], d["beta2"])
        return (d["R"], d["B"], d["G"]) + grads
    return ag.ag_dropout(s["X"], s["p"], s["seed"], s["offset"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- in 64 bits

def _exact_mask(n, p, seed, offset):
    """The kept elements' factors, with each 32-bit product from 16-bit halves."""
    def both(a, b):
        al, ah, bl, bh = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
        mid = (al * bl >> 16) + (ah * bl & 0xFFFF) + (al * bh & 0xFFFF)
        return ah * bh + (ah * bl >> 16) + (al * bh >> 16) + (mid >> 16), (mid << 16 | al * bl & 0xFFFF) & U32
    quad = torch.arange((n + 3) // 4, dtype=torch.int64, device=DEV)
    x = [quad & U32, quad >> 32, torch.zeros_like(quad) + (offset & U32), torch.zeros_like(quad) + (offset >> 32)]
    key = [seed & U32, seed >> 32 & U32]
    for r in range(10):
        h0, l0 = both(x[0], 0xD2511F53)
        h1, l1 = both(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ ((key[0] + r * 0x9E3779B9) & U32), l1, h0 ^ x[3] ^ ((key[1] + r * 0xBB67AE85) & U32), l0]
    kept = torch.stack(x, dim=-1).reshape(-1)[:n] >= int(p * 2 ** 32 + 0.5)
    return torch.where(kept, 1.0 / (1.0 - p), 0.0).double()


def _exact_diff(s):
    N, h = s["N"], s["heads"]
    leaves = {k: s[k].double().requires_grad_(s["train"]) for k in ("Q", "K", "V", "lam")}
    order = torch.argsort(s["dst"].long(), stable=True)                              # edges by destination
    src, dst = s["src"].long()[order], s["dst"].long()[order]
    q = leaves["Q"].view(N, 2 * h, -1).index_select(0, dst)
    k = leaves["K"].view(N, 2 * h, -1).index_select(0, src)
    logit = torch.einsum("emd,emd->em", q, k) * s["scale"]                           # [E, 2h]
    deg = torch.bincount(dst, minlength=N)
    with torch.no_grad():
        peak = torch.segment_reduce(logit.detach(), "max", lengths=deg, axis=0, initial=-math.inf)
    w = (logit - peak[dst]).exp()
    norm = torch.zeros(N, 2 * h, dtype=torch.float64, device=DEV).index_add(0, dst, w)
    a = (w / norm[dst]).view(-1, h, 2)
    coef = a[..., 0] - leaves["lam"] * a[..., 1]
    if s["p"] > 0:
        coef = coef * _exact_mask(s["E"] * h, s["p"], s["seed"], s["offset"]).view(-1, h)[order]
    v = leaves["V"].view(N, h, -1).index_select(0, src)
    Y = torch.zeros(N, h, v.shape[2], dtype=torch.float64, device=DEV).index_add(0, dst, coef.unsqueeze(-1) * v)
    lse = (peak + norm.detach().log()).view(N, h, 2)
    if not s["train"]:
        return Y.reshape(N, -1).detach(), lse
    grads = torch.autograd.grad((Y.reshape(N, -1) * s["dY"].double()).sum(), [leaves[k] for k in ("Q", "K", "V", "lam")])
    return (Y.detach().reshape(N, -1), lse) + tuple(grads)


def _exact_rotary(s, X):
    N, h, rot = s["N"], s["heads"], s["rot"]
    x = X.double().view(N, h, -1)
    if s["layout"] == "half":
        z = torch.complex(x[..., : rot // 2], x[..., rot // 2: rot])
    else:
        z = torch.view_as_complex(x[..., :rot].reshape(N, h, rot // 2, 2).contiguous())
    angle = torch.outer(s["pos"].double(), s["inv_freq"])
    turn = torch.polar(torch.full_like(angle, s["factor"]), -angle if s["inverse"] else angle)
    z = z * turn.unsqueeze(1)
    first = torch.cat([z.real, z.imag], -1) if s["layout"] == "half" else torch.view_as_real(z).reshape(N, h, rot)
    return torch.cat([first, x[..., rot:]], -1).reshape(N, -1)


def _exact_resnorm(s):
    back, layer = s["back"], s["norm"] == "layer"
    names = ["X" if back else "R", "B", "G", "gamma1", "rscale", "gamma2"] + (["beta1", "beta2"] if layer else [])
    v = {k: s[k].double().requires_grad_(back) for k in names}

    def normed(x, gamma, beta):
        mean = x.mean(-1, keepdim=True) if layer else 0.0
        power = (x - mean).square().mean(-1, keepdim=True)
        y = (x - mean) / (power + s["eps"]).sqrt() * v[gamma]
        return y + v[beta] if layer else y

    gate = torch.sigmoid(v["G"]) if s["act"] == "sigmoid" else v["G"] * torch.sigmoid(v["G"])
    branch = gate * normed(v["B"], "gamma1", "beta1")
    if s["p"] > 0:
        branch = branch * _exact_mask(branch.numel(), s["p"], s["seed"], s["offset"]).view_as(branch)
    if not back:
        X = v["R"] + v["rscale"] * branch
        return X, normed(X, "gamma2", "beta2")
    second = ["X", "gamma2"] + (["beta2"] if layer else [])
    g2 = dict(zip(second, torch.autograd.grad(normed(v["X"], "gamma2", "beta2"), [v[k] for k in second], s["dZ"].double())))
    dR = s["dX"].double() + g2["X"]
    first = ["B", "G", "gamma1", "rscale"] + (["beta1"] if layer else [])
    g1 = dict(zip(first, torch.autograd.grad(v["rscale"] * branch, [v[k] for k in first], dR)))
    out = (dR, g1["B"], g1["G"], g1["gamma1"], g1["rscale"], g2["gamma2"])
    return out + ((g1["beta1"], g2["beta2"]) if layer else ())


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "diff":
        return _exact_diff(s)
    if s["op"] == "rotary":
        return _exact_rotary(s, s["Q"]), _exact_rotary(s, s["K"])
    if s["op"] == "resnorm":
        return _exact_resnorm(s)
    X = s["X"].double()
    return X * _exact_mask(X.numel(), s["p"], s["seed"], s["offset"]).view_as(X)


# ------------------------------------------------------------------- work

def work(case):
    """Each input read once, each output written once; the products' flops."""
    b = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "diff":
        N, E, H, h = case["N"], case["E"], case["H"], case["heads"]
        index = 4 * (N + 1) + 4 * E + (4 * E if case["p"] > 0 else 0)
        n = index + 4 * N * H * b + 8 * N * h + 4 * h
        f = 4 * E * H
        if case["train"]:
            n += 2 * index + 7 * N * H * b + 8 * N * h + 8 * h
            f += 10 * E * H
        return {"bytes": n, "flops": f}
    if case["op"] == "rotary":
        return {"bytes": 4 * case["N"] * case["H"] * b + 8 * case["N"] + 4 * case["rot"],
                "flops": 6 * case["N"] * case["heads"] * case["rot"]}
    if case["op"] == "resnorm":
        n = case["N"] * case["H"]
        per = 8 if case["back"] else 5
        return {"bytes": per * n * b + 20 * case["H"], "flops": (45 if case["back"] else 20) * n}
    n = case["rows"] * case["H"]
    return {"bytes": 2 * n * b, "flops": n}
