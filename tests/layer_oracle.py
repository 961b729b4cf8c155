"""Plain 64-bit forms of the differential attention layer's operators (numpy
and torch on the CPU; imported only by test files).  They share no code with
the library."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------- the generator

def philox(counter, key):
    """Philox4x32-10 of [n, 4] counters and [n, 2] keys (uint64 arrays holding 32-bit words)."""
    c = [np.asarray(counter[..., i], np.uint64) for i in range(4)]
    k = [np.asarray(key[..., i], np.uint64) for i in range(2)]
    low, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        m0, m1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(m1 >> s32) ^ c[1] ^ k[0], m1 & low, (m0 >> s32) ^ c[3] ^ k[1], m0 & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return np.stack(c, -1)


def keep_mask(n, p, seed, offset, first=0):
    """Truth values of elements first .. first + n - 1."""
    i = np.arange(first, first + n, dtype=np.uint64)
    block, word = i >> np.uint64(2), (i & np.uint64(3)).astype(np.int64)
    low, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    off, sd = np.uint64(offset), np.uint64(seed)
    ctr = np.stack([block & low, block >> s32, np.full_like(block, off & low), np.full_like(block, off >> s32)], -1)
    key = np.stack([np.full_like(block, sd & low), np.full_like(block, sd >> s32)], -1)
    w = philox(ctr, key)[np.arange(n), word]
    return w >= np.uint64(int(np.rint(p * 2.0 ** 32)))


def drop_factors(n, p, seed, offset):
    if p == 0:
        return np.ones(n)
    return keep_mask(n, p, seed, offset) / (1.0 - p)


# ------------------------------------------------------------------- differential attention

def diff_attention(src, dst, N, Q, K, V, lam, scale, u=None, dY=None):
    """fp64 arrays: a dict of Y, lse and, with dY, dQ, dK, dV, dlam; and the
    per-edge terms that the error bounds are made of.  u: [E, heads] factors."""
    h = lam.shape[0]
    d = Q.shape[1] // (2 * h)
    E = src.shape[0]
    q, k = Q.reshape(N, h, 2, d), K.reshape(N, h, 2, d)
    v = V.reshape(N, h, 2 * d)
    u = np.ones((E, h)) if u is None else u
    s = np.einsum("ehmd,ehmd->ehm", q[dst], k[src]) * scale
    top = np.full((N, h, 2), -np.inf)
    np.maximum.at(top, dst, s)
    e = np.exp(s - top[dst])
    total = np.zeros((N, h, 2))
    np.add.at(total, dst, e)
    a = e / total[dst]
    with np.errstate(divide="ignore"):
        lse = top + np.log(total)
    w = u * (a[..., 0] - lam * a[..., 1])
    Y = np.zeros((N, h, 2 * d))
    np.add.at(Y, dst, w[..., None] * v[src])
    out = dict(Y=Y.reshape(N, -1), lse=lse, s=s, a=a, w=w)
    if dY is None:
        return out
    g = dY.reshape(N, h, 2 * d)
    da = u * np.einsum("ehd,ehd->eh", g[dst], v[src])
    D = np.zeros((N, h, 2))
    np.add.at(D, dst, a * da[..., None])
    coef = np.stack([np.ones(h), -lam], 1) * scale
    ds = coef * a * (da[..., None] - D[dst])
    dQ, dK, dV = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    np.add.at(dQ, dst, ds[..., None] * k[src])
    np.add.at(dK, src, ds[..., None] * q[dst])
    np.add.at(dV, src, w[..., None] * g[dst])
    out.update(dQ=dQ.reshape(N, -1), dK=dK.reshape(N, -1), dV=dV.reshape(N, -1), dlam=-D[..., 1].sum(0), da=da)
    return out


def diff_bounds(src, dst, N, Q, K, V, lam, scale, u, ref, dtype, dY=None):
    """Error bounds per element of the fp32 path, from its arithmetic.

    * A score is d products and sums in fp32, a scaling and the subtraction of
      the row's maximum: off by at most t_r = (d + 16) U scale max_e sum |q k|
      over the row's edges (|s| itself is at most scale sum |q k|).  Both that
      and the maximum move a map's value by at most expm1(2 t_r), relative.
    * ex2 is off by 4 U, relative.  A row's sums run over at most 256 positions
      of a tile, then over its tiles (at least 32 positions each), each step
      rounding the sum and possibly a rescaling: depth_r = 16 + min(cnt, 256)
      + cnt / 32 steps of at most 4 U.  rho_r is the two together.
    * da is 2 d products and sums: (2 d + 8) U sum |dY v| u, at most
      M_r = max over the row's edges of u sum |dY v|.  da - c and D are at most
      2 M_r, so ds is off by (rho_r + (2 d + 8) U) 4 M_r scale alpha.
    * outputs are rounded once to their type: half a step of the value.
    """
    h = lam.shape[0]
    d = Q.shape[1] // (2 * h)
    al = np.abs(np.stack([np.ones(h), lam], 1))
    q, k = np.abs(Q).reshape(N, h, 2, d), np.abs(K).reshape(N, h, 2, d)
    v = np.abs(V).reshape(N, h, 2 * d)
    B = np.einsum("ehmd,ehmd->ehm", q[dst], k[src]) * abs(scale)
    Bmax = np.zeros((N, h, 2))
    np.maximum.at(Bmax, dst, B)
    cnt = np.bincount(dst, minlength=N).astype(np.float64)[:, None, None]
    cnt_s = np.bincount(src, minlength=N).astype(np.float64)[:, None, None]
    steps = lambda c: 4 * U * (16 + np.minimum(c, 256) + c / 32)
    t = (d + 16) * U * Bmax
    rho = np.expm1(2 * t) + steps(cnt)                                   # [N, h, 2]
    half = half_step(dtype)
    a, absw = ref["a"], u[..., None] * al * ref["a"]                     # [E, h, 2]
    bY = np.zeros((N, h, 2 * d))
    np.add.at(bY, dst, (absw * rho[dst]).sum(-1)[..., None] * v[src])
    out = dict(Y=bY.reshape(N, -1) + half * np.abs(ref["Y"]),
               lse=np.where(np.isfinite(ref["lse"]), t + steps(cnt) + 4 * U * np.abs(ref["lse"]), 0.0))
    if dY is None:
        return out
    g = np.abs(dY).reshape(N, h, 2 * d)
    Bda = u * np.einsum("ehd,ehd->eh", g[dst], v[src])
    M = np.zeros((N, h))
    np.maximum.at(M, dst, Bda)
    r = rho[dst] + (2 * d + 8) * U
    dds = 4 * abs(scale) * al * a * r * M[dst][..., None]
    full = abs(scale) * al * a * 2 * M[dst][..., None]                   # at least |ds|
    bQ, bK, bV = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    np.add.at(bQ, dst, dds[..., None] * k[src])
    np.add.at(bK, src, (dds + full * steps(cnt_s)[src])[..., None] * q[dst])
    np.add.at(bV, src, (absw * (rho[dst] + steps(cnt_s)[src])).sum(-1)[..., None] * g[dst])
    bl = (4 * a * r * M[dst][..., None])[..., 1].sum(0) + half_step(torch.float32) * np.abs(ref["dlam"])
    out.update({k_: b.reshape(N, -1) + half * np.abs(ref[k_]) for k_, b in (("dQ", bQ), ("dK", bK), ("dV", bV))}, dlam=bl)
    return out


# ------------------------------------------------------------------- rotary positions

def rotary(X, pos, inv_freq, heads, interleaved, factor, inverse):
    N, H = X.shape
    rot = 2 * inv_freq.shape[0]
    x = X.reshape(N, heads, -1).astype(np.float64).copy()
    a = pos[:, None].astype(np.longdouble) * inv_freq.astype(np.longdouble)
    c, s = (factor * np.cos(a)).astype(np.float64)[:, None], (factor * np.sin(a)).astype(np.float64)[:, None]
    if inverse:
        s = -s
    i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    x0, x1 = x[..., i0].copy(), x[..., i1].copy()
    x[..., i0], x[..., i1] = x0 * c - x1 * s, x1 * c + x0 * s
    return x.reshape(N, H)


# ------------------------------------------------------------------- norm, gate and residual

def resnorm(R, B, G, v, eps, layer, silu, u=None, dX=None, dZ=None, X=None):
    """torch fp64 tensors (None: absent); v: dict of gamma1, beta1, scale,
    gamma2, beta2 (None: absent).  Without dX and dZ: (X, Z).  With either: a
    dict of the gradients, by autograd, from the stored sum X."""
    own = lambda t: None if t is None else t.clone()
    B, G, v = own(B), own(G), {k: own(t) for k, t in v.items()}

    def norm(x, gamma, beta):
        c = x - x.mean(1, keepdim=True) if layer else x
        y = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
        y = y if v[gamma] is None else y * v[gamma]
        return y if v[beta] is None else y + v[beta]

    def branch():
        y = norm(B, "gamma1", "beta1")
        if G is not None:
            s = torch.sigmoid(G)
            y = y * (G * s if silu else s)
        y = y if u is None else y * u
        return y if v["scale"] is None else y * v["scale"]

    if dX is None and dZ is None:
        X = R if B is None else (branch() if R is None else R + branch())
        return X, norm(X, "gamma2", "beta2")
    leaves = {"B": B, "G": G, **{k: t for k, t in v.items() if t is not None}}
    leaves = {k: t for k, t in leaves.items() if t is not None}
    for t in leaves.values():
        t.requires_grad_(True)
    out = {}
    dR = torch.zeros_like(dZ if dX is None else dX) if dX is None else dX.clone()
    if dZ is not None:
        x = X.clone().requires_grad_(True)
        second = [k for k in ("gamma2", "beta2") if k in leaves]
        got = torch.autograd.grad(norm(x, "gamma2", "beta2"), [x] + [leaves[k] for k in second], dZ)
        dR = dR + got[0]
        out.update(zip(second, got[1:]))
    out["R"] = dR
    if B is not None:
        first = [k for k in ("B", "G", "gamma1", "beta1", "scale") if k in leaves]
        out.update(zip(first, torch.autograd.grad(branch(), [leaves[k] for k in first], dR)))
    return {k: t.detach() for k, t in out.items()}
