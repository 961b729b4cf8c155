"""Differential edge-softmax attention in 64 bits, and error bounds of its fp32
path that weigh every edge by its softmax weight (torch, on any device;
imported only by test files; no code shared with the library).

layer_oracle.diff_bounds takes the largest |dY| |V| of a row for all of its
edges, which says nothing where an edge of negligible weight has a large V row,
and sums a row over at most 256 positions of a tile.  Here an edge's terms count
by their weight, and a walk's tile is TILE positions.

Arithmetic, with U = 2^-24, B_e = scale sum |q k| of an edge and row r = dst_e:
  rho_e  a score is d products and sums and a scaling: (d + 8) U B_e.  The
         exponent less its reference is rounded to |ln alpha_e| + ln cnt + 8
         at most (a reference is at most 8 powers of two below the row's
         maximum), ex2 and the division are off by 8 U together.  Twice that.
         A weight below 2^-125 may be taken for 0 (fp32 has no normal number
         below 2^-126): 1.
  steps  16 + min(cnt, TILE) + cnt / 32 roundings of a row's sums.
  weight alpha_e is off by rho_e, and by the row's sum: rho_r = sum alpha rho
         + steps U.
  del_e  da is 2 d products and sums: (2 d + 8) U M_e, M_e = u sum |dY v|.
  D      sum alpha da: Dd_r = sum alpha (rho_e + rho_r) |da| + sum alpha del_e
         + steps U sum alpha |da|.
  ds     scale alpha (da - D): scale alpha ((rho_e + rho_r)(|da| + |D|) + del_e + Dd_r).
  dq     the sum of ds k, walked as sums of alpha da k and of alpha k: their
         roundings are steps U times the sums of alpha |da| |k| and of
         sum alpha |da| alpha |k|, twice.
  lse    sum alpha rho + steps U + 4 U |lse|.
  dK, dV recompute alpha from the rounded lse: 8 U (|lse| + 1) more.
  Outputs are rounded once to their type, half a step, or 2^-126 below its normal
  numbers.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
TILE = 1024
TINY = 2.0 ** -126


def reference(src, dst, N, Q, K, V, lam, scale, u=None, dY=None):
    """fp64 tensors (src, dst int64; u [E, heads] or None): Y, lse and, with dY,
    dQ, dK, dV, dlam; the terms s, a, w, da, D that the bounds use."""
    h = lam.shape[0]
    d = Q.shape[1] // (2 * h)
    E, dev = src.shape[0], Q.device
    total = lambda i, x: torch.zeros((N,) + x.shape[1:], dtype=torch.float64, device=dev).index_add_(0, i, x)
    q, k, v = Q.view(N, h, 2, d), K.view(N, h, 2, d), V.view(N, h, 2 * d)
    u = torch.ones(E, h, dtype=torch.float64, device=dev) if u is None else u
    s = (q[dst] * k[src]).sum(3) * scale
    top = torch.full((N, h, 2), -torch.inf, dtype=torch.float64, device=dev)
    top = top.scatter_reduce(0, dst.view(E, 1, 1).expand(E, h, 2), s, "amax")
    e = torch.exp(s - top[dst])
    z = total(dst, e)
    a = e / z[dst]
    w = u * (a[..., 0] - lam * a[..., 1])
    out = dict(Y=total(dst, w[..., None] * v[src]).view(N, -1), lse=top + torch.log(z), s=s, a=a, w=w)
    if dY is None:
        return out
    g = dY.view(N, h, 2 * d)
    da = u * (g[dst] * v[src]).sum(2)
    D = total(dst, a * da[..., None])
    coef = torch.stack([torch.ones_like(lam), -lam], 1) * scale
    ds = coef * a * (da[..., None] - D[dst])
    out.update(dQ=total(dst, ds[..., None] * k[src]).view(N, -1), dK=total(src, ds[..., None] * q[dst]).view(N, -1),
               dV=total(src, w[..., None] * g[dst]).view(N, -1), dlam=-D[..., 1].sum(0), da=da, D=D)
    return out


def bounds(src, dst, N, Q, K, V, lam, scale, u, ref, dtype, dY=None):
    """Bounds per element of what `reference` computes, outputs rounded to `dtype`."""
    h = lam.shape[0]
    d = Q.shape[1] // (2 * h)
    E, dev = src.shape[0], Q.device
    total = lambda i, x: torch.zeros((N,) + x.shape[1:], dtype=torch.float64, device=dev).index_add_(0, i, x)
    u = torch.ones(E, h, dtype=torch.float64, device=dev) if u is None else u
    q, k, v = Q.abs().view(N, h, 2, d), K.abs().view(N, h, 2, d), V.abs().view(N, h, 2 * d)
    half = torch.finfo(dtype).eps / 2
    al = torch.stack([torch.ones_like(lam), lam.abs()], 1)                       # [h, 2]
    a, sc = ref["a"], abs(scale)
    cnt = torch.bincount(dst, minlength=N).double().view(N, 1, 1)
    cnt_s = torch.bincount(src, minlength=N).double().view(N, 1, 1)
    steps = lambda c: (16 + c.clamp(max=TILE) + c / 32) * U
    B = (q[dst] * k[src]).sum(3) * sc
    far = (a.clamp(min=1e-300).log().abs() + torch.log(cnt)[dst] + 8).clamp(max=200.0)   # (smaller weights: below)
    rho = 2 * ((d + 8) * U * B + U * far + 8 * U) + (a < 2 * TINY).double()      # [E, h, 2]
    rho_r = total(dst, a * rho) + steps(cnt)
    both = rho + rho_r[dst]
    lse = ref["lse"]
    fin = torch.isfinite(lse)
    out = dict(lse=torch.where(fin, rho_r + 4 * U * torch.where(fin, lse, 0.0).abs(), 0.0))
    absw = u[..., None] * al * a
    out["Y"] = total(dst, (absw * both).sum(2)[..., None] * v[src]).view(N, -1) + half * ref["Y"].abs() + TINY
    if dY is None:
        return out
    g = dY.abs().view(N, h, 2 * d)
    M = u * (g[dst] * v[src]).sum(2)                                             # [E, h]
    da, D = ref["da"].abs()[..., None], ref["D"].abs()
    dele = ((2 * d + 8) * U * M)[..., None]
    ada = a * da
    A1 = total(dst, ada)                                                         # sum alpha |da|
    Dd = total(dst, ada * both + a * dele) + steps(cnt) * A1
    own = a * (both * (da + D[dst]) + dele + Dd[dst])                            # ds / scale
    bq = total(dst, own[..., None] * k[src])
    ak = total(dst, a[..., None] * k[src])
    round_q = 2 * steps(cnt)[..., None] * (total(dst, ada[..., None] * k[src]) + A1[..., None] * ak)
    out["dQ"] = ((bq + round_q) * (sc * al)[..., None]).view(N, -1) + half * ref["dQ"].abs() + TINY
    again = 8 * U * (torch.where(fin, lse, 0.0).abs() + 1)[dst]                  # alpha from the rounded lse
    full = a * (da + D[dst])
    bk = (own + full * (again + steps(cnt_s)[src])) * sc * al
    out["dK"] = total(src, bk[..., None] * q[dst]).view(N, -1) + half * ref["dK"].abs() + TINY
    bv = (absw * (both + again + steps(cnt_s)[src])).sum(2)
    out["dV"] = total(src, bv[..., None] * g[dst]).view(N, -1) + half * ref["dV"].abs() + TINY
    out["dlam"] = Dd[..., 1].sum(0) + U * ref["dlam"].abs()
    return out
