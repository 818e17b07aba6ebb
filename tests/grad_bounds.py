"""The gradients of the layer in float64 from their formulas, each element
with a bound on the error of a computation that accumulates in fp32 and
rounds to the layer's type where the kernels are documented to round: the
hidden activations and their gradients between two products, the results
once, the logits' gradient to two parts.  A bound is first order and linear
in the number of roundings: u = 2^-24 for each fp32 operation that a value
passes, half a step for each rounding to the layer's type."""
from __future__ import annotations

import math

import torch

F64 = torch.float64
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def dlogits(x, wr, br, eb, r, dw, e_dw, choice, alpha, aux, z):
    """Gradient [T, E] of sum dw * topk_w + aux * l_aux + z * z-loss by the
    logits, and its bound; e_dw: the bound of dw."""
    T, d = x.shape
    E = wr.shape[0]
    l = x @ wr.t() + br - eb
    # products and sums of d terms and the two biases
    el = U * (d + 4) * (x.abs() @ wr.abs().t() + br.abs() + eb.abs())
    worst = el.max(1, keepdim=True).values
    lse = torch.logsumexp(l, 1, keepdim=True)
    p = torch.exp(l - lse)
    # relative: both logits' errors, the rounding of their difference, the
    # exponential, the sum and the division
    rel = 2 * worst + U * (E + 16 + 2 * l.abs().max(1, keepdim=True).values)
    w = r["topk_w"]
    dl, err = torch.zeros(T, E, dtype=F64), torch.zeros(T, E, dtype=F64)
    if not choice:
        mean = (w * dw).sum(1, keepdim=True)
        size = (w * dw.abs()).sum(1, keepdim=True)
        k = w.shape[1]
        e_part = w * (e_dw + (w * e_dw).sum(1, keepdim=True) +
                      U * (k + 6) * (dw.abs() + size))
        dl.scatter_add_(1, r["topk_idx"], w * (dw - mean))
        err.scatter_add_(1, r["topk_idx"], e_part)
    if choice or aux:
        # expert choice: the weight is the given p itself
        pe, pr = (w, 0.0) if choice else (p, rel)
        dp = aux * alpha * E / T * r["f"].expand(T, E)
        e_dp = 4 * U * dp.abs()
        if choice:
            dp, e_dp = dp + dw, e_dp + e_dw + U * dw.abs()
        dot = (pe * dp).sum(1, keepdim=True)
        size = (pe * dp.abs()).sum(1, keepdim=True)
        dl += pe * (dp - dot)
        err += pe * (e_dp + (pe * e_dp).sum(1, keepdim=True) +
                     pr * ((dp - dot).abs() + size) +
                     U * (E + 8) * (dp.abs() + size))
    if z:
        c = 2 * z / T
        dl += c * lse * p
        e_lse = worst + U * (E + 8 + lse.abs())
        err += c * p * (lse.abs() * (rel + 6 * U) + e_lse)
    return dl, err + 3 * U * dl.abs()


def router(x, wr, dl, e_dl, dtype):
    """dl Wr, dl^T x and the sum of dl, with bounds (before the rounding of
    a result): dl enters the bf16 products in two parts, off by half a step
    of half a step."""
    T, E = dl.shape
    e = e_dl + (HALF["bf16"] ** 2 if dtype == "bf16" else U) * dl.abs()
    a = dl.abs()
    gx = dl @ wr, e @ wr.abs() + U * (2 * E + 4) * (a @ wr.abs())
    gw = dl.t() @ x, e.t() @ x.abs() + U * (2 * T + 4) * (a.t() @ x.abs())
    gb = dl.sum(0), e_dl.sum(0) + U * (T + 4) * a.sum(0)
    return gx, gw, gb


def _act(act, z, ez):
    """h and dh/dz with bounds; |gelu'| < 1.13, |gelu''| < 0.8, |silu'| <
    1.1, |silu''| <= 0.5; the functions themselves to 2^-20 of z and 1."""
    own = 2.0 ** -20 * (1 + z.abs())
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        h = z * cdf
        hz = cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return h, 1.13 * ez + 2.0 ** -20 * z.abs(), hz, 0.8 * ez + own
    s = torch.sigmoid(z)
    return (z * s, 1.1 * ez + 2.0 ** -20 * z.abs(),
            s * (1 + z * (1 - s)), 0.5 * ez + own)


def expert(act, x, dy, w, wts, dtype):
    """One expert on its n rows, row weights w [n]: (rows' dx, its bound),
    (dr, its bound), {name: (gradient, bound with its own rounding)}."""
    half = HALF[dtype]
    n, d = x.shape
    w1, b1, w2, b2, w3, b3 = wts
    F = w1.shape[0]
    w = w[:, None]

    def up(a, m, b):
        v = a @ m.t()
        s = a.abs() @ m.abs().t()
        if b is not None:
            v, s = v + b, s + b.abs()
        return v, U * (a.shape[1] + 4) * s

    z, ez = up(x, w1, b1)
    q, eq = up(dy, w2.t(), None)
    h, eh, hz, ehz = _act(act, z, ez)
    hu = ehu = None
    if act == "swiglu":
        u, eu = up(x, w3, b3)
        a, ea, da, eda = h, eh, hz, ehz
        h, eh = a * u, ea * u.abs() + a.abs() * eu + ea * eu
        hz, ehz = da * u, eda * u.abs() + da.abs() * eu + eda * eu
        hu, ehu = a, ea
    rh = w * h
    e_rh = w * eh + (half + 2 * U) * rh.abs()

    def back(g, eg):
        v = w * q * g
        return v, w * (q.abs() * eg + eq * (g.abs() + eg)) + \
            (half + 4 * U) * v.abs()

    dz, e_dz = back(hz, ehz)
    size = (q.abs() * h.abs()).sum(1)
    dr, e_dr = (q * h).sum(1), (q.abs() * eh + eq * (h.abs() + eh)).sum(1)
    if b2 is not None:
        dr, size = dr + dy @ b2, size + dy.abs() @ b2.abs()
    e_dr = e_dr + U * (F + d + 16) * size

    def grad(l, el, r, er):
        """l^T r over the rows, rounded."""
        v = l.t() @ r
        e = el.t() @ r.abs() + U * (n + 4) * (l.abs().t() @ r.abs())
        if er is not None:
            e = e + l.abs().t() @ er
        return v, e + half * v.abs()

    def bias(v, e):
        s = v.sum(0)
        return s, e.sum(0) + U * (n + 8) * v.abs().sum(0) + half * s.abs()

    none = torch.zeros_like(dy)
    g = {"w1": grad(dz, e_dz, x, None), "b1": bias(dz, e_dz),
         "w2": grad(dy, none, rh, e_rh), "b2": bias(w * dy, U * (w * dy).abs())}
    dx, e_dx = dz @ w1, e_dz @ w1.abs()
    size = dz.abs() @ w1.abs()
    if act == "swiglu":
        du, e_du = back(hu, ehu)
        g["w3"], g["b3"] = grad(du, e_du, x, None), bias(du, e_du)
        dx, e_dx = dx + du @ w3, e_dx + e_du @ w3.abs()
        size = size + du.abs() @ w3.abs()
    return (dx, e_dx + U * (2 * F + 8) * size), (dr, e_dr), g


def layer(w, x, dy, r, act, choice, n_shared, alpha, aux, z, dtype):
    """{name: (gradient, bound)} of the whole layer, weights ``w`` and all
    else in float64."""
    T, d = x.shape
    wr = w["w_router"]
    E = wr.shape[0]
    zero = torch.zeros(E, dtype=F64)
    br, eb = (zero if w.get(n) is None else w[n]
              for n in ("b_router", "expert_bias"))
    dx, e_dx, size = (torch.zeros(T, d, dtype=F64) for _ in range(3))
    dw, e_dw = (torch.zeros(r["topk_w"].shape, dtype=F64) for _ in range(2))
    out = {n: tuple(torch.zeros(w[n].shape, dtype=F64) for _ in range(2))
           for n in ("w1", "b1", "w2", "b2", "w3", "b3")
           if w.get(n) is not None}
    for e in range(E):
        t, j = ((r["topk_idx"] == e) & (r["slot_of"] >= 0)) \
            .nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        mine = [None if w.get(n) is None else w[n][e]
                for n in ("w1", "b1", "w2", "b2", "w3", "b3")]
        rows, dr, g = expert(act, x[t], dy[t], r["topk_w"][t, j], mine, dtype)
        dx.index_add_(0, t, rows[0])
        e_dx.index_add_(0, t, rows[1])
        size.index_add_(0, t, rows[0].abs())
        dw[t, j], e_dw[t, j] = dr
        for n in out:
            out[n][0][e], out[n][1][e] = g[n]
    if n_shared:
        mine = [w.get(n) for n in ("ws1", "bs1", "ws2", "bs2", "ws3", "bs3")]
        rows, _, g = expert(act, x, dy, torch.ones(T, dtype=F64), mine, dtype)
        dx, e_dx, size = dx + rows[0], e_dx + rows[1], size + rows[0].abs()
        for n, v in g.items():
            s = n[0] + "s" + n[1]
            if w.get(s) is not None:
                out[s] = v
    dl, e_dl = dlogits(x, wr, br, eb, r, dw, e_dw, choice, alpha, aux, z)
    gx, gw, gb = router(x, wr, dl, e_dl, dtype)
    v = dx + gx[0]
    e = e_dx + gx[1] + U * (r["topk_w"].shape[1] + 4) * (size + gx[0].abs())
    out["x"] = v, e + HALF[dtype] * v.abs()
    out["w_router"] = gw[0], gw[1] + HALF[dtype] * gw[0].abs()
    out["b_router"] = gb[0], gb[1] + U * gb[0].abs()
    return out
