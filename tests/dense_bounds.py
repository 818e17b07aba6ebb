"""Linear layers, the feed-forward block and their gradients in float64 from
their formulas, each element with a bound on the error of a computation that
accumulates in fp32 and rounds to the layer's type where the kernels are
documented to round: hidden activations and pre-activations' gradients
between two products, results once.  A bound is first order and linear in the
number of roundings: U = 2^-24 for each fp32 operation that a value passes,
half a step for each rounding to the layer's type.  Nothing here uses the
package."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
GATED = {"swiglu": "silu", "geglu": "gelu"}
# largest slopes of GELU and SiLU (1.129, 1.100) and of their derivatives
# (2 phi(0) = 0.798, 0.5); errors of the kernels' own GELU and SiLU: 1.2e-7
# of the tail, a few U of the rest
SLOPE, CURVE, OWN = 1.13, 0.8, 32 * U


def act(name, z, u=None):
    """h, dh/dz, dh/du."""
    if name == "none":
        return z, torch.ones_like(z), None
    if GATED.get(name, name) == "gelu":
        cdf = torch.special.ndtr(z)
        a = z * cdf
        da = cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        s = torch.sigmoid(z)
        a, da = z * s, s * (1 + z * (1 - s))
    return (a, da, None) if u is None else (a * u, da * u, a)


def project(x, w, b):
    """x w^T + b and its error."""
    z, size = x @ w.t(), x.abs() @ w.abs().t()
    if b is not None:
        z, size = z + b, size + b.abs()
    return z, U * (x.shape[1] + 4) * size


def unit(name, x, w, b, w3, b3):
    """(value, error) of h, dh/dz and dh/du (None)."""
    z, ez = project(x, w, b)
    if name == "none":
        return (z, ez), (torch.ones_like(z), 0 * z), None
    a, da, _ = act(GATED.get(name, name), z)
    ea = SLOPE * ez + OWN * z.abs()
    eda = CURVE * ez + OWN * (1 + z.abs())
    if name not in GATED:
        return (a, ea), (da, eda), None
    u, eu = project(x, w3, b3)
    return ((a * u, ea * u.abs() + (a.abs() + ea) * eu + U * (a * u).abs()),
            (da * u, eda * u.abs() + (da.abs() + eda) * eu +
             U * (da * u).abs()), (a, ea))


def rounded(v, e, half):
    return v, e + half * v.abs()


def add(v, e, other, half):
    """(v + other), rounded to the type."""
    if other is not None:
        e = e + U * (v.abs() + other.abs())
        v = v + other
    return rounded(v, e, half)


def times(a, b):
    (v, e), (w, f) = a, b
    return v * w, e * w.abs() + (v.abs() + e) * f + U * (v * w).abs()


def matmul(a, b, more=0):
    """The product of two (value, error)s, ``more`` terms beside its own."""
    (v, e), (w, f) = a, b
    n = v.shape[1] + 8 + more
    return v @ w, e @ w.abs() + (v.abs() + e) @ f + U * n * (v.abs() @ w.abs())


def total(a):
    v, e = a
    return v.sum(0), e.sum(0) + U * (v.shape[0] + 8) * v.abs().sum(0)


def plus(a, b):
    return a[0] + b[0], a[1] + b[1] + U * (a[0].abs() + b[0].abs())


def exactly(v):
    return v, torch.zeros_like(v)


def turned(a):
    return a[0].t(), a[1].t()


def linear(name, half, x, w, b, w3, b3, res):
    h, _, _ = unit(name, x, w, b, w3, b3)
    return add(*h, res, half)


def _down(dz, du, w, w3, dx_add, half):
    dx = matmul(dz, exactly(w))
    if du is not None:
        dx = plus(dx, matmul(du, exactly(w3)))
    return add(*dx, dx_add, half)


def linear_grad(name, half, x, w, b, w3, b3, dy, dx_add):
    _, hz, hu = unit(name, x, w, b, w3, b3)
    q = exactly(dy)
    dz = q if name == "none" else rounded(*times(q, hz), half)
    du = None if hu is None else rounded(*times(q, hu), half)
    g = {"x": _down(dz, du, w, w3, dx_add, half),
         "w": rounded(*matmul(turned(dz), exactly(x)), half),
         "b": rounded(*total(dz), half)}
    if du is not None:
        g["w3"] = rounded(*matmul(turned(du), exactly(x)), half)
        g["b3"] = rounded(*total(du), half)
    return g


def dense(name, half, x, w1, w2, w3, b1, b2, b3, res):
    h, _, _ = unit(name, x, w1, b1, w3, b3)
    y = matmul(rounded(*h, half), exactly(w2.t()), 4)
    if b2 is not None:
        y = plus(y, exactly(b2.expand_as(y[0])))
    return add(*y, res, half)


def dense_grad(name, half, x, w1, w2, w3, b1, b2, b3, dy, dx_add):
    h, hz, hu = unit(name, x, w1, b1, w3, b3)
    q = matmul(exactly(dy), exactly(w2))
    dz = rounded(*times(q, hz), half)
    du = None if hu is None else rounded(*times(q, hu), half)
    g = {"x": _down(dz, du, w1, w3, dx_add, half),
         "w1": rounded(*matmul(turned(dz), exactly(x)), half),
         "w2": rounded(*matmul(exactly(dy.t()), rounded(*h, half)), half),
         "b1": rounded(*total(dz), half),
         "b2": rounded(*total(exactly(dy)), half)}
    if du is not None:
        g["w3"] = rounded(*matmul(turned(du), exactly(x)), half)
        g["b3"] = rounded(*total(du), half)
    return g


def check(got, want, half, roundings, what):
    """Each element within its bound; and, of many elements, the norm: a
    rounding to the type is off by at most half a step of each value, evenly
    spread between -1 and 1 of it, and so by 1/sqrt(3) of it in the mean of
    squares; ``roundings`` of them behind one another are independent."""
    value, bound = want
    got = got.double()
    assert got.shape == value.shape, f"{what}: shape {tuple(got.shape)}"
    over = (got - value).abs() > bound * 1.001 + 1e-37
    bad = int((over | ~torch.isfinite(got)).sum())
    assert bad == 0, f"{what}: {bad} of {value.numel()} elements off"
    if value.numel() >= 4096 and half > U:
        size, err = float(value.norm()), float((got - value).norm())
        most = 1.1 * half * math.sqrt(roundings / 3)
        assert err <= most * size, \
            f"{what}: error {err / size:.3g} of the norm, allowed {most:.3g}"
