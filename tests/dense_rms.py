"""Single-precision linear layers, the feed-forward block and their gradients
in float64, each element with the variance of the error of a computation in
fp32: what dense_bounds adds up in the worst case, here as the mean square of
independent roundings.  It is for inputs of which every product's terms are
independent with zero mean (one operand is random, as the tests' inputs are):
a worst-case bound grows with the depth, this with its root, and so sees
operands that lost bits on the way.

An fp32 operation is off by at most U = 2^-24 of its result, evenly spread,
and so by U^2 / 3 in the mean of squares.  A sum of n terms t, one after
another, has partial sums of at most sum t^2 in the mean of squares, so the
variance of its error is at most n U^2 / 3 sum t^2.  Nothing here uses the
package."""
from __future__ import annotations

import math

import torch

from dense_bounds import CURVE, GATED, OWN, SLOPE, U, act, exactly, turned

V = U * U / 3


def tiled(depth):
    """Terms one after another where 64 are added up before they join the
    total."""
    return 64 + depth / 64


def streamed(depth):
    """The same where few rows may go through the streaming kernel, whose four
    waves add up a quarter of the depth each."""
    return 64 + depth / 4


def chain(rows, depth):
    return streamed(depth) if rows <= 64 else tiled(depth)


def columns(rows):
    """Of a bias gradient: ranges of 256 rows, eight side by side, and the
    ranges by fours."""
    return 32 + 8 + rows / 1024 + 4


def project(x, w, b):
    z = x @ w.t()
    e = V * chain(*x.shape) * (x ** 2 @ (w ** 2).t())
    if b is not None:
        z = z + b
    return z, e + V * z ** 2


def times(a, b):
    (v, e), (w, f) = a, b
    return v * w, e * w ** 2 + v ** 2 * f + V * (v * w) ** 2


def plus(a, b):
    v = a[0] + b[0]
    return v, a[1] + b[1] + V * v ** 2


def unit(name, x, w, b, w3, b3):
    """(value, variance) of h, dh/dz and dh/du (None)."""
    z, ez = project(x, w, b)
    if name == "none":
        return (z, ez), exactly(torch.ones_like(z)), None
    a, da, _ = act(GATED.get(name, name), z)
    ea = SLOPE ** 2 * ez + (OWN * z) ** 2
    eda = CURVE ** 2 * ez + (OWN * (1 + z.abs())) ** 2
    if name not in GATED:
        return (a, ea), (da, eda), None
    u = project(x, w3, b3)
    return times((a, ea), u), times((da, eda), u), (a, ea)


def matmul(a, b, n):
    (v, e), (w, f) = a, b
    return v @ w, e @ w ** 2 + v ** 2 @ f + V * n * (v ** 2 @ w ** 2)


def total(a):
    v, e = a
    return v.sum(0), e.sum(0) + V * columns(len(v)) * (v ** 2).sum(0)


def add(a, other):
    return a if other is None else plus(a, exactly(other))


def linear(name, x, w, b, w3, b3, res):
    return add(unit(name, x, w, b, w3, b3)[0], res)


def _down(dz, du, w, w3, dx_add):
    n = tiled(len(w)) * (1 if du is None else 2)
    dx = matmul(dz, exactly(w), n)
    if du is not None:
        dx = plus(dx, matmul(du, exactly(w3), n))
    return add(dx, dx_add)


def _weights(a, x):
    return matmul(turned(a), x, tiled(len(a[0])))


def linear_grad(name, x, w, b, w3, b3, dy, dx_add):
    _, hz, hu = unit(name, x, w, b, w3, b3)
    dz = exactly(dy) if name == "none" else times(exactly(dy), hz)
    du = None if hu is None else times(exactly(dy), hu)
    g = {"x": _down(dz, du, w, w3, dx_add), "w": _weights(dz, exactly(x)),
         "b": total(dz)}
    if du is not None:
        g["w3"], g["b3"] = _weights(du, exactly(x)), total(du)
    return g


def dense(name, x, w1, w2, w3, b1, b2, b3, res):
    h = unit(name, x, w1, b1, w3, b3)[0]
    y = matmul(h, exactly(w2.t()), chain(len(x), w2.shape[1]))
    return add(y if b2 is None else plus(y, exactly(b2.expand_as(y[0]))), res)


def dense_grad(name, x, w1, w2, w3, b1, b2, b3, dy, dx_add):
    h, hz, hu = unit(name, x, w1, b1, w3, b3)
    q = matmul(exactly(dy), exactly(w2), tiled(len(w2)))
    dz = times(q, hz)
    du = None if hu is None else times(q, hu)
    g = {"x": _down(dz, du, w1, w3, dx_add), "w1": _weights(dz, exactly(x)),
         "w2": _weights(exactly(dy), h), "b1": total(dz),
         "b2": total(exactly(dy))}
    if du is not None:
        g["w3"], g["b3"] = _weights(du, exactly(x)), total(du)
    return g


def check(got, want, what):
    """The norm of the error: its square is the sum of the variances, give or
    take sqrt(2 / n) of it for n elements, six times.  Returns it as a share
    of the values' norm."""
    value, variance = want
    assert got.shape == value.shape, f"{what}: shape {tuple(got.shape)}"
    err = float((got.double() - value).norm())
    most = math.sqrt(float(variance.sum()) *
                     (1 + 6 * math.sqrt(2 / value.numel())))
    size = float(value.norm())
    assert err <= most, \
        f"{what}: error {err / size:.3g} of the norm, allowed {most / size:.3g}"
    return err / size
