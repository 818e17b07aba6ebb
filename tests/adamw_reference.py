"""The AdamW step in float64 from its formulas, with bounds on the error of a
computation in fp32, and the 8-bit states' codes from their definition.
Nothing here uses the package."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
BLOCK = 32
MASK = 0xFFFFFFFF


def hash32(x):
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & MASK
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & MASK
    return x ^ (x >> 16)


def random_bits(n, seed, step, index, device="cpu"):
    """32 bits of each element of the index-th tensor in one step."""
    key = (seed * 0x9E3779B1 + step * 0x85EBCA77 + index * 0xC2B2AE3D) & MASK
    return hash32((torch.arange(n, device=device) & MASK) ^ key)


def blocks(x):
    more = -x.numel() % BLOCK
    return torch.cat([x, x.new_zeros(more)]).view(-1, BLOCK)


def exponents(x):
    """The least k, for each block, with every |x| <= 448 * 2^k (0 for a
    block of zeros, never under -126)."""
    top = blocks(x.abs()).amax(1)
    mant, e = torch.frexp(top)          # top = mant * 2^e, mant in [0.5, 1)
    k = e - 9 + (mant > 0.875)          # 448 = 0.875 * 2^9
    return torch.where(top == 0, 0, k.clamp(min=-126)).to(torch.int64)


def ldexp(x, k):
    """x * 2^k exactly (torch.ldexp goes through a power that is not exact on
    every device)."""
    return x * ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def per_element(k, n):
    return k.repeat_interleave(BLOCK)[:n]


def grid(y):
    """(largest e4m3 value <= y, step to the next) for 0 <= y <= 448."""
    mant, e = torch.frexp(y.clamp(min=2.0 ** -6))
    step = ldexp(torch.ones_like(y), e - 4)
    return (y / step).floor() * step, step


def quantize(x, bits16, root):
    """float64 values and 16 random bits of each -> (e4m3 values, exponents
    + 127)."""
    n = x.numel()
    k = exponents(x)
    y = ldexp(x.abs(), -per_element(k, n))
    low, step = grid(y)
    up = (y - low) / step + bits16.double() / 2 ** 16 >= 1
    q = torch.where(up, low + step, low)
    if root:
        q = torch.where((q == 0) & (x > 0), 2.0 ** -9, q)
    return torch.copysign(q, x), k + 127


def dequantize(codes, scale):
    n = codes.numel()
    return ldexp(codes.double().reshape(-1),
                       per_element(scale.long() - 127, n))


def step(x, g, m, v, t, lr, b1, b2, eps, decay, factor=1.0):
    """((x, bound), (m, bound), (v, bound)) after one step, in float64; the
    bounds are first order in U, one for each fp32 operation."""
    g = g * factor
    eg = U * g.abs()
    m1, c1 = b1 * m, (1 - b1) * g
    m = m1 + c1
    em = (1 - b1) * eg + 3 * U * (m1.abs() + c1.abs())
    v1, c2 = b2 * v, (1 - b2) * g * g
    v = v1 + c2
    ev = 2 * (1 - b2) * g.abs() * eg + 4 * U * (v1 + c2)
    size, unbias = lr / (1 - b1 ** t), (1 - b2 ** t) ** -0.5
    root = v.sqrt()
    den = root * unbias + eps
    # half of v's relative error in the root; its rounding, and three more;
    # the reciprocal and two products
    rel = torch.where(v > 0, ev / (2 * v.clamp(min=1e-300)), 0) + 8 * U
    upd = size * m / den
    eu = size * em / den + upd.abs() * rel
    new = x - (lr * decay * x + upd)
    ex = eu + 3 * U * (x.abs() + upd.abs() + lr * decay * x.abs())
    return (new, ex), (m, em), (v, ev)


def factor(norm, max_norm):
    return min(1.0, max_norm / (norm + 1e-6)) if math.isfinite(norm) else 0.0
