"""The dense layer beside the sparse one and the optimizer's step, as a user's
program calls them: sizes, inputs, the plain form of each and its definition
in 64 bits.

Operators (``case["op"]``):

``linear`` / ``linear_grad``
    y = residual + act(x W^T + b), gated: residual + a(x W^T + b) *
    (x W3^T + b3), and the gradients of x and of the weights;
``dense`` / ``dense_grad``
    the feed-forward block y = residual + W2 h + b2 with h = act(W1 x + b1),
    gated: h = a(W1 x + b1) * (W3 x + b3), and its gradient;
``adamw``
    one AdamW step over many tensors, with states in 32 or in 8 bits, with
    or without a 32-bit copy of bf16 parameters.

With ``own`` false ``run`` is the plain form in torch operations, with
``own`` true it calls the package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GATED = {"swiglu": "silu", "geglu": "gelu"}
EPS = 1e-6            # clipping: factor = min(1, max_norm / (norm + EPS))
BLOCK = 32            # elements of an 8-bit state that share a scale


def _linear(name, op, M, N, K, dtype="bf16", act="none", bias=False,
            residual=False):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "dtype": dtype,
            "act": act, "bias": bias, "residual": residual}


def _dense(name, op, T, d, d_ff, dtype="bf16", act="swiglu", bias=False,
           residual=True):
    return {"name": name, "op": op, "T": T, "d": d, "d_ff": d_ff,
            "dtype": dtype, "act": act, "bias": bias, "residual": residual}


def _adamw(name, count, low, high, dtype, bits, master=False,
           stochastic=False, clip=False, grad="same"):
    return {"name": name, "op": "adamw", "count": count, "low": low,
            "high": high, "dtype": dtype, "bits": bits, "master": master,
            "stochastic": stochastic, "clip": clip, "grad": grad}


def listed():
    return [
        # one token through a projection of a decoding step: latency, and
        # one read of the weights
        _linear("linear_one_token", "linear", 1, 4096, 4096, residual=True),
        # single precision, an odd number of rows and every part of the
        # epilogue
        _linear("linear_f32_odd", "linear", 1021, 1984, 1024, dtype="f32",
                act="gelu", bias=True, residual=True),
        # a projection over a long prompt, into the residual stream
        _linear("linear_prefill", "linear", 8192, 7168, 2048, bias=True,
                residual=True),
        # a short fine-tuning sequence: the weights and their gradient move
        _linear("linear_grad_short", "linear_grad", 33, 2816, 1024,
                act="gelu", bias=True),
        # a square projection of a training step
        _linear("linear_grad_square", "linear_grad", 4096, 4096, 4096),
        # the dense gated block at a decoding batch
        _dense("dense_decode", "dense", 32, 4096, 14336),
        # and over 4 x 1024 tokens
        _dense("dense_prefill", "dense", 4096, 4096, 14336),
        # the smallest block that the package names, with every bias
        _dense("dense_grad_tiny_f32", "dense_grad", 256, 64, 256,
               dtype="f32", act="gelu", bias=True, residual=False),
        # a training step's block, the largest
        _dense("dense_grad_large", "dense_grad", 4096, 4096, 14336),
        # the parameters of a small network, odd sizes, single precision
        _adamw("adamw_small", 20, 1, 20000, "f32", 32),
        # bf16 parameters with a 32-bit copy, clipped gradients
        _adamw("adamw_master", 10, 1 << 20, 1 << 26, "bf16", 32, master=True,
               clip=True),
        # a larger model with 8-bit states and no copy, embeddings among it
        _adamw("adamw_8bit", 10, 1 << 20, 1 << 28, "bf16", 8,
               stochastic=True, clip=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "dense",
                     "dense_grad", "adamw", "adamw"])
    if op == "adamw":
        low = _log_int(rng, 1, 1 << 20)
        high = low * _log_int(rng, 1, 1 << 10)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        c = _adamw("", rng.randint(1, 10), low, min(high, 1 << 27), dtype,
                   rng.choice([8, 32]),
                   master=dtype == "bf16" and rng.random() < 0.4,
                   stochastic=rng.random() < 0.5, clip=rng.random() < 0.5,
                   grad=rng.choice(["same", "same", "f32"]))
        del c["name"]
        return c
    dtype = rng.choice(["bf16", "bf16", "f32"])
    M = _log_int(rng, 1, 8192)
    N, K = 64 * _log_int(rng, 1, 128), 64 * _log_int(rng, 1, 128)
    limit = 2.4e11 if dtype == "bf16" else 2e10
    while M * N * K > limit:
        M = (M + 1) // 2
    bias, residual = rng.random() < 0.4, rng.random() < 0.5
    if op in ("linear", "linear_grad"):
        c = _linear("", op, M, N, K, dtype, rng.choice(
            ["none", "none", "gelu", "silu", "swiglu", "geglu"]), bias,
            residual and op == "linear")
    else:
        c = _dense("", op, M, K, N, dtype, rng.choice(
            ["gelu", "silu", "swiglu", "swiglu", "geglu"]), bias, residual)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV) \
        .normal_(0.0, std, generator=g)


def _sizes(case):
    n, low, high = case["count"], case["low"], case["high"]
    step = (high / low) ** (1.0 / max(1, n - 1))
    return [max(1, int(low * step ** i) | 1) for i in range(n)]


def _prepare_linear(case, seed):
    M, N, K, dt = case["M"], case["N"], case["K"], DTYPES[case["dtype"]]
    g = _generator(seed)
    s = {"case": case, "x": _normal(g, (M, K), 1.0, dt),
         "w": _normal(g, (N, K), K ** -0.5, dt)}
    gated = case["act"] in GATED
    s["w3"] = _normal(g, (N, K), K ** -0.5, dt) if gated else None
    s["b"] = _normal(g, (N,), 0.1, dt) if case["bias"] else None
    s["b3"] = _normal(g, (N,), 0.1, dt) if case["bias"] and gated else None
    s["res"] = _normal(g, (M, N), 1.0, dt) if case["residual"] else None
    if case["op"] == "linear_grad":
        s["dy"] = _normal(g, (M, N), N ** -0.5, dt)
    if own:
        import sparse_mixture_experts_50_amd as moe
        s["moe"] = moe
        s["desc"] = moe.make_linear_desc(M, N, K, dt, activation=case["act"])
        s["weights"] = moe.LinearWeights(s["w"], b=s["b"], w3=s["w3"],
                                         b3=s["b3"])
        if case["op"] == "linear":
            need = moe.moe_linear_workspace_size(s["desc"])
            s["y"] = torch.empty(M, N, dtype=dt, device=DEV)
        else:
            need = moe.moe_linear_grad_workspace_size(s["desc"])
            s["grads"] = moe.LinearGrads(
                s["desc"], s["x"].device,
                [n for n in ("x", "w", "b", "w3", "b3")
                 if s[n] is not None])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


def _prepare_dense(case, seed):
    T, d, F, dt = case["T"], case["d"], case["d_ff"], DTYPES[case["dtype"]]
    g = _generator(seed)
    gated = case["act"] in GATED
    s = {"case": case, "x": _normal(g, (T, d), 1.0, dt),
         "w1": _normal(g, (F, d), d ** -0.5, dt),
         "w2": _normal(g, (d, F), F ** -0.5, dt),
         "w3": _normal(g, (F, d), d ** -0.5, dt) if gated else None}
    for name, n in (("b1", F), ("b2", d), ("b3", F)):
        s[name] = _normal(g, (n,), 0.1, dt) \
            if case["bias"] and (gated or name != "b3") else None
    s["res"] = _normal(g, (T, d), 1.0, dt) if case["residual"] else None
    s["dy"] = _normal(g, (T, d), d ** -0.5, dt) \
        if case["op"] == "dense_grad" else None
    if own:
        import sparse_mixture_experts_50_amd as moe
        s["layer"] = moe.DenseLayer(
            moe.DenseWeights(s["w1"], s["w2"], w3=s["w3"], b1=s["b1"],
                             b2=s["b2"], b3=s["b3"]),
            activation=case["act"])
    return s


def _prepare_adamw(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    gdt = DTYPES["f32"] if case["grad"] == "f32" else dt
    s = {"case": case, "lr": 1e-4, "betas": (0.9, 0.95), "eps": 1e-8,
         "decay": [0.1 if i % 4 else 0.0 for i in range(case["count"])],
         "steps": 100 + seed % 1000, "seed": seed & 0x7FFFFFFF}
    s["params"], s["grads"], s["m"], s["v"], s["master"] = [], [], [], [], []
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for n in _sizes(case):
        p = _normal(g, (n,), 0.02, torch.float32)
        s["params"].append(p.to(dt))
        if case["master"]:
            s["master"].append(p)
        # elements differ in the size of their gradients, as rows of an
        # embedding or channels of a norm do
        size = _normal(g, (n,), 2.0, torch.float32).exp_().mul_(1e-4)
        s["grads"].append(
            _normal(g, (n,), 1.0, torch.float32).mul_(size).to(gdt))
        m = _normal(g, (n,), 0.3, torch.float32).mul_(size)
        v = _normal(g, (n,), 0.3, torch.float32).exp_().mul_(size)
        if case["bits"] == 8:
            half = torch.full((1,), 0x80000, device=DEV)
            s["m"].append(_quantize(m, half))
            s["v"].append(_quantize(v, half, root=True))
        else:
            s["m"].append(m)
            s["v"].append(v.square_())
        total += s["grads"][-1].double().square().sum()
        del p, size, m, v
    # the gradients' norm, measured before the step, over the limit
    s["norm"] = total.sqrt().float().reshape(1)
    s["max_norm"] = 0.5 * math.exp(4.0) * 1e-4 * math.sqrt(sum(_sizes(case)))
    if own:
        import sparse_mixture_experts_50_amd as moe
        opt = s["opt"] = moe.AdamW(
            s["params"], lr=s["lr"], betas=s["betas"], eps=s["eps"],
            weight_decay=s["decay"], state_bits=case["bits"],
            master=case["master"], stochastic=case["stochastic"],
            seed=s["seed"])
        opt.steps = s["steps"]
        for i in range(case["count"]):
            if case["master"]:
                opt.master[i].copy_(s["master"][i])
            if case["bits"] == 8:
                opt.m[i].copy_(s["m"][i][0])
                opt.m_scale[i].copy_(s["m"][i][1])
                opt.v[i].copy_(s["v"][i][0])
                opt.v_scale[i].copy_(s["v"][i][1])
            else:
                opt.m[i].copy_(s["m"][i])
                opt.v[i].copy_(s["v"][i])
        del s["m"], s["v"], s["master"]
    return s


def prepare(case, seed):
    if case["op"] == "adamw":
        return _prepare_adamw(case, seed)
    if case["op"] in ("dense", "dense_grad"):
        return _prepare_dense(case, seed)
    return _prepare_linear(case, seed)


# ------------------------------------------------------------------- run

def run(s):
    if own:
        return _own(s)
    return {"linear": _plain_linear, "linear_grad": _plain_linear_grad,
            "dense": _plain_dense, "dense_grad": _plain_dense_grad,
            "adamw": _plain_adamw}[s["case"]["op"]](s)


def _own(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        s["moe"].moe_linear(s["desc"], s["x"], s["weights"], s["y"], s["ws"],
                            residual=s["res"])
        return s["y"]
    if op == "linear_grad":
        s["moe"].moe_linear_grad(s["desc"], s["x"], s["weights"], s["dy"],
                                 s["grads"], s["ws"])
        return s["grads"].as_dict()
    if op == "dense":
        return s["layer"].forward(s["x"], residual=s["res"])
    if op == "dense_grad":
        return s["layer"].backward(s["x"], s["dy"],
                                   residual=case["residual"]).as_dict()
    opt = s["opt"]
    opt.step(s["grads"], norm=s["norm"] if case["clip"] else None,
             max_norm=s["max_norm"])
    out = {"params": s["params"], "m": opt.m, "v": opt.v}
    if case["master"]:
        out["master"] = opt.master
    if case["bits"] == 8:
        out["m_scale"], out["v_scale"] = opt.m_scale, opt.v_scale
    return out


def _activation(act, z, u):
    """h and its derivatives by z and u."""
    if act == "none":
        return z, torch.ones_like(z), None
    if GATED.get(act, act) == "gelu":
        phi = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        a = z * phi
        da = phi + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    else:
        sig = torch.sigmoid(z)
        a, da = z * sig, sig * (1.0 + z * (1.0 - sig))
    return (a, da, None) if u is None else (a * u, da * u, a)


def _f32(t):
    return None if t is None else t.float()


def _project(x, w, b):
    z = x @ w.float().t()
    return z if b is None else z + b.float()


def _plain_linear(s):
    act, x = s["case"]["act"], s["x"].float()
    z = _project(x, s["w"], s["b"])
    u = _project(x, s["w3"], s["b3"]) if act in GATED else None
    y = _activation(act, z, u)[0]
    y = y if s["res"] is None else y + s["res"].float()
    return y.to(s["x"].dtype)


def _plain_linear_grad(s):
    act, x, dy = s["case"]["act"], s["x"].float(), s["dy"].float()
    gated, dt = act in GATED, s["x"].dtype
    dz, du = dy, None
    if act != "none":
        z = _project(x, s["w"], s["b"])
        u = _project(x, s["w3"], s["b3"]) if gated else None
        _, hz, hu = _activation(act, z, u)
        dz = dy * hz
        du = dy * hu if gated else None
    g = {"x": dz @ s["w"].float(), "w": dz.t() @ x}
    if s["b"] is not None:
        g["b"] = dz.sum(0)
    if gated:
        g["x"] = g["x"] + du @ s["w3"].float()
        g["w3"] = du.t() @ x
        if s["b3"] is not None:
            g["b3"] = du.sum(0)
    return {n: t.to(dt) for n, t in g.items()}


def _plain_dense(s):
    act, x = s["case"]["act"], s["x"].float()
    z = _project(x, s["w1"], s["b1"])
    u = _project(x, s["w3"], s["b3"]) if act in GATED else None
    y = _project(_activation(act, z, u)[0], s["w2"], s["b2"])
    y = y if s["res"] is None else y + s["res"].float()
    return y.to(s["x"].dtype)


def _plain_dense_grad(s):
    case, dt = s["case"], s["x"].dtype
    act, x, dy = case["act"], s["x"].float(), s["dy"].float()
    gated = act in GATED
    z = _project(x, s["w1"], s["b1"])
    u = _project(x, s["w3"], s["b3"]) if gated else None
    h, hz, hu = _activation(act, z, u)
    q = dy @ s["w2"].float()
    dz = q * hz
    g = {"x": dz @ s["w1"].float(), "w1": dz.t() @ x, "w2": dy.t() @ h}
    if case["bias"]:
        g["b1"], g["b2"] = dz.sum(0), dy.sum(0)
    if gated:
        du = q * hu
        g["x"] = g["x"] + du @ s["w3"].float()
        g["w3"] = du.t() @ x
        if case["bias"]:
            g["b3"] = du.sum(0)
    if case["residual"]:
        g["x"] = g["x"] + dy
    return {n: t.to(dt) for n, t in g.items()}


# An 8-bit state: e4m3 codes in blocks of 32 that share a power of two, the
# least one under which the block's largest value is at most 448, held as its
# exponent + 127.  A second moment is held as its root.  Codes are rounded at
# random, up where the 20 bits that are lost, of a value scaled to have 2^20
# of them per step, carry together with 20 given ones; a root that is not 0
# does not become 0.

def _bits20(bits16):
    return bits16 << 4


def _hash32(x):
    """A mixed 32-bit value of each 32-bit value (held in int64)."""
    m = 0xFFFFFFFF
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & m
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & m
    return x ^ (x >> 16)


def _random_bits(s, i, step, n):
    """32 bits for each element of tensor i, in one step."""
    key = (s["seed"] * 0x9E3779B1 + step * 0x85EBCA77 + i * 0xC2B2AE3D) \
        & 0xFFFFFFFF
    return _hash32((torch.arange(n, device=DEV) & 0xFFFFFFFF) ^ key)


def _blocks(x):
    n = x.numel()
    more = -n % BLOCK
    if more:
        x = torch.cat([x, x.new_zeros(more)])
    return x.view(-1, BLOCK)


def _quantize(x, rnd, root=False):
    """(codes, exponents) of float32 values, ``rnd`` 20 bits for each."""
    n = x.numel()
    top = _blocks(x).abs().amax(1)
    bits = top.view(torch.int32)
    e = torch.where(top == 0, 127, ((bits + 0x1FFFFF) >> 23) - 8)
    e = e.clamp(min=1)                        # exponent + 127
    # e4m3's smallest normal number lies at float32's
    scaled = (_blocks(x).abs().double() *
              torch.exp2(-120.0 - (e - 127).double())[:, None]) \
        .float().view(torch.int32).view(-1)[:n]
    code = (scaled.long() + rnd) >> 20
    code = code.clamp(max=0x7E)
    if root:
        code = torch.where((code == 0) & (x > 0), 1, code)
    else:
        code = torch.where(x < 0, code + 128, code)
    return code.to(torch.uint8).view(torch.float8_e4m3fn), e.to(torch.uint8)


def _dequantize(state):
    codes, e = state
    n = codes.numel()
    scale = torch.exp2((e.int() - 127).float())
    return (_blocks(codes.float()) * scale[:, None]).view(-1)[:n]


def _round_bf16(p, bits16):
    """float32 rounded to bf16, up where the lost bits carry with given
    ones."""
    raw = p.view(torch.int32).long() + bits16
    return (raw & -65536).to(torch.int32).view(torch.float32) \
        .to(torch.bfloat16)


def _plain_adamw(s):
    case, (b1, b2) = s["case"], s["betas"]
    s["steps"] += 1
    t = s["steps"]
    size = s["lr"] / (1.0 - b1 ** t)
    unbias = 1.0 / math.sqrt(1.0 - b2 ** t)
    factor = None
    if case["clip"]:
        factor = (s["max_norm"] / (s["norm"].double() + EPS)) \
            .clamp(max=1.0).float()
    for i, (p, g) in enumerate(zip(s["params"], s["grads"])):
        g = g.float()
        g = g if factor is None else g * factor
        bits8 = case["bits"] == 8
        m = _dequantize(s["m"][i]) if bits8 else s["m"][i]
        v = _dequantize(s["v"][i]).square() if bits8 else s["v"][i]
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + g * g * (1.0 - b2)
        root = v.sqrt()
        x = s["master"][i] if case["master"] else p.float()
        x = x - (x * (s["lr"] * s["decay"][i]) +
                 size * m / (root * unbias + s["eps"]))
        rnd = _random_bits(s, i, t, x.numel()) \
            if bits8 or case["stochastic"] else None
        if case["master"]:
            s["master"][i].copy_(x)
            p.copy_(x)
        elif case["stochastic"] and p.dtype == torch.bfloat16:
            p.copy_(_round_bf16(x, _hash32(rnd ^ 0x5BD1E995) >> 16))
        else:
            p.copy_(x)
        if bits8:
            s["m"][i] = _quantize(m, _bits20(rnd & 0xFFFF))
            s["v"][i] = _quantize(root, _bits20(rnd >> 16), root=True)
        else:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
    out = {"params": s["params"]}
    if case["master"]:
        out["master"] = s["master"]
    if case["bits"] == 8:
        out["m"], out["m_scale"] = zip(*s["m"])
        out["v"], out["v_scale"] = zip(*s["v"])
    else:
        out["m"], out["v"] = s["m"], s["v"]
    return out


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        p = 2 if case["dtype"] == "bf16" else 4
        grad = 4 if case["grad"] == "f32" else p
        each = grad + (8 + p if case["master"] else 2 * p)
        each += 16 if case["bits"] == 32 else 4 + 4 / BLOCK
        return {"bytes": n * each, "flops": 14 * n}
    es = 4 if case["dtype"] == "f32" else 2
    gated = case["act"] in GATED
    if case["op"] in ("linear", "linear_grad"):
        M, N, K = case["M"], case["N"], case["K"]
        mats = 2 if gated else 1
        if case["op"] == "linear":
            rows = M * (K + N * (2 if case["residual"] else 1))
            return {"bytes": es * (rows + mats * N * K),
                    "flops": 2 * M * N * K * mats}
        again = 0 if case["act"] == "none" else mats
        return {"bytes": es * (M * (2 * K + N) + 2 * mats * N * K),
                "flops": 2 * M * N * K * (2 * mats + again)}
    T, d, F = case["T"], case["d"], case["d_ff"]
    mats = 3 if gated else 2
    if case["op"] == "dense":
        return {"bytes": es * (T * d * (3 if case["residual"] else 2) +
                               mats * d * F), "flops": 2 * T * d * F * mats}
    return {"bytes": es * (3 * T * d + 2 * mats * d * F),
            "flops": 2 * T * d * F * (3 * mats - 1)}


# ----------------------------------------------------------------- exact

def _f64(t):
    return None if t is None else t.double()


def _exact_unit(act, x, w, b, w3, b3):
    """h and its derivatives by the two projections, in 64 bits."""
    z = x.matmul(w.t())
    if b is not None:
        z += b
    if act == "none":
        return z, 1.0, None
    if act in ("gelu", "geglu"):
        cdf = torch.special.ndtr(z)
        a, da = z * cdf, cdf + z * (-z * z / 2).exp() / (2 * math.pi) ** 0.5
    else:
        e = 1 / (1 + (-z).exp())
        a, da = z * e, e + z * e * (1 - e)
    if act not in GATED:
        return a, da, None
    u = x.matmul(w3.t())
    if b3 is not None:
        u += b3
    return a * u, da * u, a


def _exact_linear(s):
    act = s["case"]["act"]
    x, w, b, w3, b3 = (_f64(s[n]) for n in ("x", "w", "b", "w3", "b3"))
    h, hz, hu = _exact_unit(act, x, w, b, w3, b3)
    if s["case"]["op"] == "linear":
        return h if s["res"] is None else h + _f64(s["res"])
    dy = _f64(s["dy"])
    dz = dy * hz
    out = {"x": dz.matmul(w), "w": dz.t().matmul(x)}
    if b is not None:
        out["b"] = dz.sum(0)
    if act in GATED:
        du = dy * hu
        out["x"] += du.matmul(w3)
        out["w3"] = du.t().matmul(x)
        if b3 is not None:
            out["b3"] = du.sum(0)
    return out


def _exact_dense(s):
    case = s["case"]
    x, w1, w2, w3, b1, b2, b3 = (
        _f64(s[n]) for n in ("x", "w1", "w2", "w3", "b1", "b2", "b3"))
    h, hz, hu = _exact_unit(case["act"], x, w1, b1, w3, b3)
    if case["op"] == "dense":
        y = h.matmul(w2.t())
        y = y if b2 is None else y + b2
        return y if s["res"] is None else y + _f64(s["res"])
    dy = _f64(s["dy"])
    dh = dy.matmul(w2)
    out = {"w2": dy.t().matmul(h)}
    del h
    dz = dh * hz
    out["x"] = dz.matmul(w1)
    out["w1"] = dz.t().matmul(x)
    if w3 is not None:
        du = dh * hu
        out["x"] += du.matmul(w3)
        out["w3"] = du.t().matmul(x)
    if case["residual"]:
        out["x"] += dy
    if b1 is not None:
        out["b1"], out["b2"] = dz.sum(0), dy.sum(0)
        if w3 is not None:
            out["b3"] = du.sum(0)
    return out


def _exact_codes(x, rnd, root):
    """The code of each value, by its definition on the numbers' line."""
    n = x.numel()
    top = _blocks(x.abs()).amax(1)
    # least k with top <= 448 * 2^k
    k = torch.log2(top / 448.0).ceil()
    k = torch.where(top > 448.0 * torch.exp2(k), k + 1, k)
    k = torch.where(top <= 448.0 * torch.exp2(k - 1), k - 1, k)
    k = torch.where(top == 0, 0.0, k).clamp(min=-126)
    y = (_blocks(x.abs()) / torch.exp2(k)[:, None]).view(-1)[:n]
    step = torch.exp2(torch.log2(y.clamp(min=2.0 ** -6)).floor() - 3)
    step = torch.where(y >= 16 * step, 2 * step, step)
    step = torch.where((y < 8 * step) & (step > 2.0 ** -9), step / 2, step)
    q = (y / step + rnd.double() / 2 ** 20).floor() * step
    if root:
        q = torch.where((q == 0) & (x > 0), 2.0 ** -9, q)
    return torch.where(x < 0, -q, q).clamp(-448, 448)


def _exact_adamw(s):
    case, (b1, b2), t = s["case"], s["betas"], s["steps"] + 1
    out = {"params": [], "m": [], "v": []}
    if case["master"]:
        out["master"] = []
    f = min(1.0, s["max_norm"] / (float(s["norm"]) + EPS)) \
        if case["clip"] else 1.0
    for i, n in enumerate(_sizes(case)):
        g = s["grads"][i].double() * f
        m, v = s["m"][i], s["v"][i]
        if case["bits"] == 8:
            unit = [torch.exp2(e.double() - 127).repeat_interleave(BLOCK)[:n]
                    for _, e in (m, v)]
            m, v = m[0].double() * unit[0], (v[0].double() * unit[1]) ** 2
        m = b1 * m.double() + (1 - b1) * g
        v = b2 * v.double() + (1 - b2) * g * g
        x = (s["master"][i] if case["master"] else s["params"][i]).double()
        x = x - s["lr"] * (s["decay"][i] * x + (m / (1 - b1 ** t)) /
                           ((v / (1 - b2 ** t)).sqrt() + s["eps"]))
        out["params"].append(x)
        if case["master"]:
            out["master"].append(x)
        if case["bits"] == 8:
            r = _random_bits(s, i, t, n)
            m = _exact_codes(m, (r & 0xFFFF) << 4, False)
            v = _exact_codes(v.sqrt(), (r >> 16) << 4, True)
        out["m"].append(m)
        out["v"].append(v)
        del g, x, m, v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    if case["op"] in ("dense", "dense_grad"):
        return _exact_dense(s)
    return _exact_linear(s)
