"""The training operators on the GPU against float64 references: rows into
expert order and back, the router's and the layer's gradient, clipping;
then all of them together as a training step runs them."""
import ctypes

import pytest
import torch

import grad_reference as ref
import sparse_mixture_experts_50_amd as moe
import workloads
from parity import device
from sparse_mixture_experts_50_amd import _lib

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# A rounding to the output's type is off by at most half a step.
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
FILL = 7.0


def close_elements(got, want, terms, n, dtype, what):
    """Each element within one rounding of the result and the fp32 rounding
    of a sum of n terms whose magnitudes add up to ``terms``."""
    got = got.double().cpu()
    tol = HALF[dtype] * want.abs() + 2.0 ** -24 * (n + 2) * terms + 1e-38
    bad = ((got - want).abs() > tol * 1.001).sum().item()
    assert bad == 0, f"{what}: {bad} of {want.numel()} elements off"


def close_norm(got, want, dtype, rounded, k, what):
    """2-norm of the error against that of the result.  bf16: one half step
    for the output and one for each rounded operand in a row behind it
    (independent roundings of a sum's terms do not add up to more than one
    of the sum's own size); f32: k roundings of 2^-24, k the number of
    operations that a value passes."""
    got, want = got.double().cpu(), want.double().cpu()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    tol = (1 + rounded) * HALF["bf16"] + k * 2.0 ** -24 if dtype == "bf16" \
        else k * 2.0 ** -24
    err, size = float((got - want).norm()), float(want.norm())
    assert err <= tol * size + 1e-30, \
        f"{what}: error {err / max(size, 1e-300):.3g}, allowed {tol:.3g}"


def normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def on_device(desc, r):
    """The reference routing in the package's buffers."""
    out = moe.Routing(desc.T, desc.E, desc.k, device(),
                      slots=r["slot_token"].numel())
    for name in ("topk_idx", "topk_w", "slot_of", "slot_token", "offsets",
                 "counts", "kept", "f"):
        getattr(out, name).copy_(r[name])
    # the weights as the kernels have them
    r["topk_w"] = out.topk_w.double().cpu()
    r["f"] = out.f.double().cpu()
    return out


def make(dtype, T, d, E, k, F=64, cap=-1, shared=0, choice=False,
         act="gelu", seed=0, skew=0.0, alpha=0.01):
    """(descriptor, reference routing, device routing, generator, x, wr, br)"""
    g = torch.Generator().manual_seed(seed + T + 31 * d + 7 * E)
    dt = DT[dtype]
    x = normal(g, (T, d), 1.0, dt)
    wr = normal(g, (E, d), 2.0 / d ** 0.5, dt)
    br = normal(g, (E,), 0.1 + skew, torch.float32)
    r = ref.route(x.double() @ wr.double().t() + br.double(), k, cap, choice)
    desc = moe.make_desc(T, d, E, E if choice else k, F, dt, n_shared=shared,
                         capacity=cap, aux_alpha=alpha,
                         routing="expert_choice" if choice else "topk",
                         activation=act)
    return desc, r, on_device(desc, r), g, x, wr, br


# ------------------------------------------------------------------- rows

ROWS = [
    # T, d, E, k, capacity, shared, choice
    (1, 64, 1, 1, -1, 0, False),
    (1, 4096, 8, 2, -1, 1, False),
    (7, 128, 5, 3, -1, 0, False),
    (33, 192, 8, 2, 3, 1, False),        # tokens that lose every expert
    (20, 320, 4, 4, 0, 0, False),        # nothing kept
    (20, 320, 4, 4, 0, 1, False),        # nothing but the shared expert
    (129, 1088, 64, 64, -1, 0, False),   # k = 64
    (11, 8256, 6, 2, -1, 0, False),      # wider than one block's reach
    (65, 64, 256, 8, -1, 1, False),      # more experts than tokens
    (40, 256, 256, 256, 5, 1, True),     # expert choice, 256 ballot lanes
    (9, 128, 70, 70, 1, 0, True),
    (9, 128, 3, 3, 0, 0, True),          # no rows at all
    (2100, 512, 16, 2, -1, 0, False),    # two vectors per lane
    (5000, 2048, 4, 1, 1500, 0, False),  # four vectors per lane
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,cap,shared,choice", ROWS)
def test_rows(dtype, T, d, E, k, cap, shared, choice):
    desc, r, rd, g, x, _, _ = make(dtype, T, d, E, k, cap=cap, shared=shared,
                                   choice=choice, skew=1.0)
    dev, dt = device(), DT[dtype]
    n = r["slot_token"].numel() + shared * T
    xd = x.to(dev)

    xs = torch.full((n, d), FILL, dtype=dt, device=dev)
    moe.moe_dispatch_rows(desc, rd, xd, xs)
    assert torch.equal(xs.double().cpu(),
                       ref.dispatch(r, x.double(), shared, FILL))

    # rows in no use hold what must not be read
    ys = normal(g, (n, d), 1.0, dt)
    used = torch.zeros(n, dtype=torch.bool)
    at = r["slot_of"][r["slot_of"] >= 0]
    used[at] = True
    used[n - shared * T:] = True
    ys[~used] = float("nan")
    yd = ys.to(dev)
    ys64 = torch.where(used[:, None], ys.double(), 0.0)
    terms = r["slot_of"].shape[1] + shared
    dx = torch.full((T, d), FILL, dtype=dt, device=dev)
    moe.moe_dispatch_rows_grad(desc, rd, yd, dx)
    close_elements(dx, ref.combine(r, ys64, T, shared, False),
                   ref.combine(r, ys64.abs(), T, shared, False), terms,
                   dtype, "dispatch_rows_grad")
    y = torch.full((T, d), FILL, dtype=dt, device=dev)
    moe.moe_combine_rows(desc, rd, yd, y)
    close_elements(y, ref.combine(r, ys64, T, shared),
                   ref.combine(r, ys64.abs(), T, shared), terms, dtype,
                   "combine_rows")

    dy = normal(g, (T, d), 1.0, dt)
    dw = torch.full(r["slot_of"].shape, FILL, device=dev)
    want, want_dw = ref.combine_grad(r, dy.double(), ys64, shared, FILL)
    _, size_dw = ref.combine_grad(r, dy.double().abs(), ys64.abs(), shared,
                                  FILL)
    dys = torch.full((n, d), FILL, dtype=dt, device=dev)
    moe.moe_combine_rows_grad(desc, rd, dy.to(dev), yd, dys, dw)
    close_elements(dys, want, want.abs(), 1, dtype, "combine_rows_grad rows")
    close_elements(dw, want_dw, size_dw, d, "f32", "combine_rows_grad dw")
    assert torch.equal(dw.cpu()[r["slot_of"] < 0],
                       torch.zeros(int((r["slot_of"] < 0).sum())))
    # in place: the same bits, rows in no use untouched
    dw2 = torch.empty_like(dw)
    moe.moe_combine_rows_grad(desc, rd, dy.to(dev), yd, yd, dw2)
    assert torch.equal(dw, dw2)
    assert torch.equal(yd.cpu()[used], dys.cpu()[used])
    assert torch.isnan(yd.cpu()[~used]).all()


def test_rows_match_the_layer():
    """dispatch, the caller's own experts and combine give moe_forward's
    output: the explicit rows are the layer's own order."""
    w = workloads.scaled(workloads.get("tiny_top2_f32"), T=100,
                         linear_biases=False)
    dev = device()
    inp = workloads.make_inputs(w, dev)
    layer = moe.MoeLayer(moe.Weights.from_dict(inp), w.k)
    y, r = layer.forward(inp["x"])
    desc = layer.desc(w.T)
    xs = torch.empty(w.T * w.k, w.d, device=dev)
    moe.moe_dispatch_rows(desc, r, inp["x"], xs)
    off = r.offsets.tolist()
    ys = torch.cat([
        torch.nn.functional.gelu(xs[a:b] @ inp["w1"][e].t())
        @ inp["w2"][e].t() for e, (a, b) in enumerate(zip(off, off[1:]))])
    out = torch.empty_like(y)
    moe.moe_combine_rows(desc, r, ys, out)
    # two fp32 evaluations of 64- and 256-term products
    assert float((out - y).norm()) <= 2 * 400 * 2.0 ** -24 * float(y.norm())


# ----------------------------------------------------------------- router

ROUTER = [
    # T, d, E, k, choice, capacity
    (1, 64, 2, 1, False, -1),
    (5, 64, 1, 1, False, -1),
    (33, 192, 17, 3, False, -1),
    (257, 320, 64, 8, False, 20),
    (70, 128, 256, 64, False, -1),
    (1000, 256, 65, 2, False, -1),
    (50, 128, 9, 9, True, 6),
    (130, 192, 200, 200, True, 2),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("aux,z", [(0.0, 0.0), (1.5, 0.0), (0.0, 0.25),
                                   (1.0, 0.5)])
@pytest.mark.parametrize("T,d,E,k,choice,cap", ROUTER)
def test_router_grad(dtype, aux, z, T, d, E, k, choice, cap):
    check_router_grad(dtype, aux, z, T, d, E, k, choice, cap, True)


# alone; the last ones large enough for the large tiles of its bf16 products:
# token and column tiles that end with their axes, 1 to 4 stages of experts
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k", [
    (256, 256, 128, 4), (255, 320, 192, 3), (321, 448, 192, 3),
    (700, 256, 256, 8), (513, 704, 128, 2), (300, 192, 256, 2),
    (1, 256, 128, 2), (600, 576, 100, 4), (1300, 64, 64, 2),
    (4090, 4096, 64, 4), (4090, 4096, 128, 2), (8100, 2112, 192, 3),
    (8192, 2048, 256, 8)])
def test_router_grad_alone(dtype, T, d, E, k):
    check_router_grad(dtype, 1.0, 0.25, T, d, E, k, False, -1, False)


def check_router_grad(dtype, aux, z, T, d, E, k, choice, cap, add):
    desc, r, rd, g, x, wr, br = make(dtype, T, d, E, k, cap=cap,
                                     choice=choice)
    dev, dt = device(), DT[dtype]
    ebias = normal(g, (E,), 0.2, torch.float32)
    # the routing weights of these logits, as a forward with them leaves
    logits = x.double() @ wr.double().t() + br.double() - ebias.double()
    r["topk_w"] = torch.softmax(logits if choice else torch.gather(
        logits, 1, r["topk_idx"]), 1)
    rd.topk_w.copy_(r["topk_w"])
    dw = normal(g, r["topk_w"].shape, 1.0, torch.float32)
    dw[r["slot_of"] < 0] = 0.0
    base = normal(g, (T, d), 0.1, dt)
    w = moe.RouterWeights(wr.to(dev), br.to(dev), ebias.to(dev))
    gr = moe.Grads(desc, dev, ("x", "w_router", "b_router"))
    if add:
        gr.x.copy_(base)
    else:
        base.zero_()
    ws = torch.empty(moe.moe_router_grad_workspace_size(desc),
                     dtype=torch.uint8, device=dev).fill_(255)
    moe.moe_router_grad(desc, x.to(dev), w, rd, dw.to(dev), gr, ws,
                        aux_scale=aux, z_scale=z,
                        dx_add=gr.x if add else None)

    p = {"w_router": wr.double().requires_grad_(),
         "b_router": br.double().requires_grad_(),
         "expert_bias": ebias.double()}
    xr = x.double().requires_grad_()
    total = ref.router_loss(p, xr, dw.double(), r, choice, 0.01, aux, z)
    gx, gw, gb = torch.autograd.grad(total, [xr, p["w_router"],
                                             p["b_router"]])
    # a logit's gradient is a difference of terms as large as |w dw|, p aux,
    # z p: their fp32 roundings (of d-term logits, k- and E-term sums) are
    # measured against those magnitudes, not against what is left of them
    mag = (r["topk_w"] * dw.double().abs()).norm() * 2 + \
        abs(aux) * 0.01 * E / T ** 0.5 + abs(z) * 2 / T ** 0.5 * \
        float(torch.logsumexp(logits, 1).abs().max())
    unit = 2.0 ** -24 * (d + E + 64) * float(mag)

    def check(got, want, scale, what):
        got = got.double().cpu()
        tol = unit * scale + (2 * HALF["bf16"] if dtype == "bf16" and
                              what != "b_router" else 0.0) * \
            float(want.norm())
        assert float((got - want).norm()) <= tol + 1e-30, what

    # the intermediate dl is kept to well under a bf16 half step
    check(gr.x, gx + base.double(), float(wr.double().norm()) + 1, "x")
    check(gr.w_router, gw, float(x.double().norm()), "w_router")
    check(gr.b_router, gb, T ** 0.5, "b_router")


# ---------------------------------------------------------------- backward

def layer_weights(g, dtype, d, E, F, act, shared, biases):
    dt = DT[dtype]
    w = {"w1": normal(g, (E, F, d), d ** -0.5, dt),
         "w2": normal(g, (E, d, F), F ** -0.5, dt)}
    if act == "swiglu":
        w["w3"] = normal(g, (E, F, d), d ** -0.5, dt)
    if shared:
        w["ws1"] = normal(g, (F, d), d ** -0.5, dt)
        w["ws2"] = normal(g, (d, F), F ** -0.5, dt)
        if act == "swiglu":
            w["ws3"] = normal(g, (F, d), d ** -0.5, dt)
    if biases:
        w["b1"], w["b2"] = normal(g, (E, F), 0.3, dt), \
            normal(g, (E, d), 0.3, dt)
        if act == "swiglu":
            w["b3"] = normal(g, (E, F), 0.3, dt)
        if shared:
            w["bs1"], w["bs2"] = normal(g, (F,), 0.3, dt), \
                normal(g, (d,), 0.3, dt)
            if act == "swiglu":
                w["bs3"] = normal(g, (F,), 0.3, dt)
    return w


def reference_grads(w, wr, br, x, dy, r, act, choice, shared, aux, z):
    leaves = {"x": x.double(), "w_router": wr.double(),
              "b_router": br.double(), **{n: v.double() for n, v in w.items()}}
    for v in leaves.values():
        v.requires_grad_()
    full = {n: leaves.get(n) for n in (
        "w_router", "b_router", "w1", "b1", "w2", "b2", "w3", "b3", "ws1",
        "bs1", "ws2", "bs2", "ws3", "bs3")}
    total = ref.loss(full, leaves["x"], dy.double(), r, act, choice, shared,
                     0.01, aux, z)
    got = torch.autograd.grad(total, list(leaves.values()),
                              allow_unused=True)
    return {n: torch.zeros_like(v) if t is None else t
            for (n, v), t in zip(leaves.items(), got)}


BACKWARD = [
    # T, d, E, k, F, act, shared, biases, capacity, choice
    (1, 64, 1, 1, 64, "gelu", 0, False, -1, False),
    (1, 128, 8, 2, 128, "swiglu", 1, True, -1, False),
    (3, 64, 16, 2, 192, "silu", 0, True, -1, False),     # empty experts
    (40, 192, 3, 2, 64, "gelu", 1, True, 9, False),      # dropped tokens
    (65, 256, 2, 1, 320, "silu", 0, False, 0, False),    # no rows
    (130, 128, 4, 2, 256, "swiglu", 0, False, -1, False),
    (300, 320, 3, 3, 128, "gelu", 0, True, -1, False),   # ragged tails
    (700, 256, 2, 1, 384, "swiglu", 1, False, -1, False),
    (517, 512, 2, 2, 512, "gelu", 1, False, -1, False),
    (90, 128, 6, 6, 128, "swiglu", 1, True, 17, True),
    (64, 64, 4, 4, 64, "gelu", 0, False, 64, True),
    (64, 64, 4, 4, 64, "silu", 1, False, 0, True),       # no routed rows
    (1100, 384, 1, 1, 640, "gelu", 0, True, -1, False),  # one long group
    # large tiles that end with their axes, by row and by column
    (2070, 320, 2, 1, 448, "silu", 1, True, -1, False),
    (620, 832, 3, 2, 384, "swiglu", 1, True, 300, False),
    (97, 448, 2, 2, 320, "gelu", 0, False, -1, False),
    # many rows of narrow layers, which have the small tiles
    (900, 192, 2, 1, 1088, "silu", 1, True, -1, False),
    (1000, 1024, 2, 2, 128, "swiglu", 0, False, -1, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,F,act,shared,biases,cap,choice", BACKWARD)
def test_backward(dtype, T, d, E, k, F, act, shared, biases, cap, choice):
    desc, r, rd, g, x, wr, br = make(dtype, T, d, E, k, F=F, cap=cap,
                                     shared=shared, choice=choice, act=act,
                                     skew=0.3)
    dev, dt = device(), DT[dtype]
    w = layer_weights(g, dtype, d, E, F, act, shared, biases)
    dy = normal(g, (T, d), 1.0, dt)
    aux, z = 0.5, 0.02
    weights = moe.Weights(wr.to(dev), w["w1"].to(dev), w["w2"].to(dev),
                          b_router=br.to(dev),
                          **{n: v.to(dev) for n, v in w.items()
                             if n not in ("w1", "w2")})
    gr = moe.Grads(desc, dev, ("x", "w_router", "b_router", *w))
    for t in gr.as_dict().values():
        t.fill_(FILL)
    ws = torch.empty(moe.moe_grad_workspace_size(desc), dtype=torch.uint8,
                     device=dev).fill_(255)           # NaN everywhere
    moe.moe_backward(desc, x.to(dev), weights, rd, dy.to(dev), gr, ws,
                     aux_scale=aux, z_scale=z)
    want = reference_grads(w, wr, br, x, dy, r, act, choice, shared, aux, z)
    # operations on the way: products of depth d and F twice over, the
    # group's rows, and the functions
    k32 = 2 * (d + F) + T + E + 64
    for name, t in gr.as_dict().items():
        if name in ("w_router", "b_router", "x"):
            continue
        stacked = name in ("w1", "b1", "w2", "b2", "w3", "b3")
        for e in range(E if stacked else 1):
            a, b = (t[e], want[name][e]) if stacked else (t, want[name])
            if stacked and int(r["kept"][e]) == 0:
                assert not a.any(), f"{name}[{e}]: not zero"
            else:
                close_norm(a, b, dtype, 1, k32, f"{name}[{e}]")
    close_norm(gr.x, want["x"], dtype, 1, k32, "x")
    # the router's gradients are differences of terms of the size of w dw,
    # which is what their roundings are measured against
    q = r["topk_w"].double() * float(dy.double().norm() / T ** 0.5) * 3
    scale = float(q.norm()) * k32 * 2.0 ** -24 + 1e-12
    for name, size in (("w_router", float(x.double().norm())),
                       ("b_router", T ** 0.5)):
        err = float((getattr(gr, name).double().cpu() - want[name]).norm())
        tol = scale * size
        if dtype == "bf16" and name == "w_router":
            tol += 2 * HALF["bf16"] * float(want[name].norm())
        assert err <= tol, (name, err, tol)


def small_layer(dtype="bf16", T=96, act="swiglu", shared=1, seed=1):
    w = workloads.scaled(
        workloads.get("deepseek_v3"), T=T, d=256, E=8, k=2, d_ff=256,
        dtype=dtype, n_shared=shared, activation=act, expert_bias="none",
        seed=seed)
    inp = workloads.make_inputs(w, device())
    return w, inp, moe.MoeLayer(moe.Weights.from_dict(inp), w.k)


def test_backward_of_wanted_gradients_only():
    """Any subset of the gradients is the whole set's, bit for bit."""
    w, inp, layer = small_layer()
    dev = device()
    dy = torch.randn(w.T, w.d, device=dev).bfloat16()
    _, r = layer.forward(inp["x"])
    full = {n: t.clone() for n, t in layer.backward(
        inp["x"], r, dy, z_scale=0.1).as_dict().items()}
    desc, _, ws = layer.grad_buffers(w.T)
    for names in (("x",), ("w_router",), ("w2",), ("ws1", "w3"), ("w1", "x"),
                  ()):
        g = moe.Grads(desc, dev, names)
        moe.moe_backward(desc, inp["x"], layer.w, r, dy, g, ws,
                         aux_scale=1.0, z_scale=0.1)
        assert sorted(g.as_dict()) == sorted(names)
        for n in names:
            assert torch.equal(getattr(g, n), full[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(dtype):
    dev, dt = device(), DT[dtype]
    desc = moe.make_desc(0, 64, 3, 2, 64, dt, n_shared=1)
    names = ("w_router", "b_router", "w1", "b1", "w2", "b2", "ws1", "bs1",
             "ws2", "bs2")
    g = moe.Grads(desc, dev, names)
    for t in g.as_dict().values():
        t.fill_(FILL)
    z = lambda *s: torch.zeros(s, dtype=dt, device=dev)
    w = moe.Weights(z(3, 64), z(3, 64, 64), z(3, 64, 64), ws1=z(64, 64),
                    ws2=z(64, 64))
    ws = torch.empty(moe.moe_grad_workspace_size(desc), dtype=torch.uint8,
                     device=dev)
    r = moe.Routing(0, 3, 2, dev)
    moe.moe_backward(desc, z(0, 64), w, r, z(0, 64), g, ws)
    for n, t in g.as_dict().items():
        assert not t.any(), n
    g.w_router.fill_(FILL)
    moe.moe_router_grad(desc, z(0, 64), w, r, torch.zeros(0, 2, device=dev),
                        g, ws)
    assert not g.w_router.any()
    xs = z(0, 64)
    moe.moe_dispatch_rows(desc, r, xs, xs)


# ---------------------------------------------------------------- clipping

def clip_ws(tensors):
    return torch.empty(max(1, moe.moe_clip_workspace_size(tensors)),
                       dtype=torch.uint8, device=device()).fill_(255)


@pytest.mark.parametrize("kind", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", [
    (1,), (0,), (0, 5, 0), (3, 1, 2), (16383, 16384, 16385, 8191, 8193),
    (100003, 7, 65536, 1), tuple(range(1, 98)), (200,) * 193 + (70001,),
])
@pytest.mark.parametrize("share", [0.3, 2.0])
def test_clip(kind, sizes, share):
    """Tensors of every size around the chunk, in one and several tables;
    back to back in one buffer (so at odd addresses) and apart."""
    dev = device()
    g = torch.Generator().manual_seed(len(sizes))
    types = [DT["f32" if kind == "f32" or (kind == "mixed" and i % 2)
                else "bf16"] for i in range(len(sizes))]
    src = [normal(g, (n,), 0.5 + (i % 3), t)
           for i, (n, t) in enumerate(zip(sizes, types))]
    norm, _ = ref.clip(src, 1.0)
    limit = share * norm
    norm, want = ref.clip(src, limit)
    out_norm = torch.full((1,), FILL, device=dev)
    tensors = [t.to(dev) for t in src]
    if kind != "mixed":
        # one element of room in front: nothing is 16-byte aligned
        flat = torch.empty(sum(sizes) + 1, dtype=types[0], device=dev)
        views = list(flat[1:].split(list(sizes)))
        for v, t in zip(views, tensors):
            v.copy_(t)
    else:
        views = tensors
    outs = [torch.full_like(t, FILL) for t in tensors]
    ws = clip_ws(tensors)
    moe.moe_clip_grads(views, limit, out_norm, ws, out=outs)

    def check(got):
        assert abs(float(out_norm) - norm) <= 2.0 ** -23 * norm
        for a, b, t in zip(got, want, types):
            half = HALF["bf16" if t == torch.bfloat16 else "f32"]
            # the factor's rounding to fp32, the product's, the type's
            tol = (half + 3 * 2.0 ** -24) * b.abs() + 1e-38
            assert bool(((a.double().cpu() - b).abs() <= tol).all())

    check(outs)
    moe.moe_clip_grads(views, limit, out_norm, ws)          # in place
    check(views)


def test_clip_not_finite_and_large():
    dev = device()
    a = torch.tensor([1.0, float("nan"), 2.0], device=dev)
    b = torch.ones(5, device=dev, dtype=torch.bfloat16)
    norm = torch.zeros(1, device=dev)
    ws = clip_ws([a, b])
    moe.moe_clip_grads([a, b], 1.0, norm, ws)
    assert torch.isnan(norm).all() and torch.isnan(a).all() and \
        torch.isnan(b.float()).all()
    a = torch.tensor([1.0, float("inf"), 2.0], device=dev)
    b = torch.ones(5, device=dev)
    moe.moe_clip_grads([a, b], 1.0, norm, ws)
    assert torch.isinf(norm).all() and not b.any()
    assert torch.isnan(a[1]) and float(a[0]) == 0.0
    # squares past fp32's range: norm 2e30, each element 0.5 after it
    a = torch.full((4,), 1e30, device=dev)
    moe.moe_clip_grads([a], 1.0, norm, ws)
    assert abs(float(norm) / 2e30 - 1) < 1e-6
    assert float((a - 0.5).abs().max()) < 1e-6
    # all zeros, nothing at all, a limit of zero
    a = torch.zeros(9, device=dev)
    moe.moe_clip_grads([a], 1.0, norm, ws)
    assert float(norm) == 0.0 and not a.any()
    norm.fill_(FILL)
    moe.moe_clip_grads([], 1.0, norm, clip_ws([]))
    assert float(norm) == 0.0
    a = torch.ones(9, device=dev)
    moe.moe_clip_grads([a], 0.0, norm, ws)
    assert float(norm) == 3.0 and not a.any()


def test_clip_norm_alone():
    """dst NULL: a tensor is counted and left."""
    dev = device()
    a, b = torch.full((4,), 2.0, device=dev), torch.full((9,), 1.0, device=dev)
    norm, ws = torch.zeros(1, device=dev), clip_ws([a, b])
    for dst in (None, b.data_ptr()):
        arr = (_lib.MoeTensor * 2)(
            _lib.MoeTensor(a.data_ptr(), None, 4, 0),
            _lib.MoeTensor(b.data_ptr(), dst, 9, 0))
        st = _lib.lib().moe_clip_grads(
            2, arr, 1.0, norm.data_ptr(), ws.data_ptr(), ws.numel(),
            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert float(norm) == 5.0
        assert float(a[0]) == 2.0
        assert abs(float(b[0]) - (1.0 if dst is None else 0.2)) < 1e-6


# ---------------------------------------------------------------- together

def step_reference(w, inp, r, dy, act, shared):
    rr = {n: getattr(r, n).cpu() for n in ("topk_idx", "slot_of",
                                           "slot_token", "offsets", "kept")}
    rr = {n: v.long() for n, v in rr.items()}
    rr["topk_w"], rr["f"] = r.topk_w.double().cpu(), r.f.double().cpu()
    names = [n for n in ("w1", "w2", "w3", "ws1", "ws2", "ws3")
             if inp.get(n) is not None]
    ww = {n: inp[n].cpu() for n in names}
    br = torch.zeros(w.E)
    return reference_grads(ww, inp["wr"].cpu(), br, inp["x"].cpu(), dy.cpu(),
                           rr, act, False, shared, 1.0, 0.1), names


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_step(dtype):
    """forward, backward, clipping and an update, twice, on the layer's own
    buffers; the second step sees the first one's weights."""
    w, inp, layer = small_layer(dtype)
    dev = device()
    k32 = 2 * (w.d + w.d_ff) + w.T + w.E + 64
    for step in range(2):
        dy = torch.randn(w.T, w.d, generator=torch.Generator(device=dev)
                         .manual_seed(step), device=dev).to(DT[dtype])
        _, r = layer.forward(inp["x"])
        g = layer.backward(inp["x"], r, dy, z_scale=0.1)
        want, names = step_reference(w, inp, r, dy, "swiglu", 1)
        for n in names:
            close_norm(getattr(g, n), want[n], dtype, 1, k32, n)
        close_norm(g.x, want["x"], dtype, 1, k32, "x")
        close_norm(g.w_router, want["w_router"], dtype, 1, 4 * k32,
                   "w_router")
        tensors = [getattr(g, n) for n in (*names, "w_router")]
        norm = torch.empty(1, device=dev)
        before = torch.stack([t.double().square().sum()
                              for t in tensors]).sum().sqrt()
        moe.moe_clip_grads(tensors, 1.0, norm, clip_ws(tensors))
        assert abs(float(norm) / float(before) - 1) < 1e-6
        after = torch.stack([t.double().square().sum()
                             for t in tensors]).sum().sqrt()
        assert abs(float(after) - 1.0) <= HALF[dtype] + 1e-6
        for n, key in [(n, n) for n in names] + [("w_router", "wr")]:
            inp[key].sub_(getattr(g, n), alpha=0.05)


def test_captured_step_and_streams():
    """A captured forward + backward + clipping replays on new inputs to the
    eager call's bits, with eager work in between; the eager calls run on a
    stream of their own with their own buffers."""
    w, inp, layer = small_layer()
    _, _, eager = small_layer()
    dev = device()
    x, dy = inp["x"].clone(), torch.zeros_like(inp["x"])
    norm, ws = torch.zeros(1, device=dev), None

    def step(lay, a, b):
        _, r = lay.forward(a)
        g = lay.backward(a, r, b, z_scale=0.1)
        t = list(g.as_dict().values())
        moe.moe_clip_grads(t, 0.5, norm, ws)
        return g

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = layer.grad_buffers(w.T)[1]
        ws = clip_ws(list(g.as_dict().values()))
        step(layer, x, dy)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = step(layer, x, dy)
    for i in range(4):
        gen = torch.Generator(device=dev).manual_seed(i)
        xi = torch.randn(x.shape, generator=gen, device=dev).bfloat16()
        di = torch.randn(x.shape, generator=gen, device=dev).bfloat16()
        x.copy_(xi)
        dy.copy_(di)
        for t in g.as_dict().values():
            t.fill_(FILL)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in g.as_dict().items()}
        got_norm = norm.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = step(eager, xi, di)
        torch.cuda.synchronize()
        assert torch.equal(got_norm, norm)
        for n, t in want.as_dict().items():
            assert torch.equal(got[n], t), n


def test_two_calls_at_once():
    """Two backward calls on two streams, each with its own buffers, give
    what they give alone."""
    dev = device()
    pairs = []
    for seed in (1, 2):
        w, inp, layer = small_layer(seed=seed, T=400)
        dy = torch.randn(w.T, w.d, device=dev).bfloat16()
        _, r = layer.forward(inp["x"])
        g = layer.backward(inp["x"], r, dy)
        alone = {n: t.clone() for n, t in g.as_dict().items()}
        pairs.append((layer, inp["x"], r, dy, alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for layer, x, r, dy, alone, s in pairs * 3:
        with torch.cuda.stream(s):
            layer.backward(x, r, dy)
    torch.cuda.synchronize()
    for layer, x, r, dy, alone, s in pairs:
        got = layer.grad_buffers(x.shape[0])[1].as_dict()
        for n, t in alone.items():
            assert torch.equal(got[n], t), n


def test_layer_refuses_fp8_backward():
    dev = device()
    w = workloads.scaled(workloads.get("mixtral_decode_fp8"), T=4, d=1024,
                         E=2, k=1, d_ff=1024)
    inp = workloads.make_inputs(w, dev)
    layer = moe.MoeLayer(moe.Weights.from_dict(inp), w.k)
    _, r = layer.forward(inp["x"])
    with pytest.raises(moe.MoeError) as e:
        layer.backward(inp["x"], r, inp["x"])
    assert e.value.status == _lib.MOE_ERR_UNSUPPORTED
