"""Every element of the gradients within its own bound (grad_bounds.py): the
layer's at shapes where the persistent kernels run several rounds of tiles
and where few rows split the depth, the router's at every number of tokens,
and the losses' alone, measured against nothing but themselves."""
import pytest
import torch

import grad_bounds as bounds
import sparse_mixture_experts_50_amd as moe
from parity import device
from test_train_gpu import DT, FILL, layer_weights, make, normal

pytestmark = pytest.mark.gpu


def within(got, want, what):
    """Terms of second order (products of two relative errors, each below
    2^-8 but for sums that cancel) are the hundredth."""
    value, bound = want
    got = got.double().cpu()
    assert got.shape == value.shape, what
    off = (got - value).abs()
    bad = ~(off <= 1.01 * bound + 1e-30)
    assert not bad.any(), \
        f"{what}: {int(bad.sum())} of {bad.numel()} elements off, " \
        f"{float((off / (bound + 1e-30)).max()):.3g} of the bound"


def weights_of(r, rd, x, wr, br, eb, choice):
    """The routing weights that a forward with this expert bias leaves (the
    selection may be any)."""
    logits = x.double() @ wr.double().t() + br.double() - eb.double()
    rd.topk_w.copy_(torch.softmax(logits if choice else torch.gather(
        logits, 1, r["topk_idx"]), 1))
    r["topk_w"] = rd.topk_w.double().cpu()


def backward(dtype, T, d, E, k, F, act, shared, biases, cap=-1, choice=False,
             ebias=False, aux=0.0, z=0.0, alpha=0.01, zero_dy=False):
    desc, r, rd, g, x, wr, br = make(dtype, T, d, E, k, F=F, cap=cap,
                                     shared=shared, choice=choice, act=act,
                                     skew=0.3, alpha=alpha)
    dev, dt = device(), DT[dtype]
    w = layer_weights(g, dtype, d, E, F, act, shared, biases)
    eb = None
    if ebias:
        eb = normal(g, (E,), 0.2, torch.float32)
        weights_of(r, rd, x, wr, br, eb, choice)
    dy = torch.zeros(T, d, dtype=dt) if zero_dy else normal(g, (T, d), 1.0, dt)
    weights = moe.Weights(wr.to(dev), w["w1"].to(dev), w["w2"].to(dev),
                          b_router=br.to(dev),
                          expert_bias=None if eb is None else eb.to(dev),
                          **{n: v.to(dev) for n, v in w.items()
                             if n not in ("w1", "w2")})
    gr = moe.Grads(desc, dev, ("x", "w_router", "b_router", *w))
    for t in gr.as_dict().values():
        t.fill_(FILL)
    ws = torch.empty(moe.moe_grad_workspace_size(desc), dtype=torch.uint8,
                     device=dev).fill_(255)
    moe.moe_backward(desc, x.to(dev), weights, rd, dy.to(dev), gr, ws,
                     aux_scale=aux, z_scale=z)
    w64 = {n: v.double() for n, v in w.items()}
    w64.update(w_router=wr.double(), b_router=br.double(),
               expert_bias=None if eb is None else eb.double())
    want = bounds.layer(w64, x.double(), dy.double(), r, act, choice, shared,
                        alpha, aux, z, dtype)
    assert sorted(want) == sorted(gr.as_dict())
    for name, t in gr.as_dict().items():
        within(t, want[name], name)


# Large tiles: more of them than the 256 blocks of a launch, in every product.
@pytest.mark.parametrize("T,d,E,k,F,act,shared,biases,cap,choice", [
    # 600 tiles of q and z, 400 of dx, 2400 of the weights
    (5000, 512, 200, 2, 768, "gelu", 0, False, -1, False),
    # tiles that end with their axes, an odd number of stages, three matrices
    (4000, 320, 150, 2, 384, "swiglu", 1, True, -1, False),
    (3600, 448, 140, 2, 320, "silu", 0, True, 70, False),
    # groups of many row tiles, every height of them
    (9000, 512, 3, 2, 1024, "gelu", 1, False, -1, False),
    (1200, 320, 130, 1, 512, "swiglu", 0, False, 100, True),
])
def test_rounds_of_large_tiles(T, d, E, k, F, act, shared, biases, cap,
                               choice):
    backward("bf16", T, d, E, k, F, act, shared, biases, cap, choice,
             ebias=True, aux=1.0, z=0.1)


# Small tiles: more than the 512 blocks of a launch.
@pytest.mark.parametrize("T,d,E,k,F,act,shared,biases", [
    (500, 384, 250, 8, 512, "silu", 0, True),
    (700, 384, 256, 6, 640, "swiglu", 1, False),
])
def test_rounds_of_small_tiles(T, d, E, k, F, act, shared, biases):
    backward("bf16", T, d, E, k, F, act, shared, biases, ebias=True, aux=1.0,
             z=0.1)


# Few rows: the depth of q and of dx in ranges, of uneven lengths, which for
# a gated dx start in, or reach over to, the second product.
@pytest.mark.parametrize("shared,biases", [(0, False), (1, True)])
@pytest.mark.parametrize("T,d,E,k,F,act", [
    (9, 256, 8, 2, 640, "swiglu"),        # dx: 2 ranges
    (33, 256, 16, 4, 1408, "swiglu"),     # 5
    (5, 256, 4, 1, 2816, "swiglu"),       # 8
    (7, 2048, 4, 2, 640, "swiglu"),       # q: 4
    (12, 1728, 3, 1, 1088, "gelu"),       # q: 3, dx: 2
])
def test_depth_in_ranges(T, d, E, k, F, act, shared, biases):
    backward("bf16", T, d, E, k, F, act, shared, biases, aux=1.0, z=0.1)


@pytest.mark.parametrize("T,d,E,k,F,act,shared,biases,cap,choice", [
    (700, 256, 20, 3, 192, "swiglu", 1, True, 90, False),
    (300, 192, 7, 1, 320, "gelu", 0, True, 60, True),
])
def test_f32_elements(T, d, E, k, F, act, shared, biases, cap, choice):
    backward("f32", T, d, E, k, F, act, shared, biases, cap, choice,
             ebias=True, aux=1.0, z=0.1)


# With dy = 0 nothing is left but the losses' gradient.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("aux,z", [(1.0, 0.0), (0.0, 1.0), (1.0, 1.0)])
@pytest.mark.parametrize("T,d,E,k,F,act,shared,cap,choice", [
    (300, 320, 3, 1, 128, "gelu", 0, -1, False),
    (1100, 384, 5, 2, 256, "swiglu", 1, -1, False),
    (2070, 320, 2, 1, 448, "silu", 1, -1, False),
    (517, 512, 65, 2, 128, "gelu", 0, 9, False),
    (900, 192, 192, 4, 64, "silu", 0, -1, False),
    (260, 128, 256, 1, 64, "gelu", 0, 2, True),
])
def test_backward_losses_alone(dtype, aux, z, T, d, E, k, F, act, shared, cap,
                               choice):
    backward(dtype, T, d, E, k, F, act, shared, False, cap, choice,
             ebias=True, aux=aux, z=z, alpha=0.5, zero_dy=True)


def router(dtype, T, d, E, k, choice, cap, aux, z, alpha, dw_size):
    desc, r, rd, g, x, wr, br = make(dtype, T, d, E, k, cap=cap,
                                     choice=choice, skew=1.0, alpha=alpha)
    dev = device()
    eb = normal(g, (E,), 0.2, torch.float32)
    weights_of(r, rd, x, wr, br, eb, choice)
    dw = normal(g, r["topk_w"].shape, dw_size, torch.float32)
    dw[r["slot_of"] < 0] = 0.0
    w = moe.RouterWeights(wr.to(dev), br.to(dev), eb.to(dev))
    gr = moe.Grads(desc, dev, ("x", "w_router", "b_router"))
    ws = torch.empty(moe.moe_router_grad_workspace_size(desc),
                     dtype=torch.uint8, device=dev).fill_(255)
    moe.moe_router_grad(desc, x.to(dev), w, rd, dw.to(dev), gr, ws,
                        aux_scale=aux, z_scale=z)
    dl, e_dl = bounds.dlogits(x.double(), wr.double(), br.double(),
                              eb.double(), r, dw.double(),
                              torch.zeros_like(dw, dtype=torch.float64),
                              choice, alpha, aux, z)
    want = bounds.router(x.double(), wr.double(), dl, e_dl, dtype)
    for got, (v, e), half, what in zip(
            (gr.x, gr.w_router, gr.b_router), want,
            (bounds.HALF[dtype], bounds.HALF[dtype], bounds.U),
            ("x", "w_router", "b_router")):
        within(got, (v, e + half * v.abs()), what)


# The logits' gradient loses no bits to the layer's type, whatever T is.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,choice,cap", [
    (1, 64, 2, 2, False, -1), (1023, 256, 64, 8, False, -1),
    (1024, 256, 64, 8, False, -1), (1025, 320, 192, 3, False, 20),
    (1500, 576, 100, 4, False, -1), (2050, 192, 65, 2, False, -1),
    (4090, 4096, 64, 4, False, -1), (8100, 2112, 192, 3, False, -1),
    (4097, 4096, 128, 2, False, -1), (8192, 2048, 256, 8, False, -1),
    (1030, 256, 60, 60, True, 40),
    # wide rows: the large tiles with few tokens
    (513, 11008, 64, 2, False, -1), (300, 16448, 128, 2, False, -1),
    (500, 8192, 200, 3, False, -1), (1100, 8192, 100, 2, False, -1)])
def test_router_elements(dtype, T, d, E, k, choice, cap):
    router(dtype, T, d, E, k, choice, cap, 1.0, 0.25, 0.01, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("aux,z", [(1.0, 0.0), (0.0, 1.0)])
@pytest.mark.parametrize("T,d,E,k,choice,cap", [
    (1000, 256, 65, 2, False, -1), (321, 448, 192, 3, False, -1),
    (1300, 128, 192, 2, False, 9), (70, 128, 256, 64, False, -1),
    (2048, 320, 256, 8, False, -1), (130, 192, 200, 200, True, 2)])
def test_router_losses_alone(dtype, aux, z, T, d, E, k, choice, cap):
    router(dtype, T, d, E, k, choice, cap, aux, z, 0.5, 0.0)
