"""Every element of the gradients within its own bound (grad_bounds.py): the
router's at every number of tokens, and the losses' alone, measured against
nothing but themselves."""
import pytest
import torch

import grad_bounds as bounds
import sparse_mixture_experts_50_amd as moe
from parity import device
from test_train_gpu import make, normal

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
    (1030, 256, 60, 60, True, 40)])
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
