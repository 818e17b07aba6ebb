"""Single-precision dense layers: the norm of every output's error (dense_rms),
on the GPU at the sizes where the kernels change; and, without one, that
operands or activations with fewer bits are seen."""
import pytest
import torch

import dense_bounds
import dense_rms as ref
import sparse_mixture_experts_50_amd as moe
import test_dense_gpu as sizes
from parity import device

F32 = torch.float32


def bf16(t):
    return t.to(torch.bfloat16).to(t.dtype)


def ten_bits(t):
    """Rounded to 10 bits behind the point, as reduced matrix cores do."""
    m, e = torch.frexp(t)
    return torch.ldexp((m * 2 ** 11).round() / 2 ** 11, e)


# -------------------------------------------------------------- planted

def normal(g, shape, std=1.0):
    """float64 values that fp32 holds."""
    return (torch.randn(shape, generator=g) * std).float().double()


def fp32_linear(x, w):
    return x.float() @ w.float().t()


@pytest.mark.parametrize("lose", [bf16, ten_bits])
@pytest.mark.parametrize("M,N,K", [(64, 128, 8192), (64, 64, 16384),
                                   (69, 128, 3200), (8, 128, 64)])
def test_lost_bits_of_a_product(lose, M, N, K):
    g = torch.Generator().manual_seed(M + K)
    x, w = normal(g, (M, K)), normal(g, (N, K), K ** -0.5)
    want = ref.linear("none", x, w, None, None, None, None)
    ref.check(fp32_linear(x, w), want, "y")
    for a, b in ((lose(x), lose(w)), (x, lose(w))):
        with pytest.raises(AssertionError):
            ref.check(fp32_linear(a, b), want, "y")


@pytest.mark.parametrize("lose", [bf16, ten_bits])
@pytest.mark.parametrize("M,N,K", [(4100, 80, 64), (2000, 64, 64)])
def test_lost_bits_of_a_weight_gradient(lose, M, N, K):
    g = torch.Generator().manual_seed(M)
    x, w = normal(g, (M, K)), normal(g, (N, K), K ** -0.5)
    dy = normal(g, (M, N))
    want = ref.linear_grad("gelu", x, w, None, None, None, dy, None)
    z = x @ w.t()
    dz = dy * dense_bounds.act("gelu", z)[1]
    ref.check(dz.float().t() @ x.float(), want["w"], "w")
    ref.check(dz.float() @ w.float(), want["x"], "x")
    with pytest.raises(AssertionError):
        ref.check(lose(dz).float().t() @ lose(x).float(), want["w"], "w")
    with pytest.raises(AssertionError):
        ref.check(lose(dz).float() @ w.float(), want["x"], "x")
    with pytest.raises(AssertionError):
        ref.check(lose(dz).float().sum(0), want["b"], "b")


@pytest.mark.parametrize("lose", [bf16, ten_bits])
@pytest.mark.parametrize("T,d,F", [(257, 64, 2000), (300, 128, 1760)])
def test_lost_bits_between_products(lose, T, d, F):
    g = torch.Generator().manual_seed(T)
    t = [normal(g, (T, d)), normal(g, (F, d), d ** -0.5),
         normal(g, (d, F), F ** -0.5), normal(g, (F, d), d ** -0.5),
         None, None, None]
    want = ref.dense("swiglu", *t, None)
    h = dense_bounds.act("swiglu", t[0] @ t[1].t(), t[0] @ t[3].t())[0]
    ref.check(fp32_linear(h, t[2]), want, "y")
    with pytest.raises(AssertionError):
        ref.check(fp32_linear(lose(h), t[2]), want, "y")


# ------------------------------------------------------------ on the GPU

def single(cases):
    """The f32 ones of a list with or without types."""
    return [c[1:] if c[0] == "f32" else c for c in cases if c[0] != "bf16"]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,act", single(
    sizes.LINEAR + sizes.LARGE + sizes.FEW))
def test_linear(M, N, K, act):
    desc, t = sizes.linear_case("f32", M, N, K, act, True, True, seed=3)
    y = sizes.nan_like((M, N), F32)
    moe.moe_linear(desc, t["x"], sizes.weights(t), y,
                   sizes.workspace(moe.moe_linear_workspace_size(desc)),
                   residual=t["res"])
    ref.check(y, ref.linear(act, *(sizes.f64(t[n]) for n in (
        "x", "w", "b", "w3", "b3", "res"))), "y")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,act", single(
    sizes.LINEAR_GRAD + sizes.LARGE_GRAD + sizes.FEW))
def test_linear_grad(M, N, K, act):
    desc, t = sizes.linear_case("f32", M, N, K, act, True, True, seed=3)
    names = [n for n in ("x", "w", "b", "w3", "b3")
             if n in ("x", "w", "b") or t["w3"] is not None]
    g = moe.LinearGrads(desc, device(), names)
    moe.moe_linear_grad(desc, t["x"], sizes.weights(t), t["dy"], g,
                        sizes.workspace(
                            moe.moe_linear_grad_workspace_size(desc)),
                        dx_add=t["dx_add"])
    want = ref.linear_grad(act, *(sizes.f64(t[n]) for n in (
        "x", "w", "b", "w3", "b3", "dy", "dx_add")))
    for n in names:
        ref.check(getattr(g, n), want[n], n)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,F,act", sizes.DENSE + sizes.DENSE_LARGE)
def test_dense(T, d, F, act):
    t, layer = sizes.dense_case("f32", T, d, F, act, True, seed=3)
    args = [sizes.f64(t[n]) for n in sizes.OF_BLOCK]
    y = layer.forward(t["x"], residual=t["res"])
    ref.check(y, ref.dense(act, *args, sizes.f64(t["res"])), "y")
    g = layer.backward(t["x"], t["dy"], residual=True).as_dict()
    dy = sizes.f64(t["dy"])
    want = ref.dense_grad(act, *args, dy, dy)
    for n in g:
        ref.check(g[n], want[n], n)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,terms", [
    # 64 terms at a time, then the total
    (1024, 1024, 4096, 64 + 64), (300, 512, 16384, 64 + 256),
    # streamed: a quarter of the depth in one chain, then four waves
    (32, 16384, 4096, 1024 + 4), (16, 8192, 16384, 4096 + 4)])
def test_error_of_a_product(M, N, K, terms):
    """The error of the sums alone, as a share of the norm: n terms in a row
    have partial sums of half of the whole sum's square in the mean, so U^2 /
    3 n / 2; and one rounding more.  (The share's square is off by sqrt(2 / n)
    for n elements: far less than the tenth that is allowed.)"""
    desc, t = sizes.linear_case("f32", M, N, K, "none", False, False)
    y = sizes.nan_like((M, N), F32)
    moe.moe_linear(desc, t["x"], sizes.weights(t), y,
                   sizes.workspace(moe.moe_linear_workspace_size(desc)))
    err = ref.check(y, ref.linear("none", *(sizes.f64(t[n]) for n in (
        "x", "w", "b", "w3", "b3", "res"))), "y")
    print(f"{M} x {N} x {K}: {err:.2e} of the norm")
    assert err <= 1.1 * ref.U * (terms / 6 + 1) ** 0.5
