"""The bounded float64 gradients that the kernels' elements are held to:
their values against autograd of the layer's definition, and mistakes that
their bounds have to show (planted here, in the reference)."""
import pytest
import torch

import grad_bounds as bounds
import grad_reference as ref

F64 = torch.float64


def layer_case(T, d, E, k, F, act, shared, biases, choice, cap, seed=0):
    g = torch.Generator().manual_seed(seed)

    def n(*s, v=1.0):
        return torch.randn(*s, generator=g, dtype=F64) * v

    w = {"w_router": n(E, d, v=2 * d ** -0.5), "b_router": n(E, v=0.5),
         "expert_bias": n(E, v=0.2), "w1": n(E, F, d, v=d ** -0.5),
         "w2": n(E, d, F, v=F ** -0.5)}
    if act == "swiglu":
        w["w3"] = n(E, F, d, v=d ** -0.5)
    if biases:
        w.update(b1=n(E, F, v=0.3), b2=n(E, d, v=0.3))
        if act == "swiglu":
            w["b3"] = n(E, F, v=0.3)
    if shared:
        w.update(ws1=n(F, d, v=d ** -0.5), ws2=n(d, F, v=F ** -0.5))
        if act == "swiglu":
            w["ws3"] = n(F, d, v=d ** -0.5)
        if biases:
            w.update(bs1=n(F, v=0.3), bs2=n(d, v=0.3))
            if act == "swiglu":
                w["bs3"] = n(F, v=0.3)
    x, dy = n(T, d), n(T, d)
    logits = x @ w["w_router"].t() + w["b_router"] - w["expert_bias"]
    return w, x, dy, ref.route(logits, k, cap, choice)


@pytest.mark.parametrize("act,choice,shared,biases,cap", [
    ("gelu", False, 0, True, -1), ("silu", False, 1, False, 3),
    ("swiglu", False, 1, True, 4), ("swiglu", True, 0, True, 5)])
def test_values_are_the_definition_s(act, choice, shared, biases, cap):
    T, E, alpha, aux, z = 13, 4, 0.3, 0.7, 0.4
    w, x, dy, r = layer_case(T, 8, E, 2, 12, act, shared, biases, choice, cap)
    got = bounds.layer(w, x, dy, r, act, choice, shared, alpha, aux, z, "f32")
    leaves = {"x": x, **{n: v for n, v in w.items() if n != "expert_bias"}}
    for v in leaves.values():
        v.requires_grad_()
    total = ref.loss(w, x, dy, r, act, choice, shared, alpha, aux, z)
    want = torch.autograd.grad(total, list(leaves.values()))
    assert sorted(got) == sorted(leaves)
    for (n, _), t in zip(leaves.items(), want):
        v, e = got[n]
        # both in float64, sums of tens of terms of order 1
        assert float((v - t).abs().max()) < 1e-11, n
        assert bool((e >= 0).all()), n


def off(a, b):
    """Largest difference of two values in bounds of the first."""
    return float(((a[0] - b[0]).abs() / (a[1] + 1e-300)).max())


def close(a, half):
    return a[0], a[1] + half * a[0].abs()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,k,choice,cap", [
    (1000, 256, 65, 2, False, -1), (321, 448, 192, 3, False, -1),
    (70, 128, 256, 64, False, -1), (130, 192, 200, 200, True, 2)])
def test_lost_losses_show(dtype, T, d, E, k, choice, cap):
    """The losses' gradient alone: its loss, another factor, other experts'
    f and another token count lie far outside the bounds of x, of the
    router's weights and of its bias."""
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, d, generator=g, dtype=F64)
    wr = torch.randn(E, d, generator=g, dtype=F64) * 2 * d ** -0.5
    br = torch.randn(E, generator=g, dtype=F64)
    eb = torch.randn(E, generator=g, dtype=F64) * 0.2
    r = ref.route(x @ wr.t() + br - eb, k, cap, choice)
    dw = torch.zeros(r["topk_w"].shape, dtype=F64)

    def grads(aux, z, **other):
        dl, e = bounds.dlogits(x, wr, br, other.get("eb", eb),
                               {**r, **other}, dw, dw, choice, 0.5, aux, z)
        half = bounds.HALF[dtype]
        gx, gw, gb = bounds.router(x, wr, dl, e, dtype)
        return close(gx, half), close(gw, half), close(gb, bounds.U)

    f = r["f"].clone()
    if not choice:
        f[E // 2:] = f[E // 2:].roll(1)      # other experts' shares
    for (aux, z), wrong in (
            ((1.0, 0.0), [grads(0.0, 0.0), grads(1.1, 0.0)]),
            ((0.0, 1.0), [grads(0.0, 0.0), grads(0.0, 1.1),
                          grads(0.0, 1.0, eb=eb * 0)]),
            ((1.0, 0.0), [] if choice else [grads(1.0, 0.0, f=f)])):
        right = grads(aux, z)
        for bad in wrong:
            for name, a, b in zip(("x", "w_router", "b_router"), right, bad):
                if choice and aux and not z:
                    continue       # equal shares: the gradient is zero
                assert off(a, b) > 4, (aux, z, name, off(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lost_rows_show(dtype):
    """A row, a column block of the hidden values, a routing weight or a
    bias left out moves an element past its bound."""
    act = "swiglu"
    w, x, dy, r = layer_case(150, 64, 3, 2, 128, act, 1, True, False, -1)

    def run(w, x=x, dy=dy, r=r):
        return bounds.layer(w, x, dy, r, act, False, 1, 0.01, 1.0, 0.1, dtype)

    right = run(w)
    lost = r["topk_w"].clone()
    lost[:, 1] = lost[:, 1] * 1.02
    cases = {
        "w1": run({**w, "b1": w["b1"] * 0}), "b1": run(w, dy=dy * 1.02),
        "w2": run({**w, "b3": w["b3"] * 0}), "x": run(w, r={**r,
                                                           "topk_w": lost}),
        "ws2": run({**w, "bs1": w["bs1"] * 0}),
        "w_router": run({**w, "b2": w["b2"] * 0}),
        "b_router": run({**w, "b2": w["b2"] * 0}),
    }
    for name, bad in cases.items():
        # (1.01: what the comparison allows)
        assert off(right[name], bad[name]) > 1.01, name
