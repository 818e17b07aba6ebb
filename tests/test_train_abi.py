"""The training entry points on a host without a GPU: sizes, refusals and
the binding's own checks, all before any HIP call; and the float64
reference against differences."""
import ctypes

import pytest
import torch

import grad_reference as ref
import sparse_mixture_experts_50_amd as moe
from sparse_mixture_experts_50_amd import _lib

FAKE = 0x1000      # never dereferenced: every call below fails validation
ROWS = {"moe_dispatch_rows": 2, "moe_dispatch_rows_grad": 2,
        "moe_combine_rows": 2, "moe_combine_rows_grad": 4}


def desc(**kw):
    base = dict(T=64, d=128, E=8, k=2, d_ff=256, n_shared=0, dtype=1,
                capacity=-1, aux_alpha=0.01)
    base.update(kw)
    return _lib.MoeDesc(**base)


def weights(**kw):
    base = dict(w_router=FAKE, w1=FAKE, w2=FAKE)
    base.update(kw)
    return _lib.MoeWeights(**base)


def routing(**kw):
    base = {n: FAKE for n, _ in _lib.MoeRouting._fields_}
    base.update(kw)
    return _lib.MoeRouting(**base)


def grads(**kw):
    return _lib.MoeGrads(**(kw or dict(x=FAKE, w1=FAKE)))


def backward(d, w=None, r=None, g=None, x=FAKE, dy=FAKE, ws=FAKE,
             ws_bytes=1 << 50, aux=1.0):
    return _lib.lib().moe_backward(
        ctypes.byref(d), x, ctypes.byref(w or weights()),
        ctypes.byref(r or routing()), dy, aux, 0.0,
        ctypes.byref(g or grads()), ws, ws_bytes, None)


def router_grad(d, w=None, r=None, g=None, x=FAKE, dw=FAKE, ws=FAKE,
                ws_bytes=1 << 50, aux=1.0):
    return _lib.lib().moe_router_grad(
        ctypes.byref(d), x, ctypes.byref(w or weights()),
        ctypes.byref(r or routing()), dw, None, aux, 0.0,
        ctypes.byref(g or grads()), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), _lib.MOE_ERR_INVALID_ARG),
    (dict(k=9), _lib.MOE_ERR_INVALID_ARG),
    (dict(dtype=7), _lib.MOE_ERR_UNSUPPORTED),
    (dict(d=100), _lib.MOE_ERR_UNSUPPORTED),
    (dict(E=300), _lib.MOE_ERR_UNSUPPORTED),
    (dict(routing=1, k=8, capacity=65), _lib.MOE_ERR_INVALID_ARG),
    (dict(activation=2, d_ff=192), _lib.MOE_ERR_UNSUPPORTED),
])
def test_descriptor_refused(kw, status):
    L, d = _lib.lib(), desc(**kw)
    assert L.moe_grad_workspace_size(ctypes.byref(d)) == 0
    assert L.moe_router_grad_workspace_size(ctypes.byref(d)) == 0
    assert backward(d) == status
    assert router_grad(d) == status
    for name, n in ROWS.items():
        assert getattr(L, name)(ctypes.byref(d), ctypes.byref(routing()),
                                *([FAKE] * n), None) == status


def test_fp8_experts_have_no_gradient():
    L, d = _lib.lib(), desc(expert_fp8=1, d=1024, d_ff=1024)
    assert L.moe_grad_workspace_size(ctypes.byref(d)) == 0
    assert backward(d) == _lib.MOE_ERR_UNSUPPORTED
    # the router of such a layer has one
    assert L.moe_router_grad_workspace_size(ctypes.byref(d)) > 0
    with pytest.raises(moe.MoeError) as e:
        moe.moe_grad_workspace_size(d)
    assert e.value.status == _lib.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", sorted(ROWS))
def test_row_operators_refuse_null(name):
    fn, d, n = getattr(_lib.lib(), name), desc(), ROWS[name]
    for i in range(n):
        args = [FAKE] * n
        args[i] = None
        assert fn(ctypes.byref(d), ctypes.byref(routing()), *args, None) == \
            _lib.MOE_ERR_INVALID_ARG
    assert fn(ctypes.byref(d), None, *([FAKE] * n), None) == -1
    assert fn(ctypes.byref(d), ctypes.byref(routing(slot_of=None)),
              *([FAKE] * n), None) == -1
    if "combine" in name:
        assert fn(ctypes.byref(d), ctypes.byref(routing(topk_w=None)),
                  *([FAKE] * n), None) == -1
    # no tokens: nothing is looked at
    assert fn(ctypes.byref(desc(T=0)), None, *([None] * n), None) == 0


def test_backward_refuses_missing_arguments():
    d = desc()
    need = _lib.lib().moe_grad_workspace_size(ctypes.byref(d))
    assert need > 0
    assert backward(d, x=None) == -1
    assert backward(d, dy=None) == -1
    for name in ("w_router", "w1", "w2"):
        assert backward(d, w=weights(**{name: None})) == -1
    for name in ("topk_idx", "topk_w", "offsets", "slot_of", "f"):
        assert backward(d, r=routing(**{name: None})) == -1
    assert backward(d, ws=None) == _lib.MOE_ERR_WORKSPACE
    assert backward(d, ws_bytes=need - 1) == _lib.MOE_ERR_WORKSPACE
    s = desc(n_shared=1)
    assert backward(s) == -1
    assert backward(s, w=weights(ws1=FAKE)) == -1
    g = desc(activation=2)
    assert backward(g) == -1
    assert backward(desc(activation=2, n_shared=1),
                    w=weights(w3=FAKE, ws1=FAKE, ws2=FAKE)) == -1
    # nothing wanted, and nothing to zero: no work
    assert backward(d, g=_lib.MoeGrads()) == 0
    assert backward(desc(T=0), g=_lib.MoeGrads()) == 0


def test_router_grad_refuses_missing_arguments():
    d = desc()
    need = _lib.lib().moe_router_grad_workspace_size(ctypes.byref(d))
    assert 0 < need < _lib.lib().moe_grad_workspace_size(ctypes.byref(d))
    assert router_grad(d, x=None) == -1
    assert router_grad(d, dw=None) == -1
    assert router_grad(d, w=weights(w_router=None)) == -1
    for name in ("topk_idx", "topk_w", "slot_of", "f"):
        assert router_grad(d, r=routing(**{name: None})) == -1
    assert router_grad(d, ws=None) == _lib.MOE_ERR_WORKSPACE
    assert router_grad(d, ws_bytes=need - 1) == _lib.MOE_ERR_WORKSPACE
    assert router_grad(desc(T=0), g=_lib.MoeGrads()) == 0


def test_misaligned_tensors_are_refused():
    d, odd = desc(n_shared=1, activation=2), FAKE + 8
    ws = dict(ws1=FAKE, ws2=FAKE, w3=FAKE, ws3=FAKE)
    for name, n in ROWS.items():
        fn = getattr(_lib.lib(), name)
        for i in range(2 if n == 2 else 3):     # (dw is plain float)
            args = [FAKE + 4096 * i for i in range(n)]
            args[i] += 8
            assert fn(ctypes.byref(d), ctypes.byref(routing()), *args,
                      None) == -1
    out = grads(x=FAKE + 4096)
    for kw in (dict(x=odd), dict(dy=odd)):
        assert backward(d, w=weights(**ws), g=out, **kw) == -1
    for name in ("w_router", "w1", "b1", "w2", "b2", "w3", "ws1", "bs2"):
        assert backward(d, w=weights(**{**ws, name: odd}), g=out) == -1
    for name, _ in _lib.MoeGrads._fields_:
        if name != "b_router":
            assert backward(d, w=weights(**ws), g=grads(**{name: odd})) == -1
    assert backward(d, w=weights(**ws), g=out,
                    ws=odd) == _lib.MOE_ERR_WORKSPACE
    assert router_grad(d, x=odd, g=out) == -1
    assert router_grad(d, w=weights(w_router=odd), g=out) == -1
    assert router_grad(d, g=grads(w_router=odd)) == -1
    assert router_grad(d, g=out, ws=odd) == _lib.MOE_ERR_WORKSPACE


def test_outputs_over_inputs_are_refused():
    d, a, b, c = desc(), FAKE, FAKE + 4096, FAKE + 8192
    L, r = _lib.lib(), routing()
    for name, args in (("moe_dispatch_rows", (a, a)),
                       ("moe_dispatch_rows_grad", (a, a)),
                       ("moe_combine_rows", (a, a)),
                       ("moe_combine_rows_grad", (a, b, a, c))):
        assert getattr(L, name)(ctypes.byref(d), ctypes.byref(r), *args,
                                None) == -1
    assert backward(d, g=grads(x=FAKE)) == -1
    assert router_grad(d, g=grads(x=FAKE)) == -1


def clip(items, max_norm=1.0, norm=FAKE, ws=FAKE, ws_bytes=1 << 30, n=None):
    arr = (_lib.MoeTensor * max(1, len(items)))(*items)
    return _lib.lib().moe_clip_grads(len(items) if n is None else n, arr,
                                     max_norm, norm, ws, ws_bytes, None)


def test_clip_refusals():
    ok = (FAKE, FAKE, 8, 0)
    assert clip([ok], n=-1) == -1
    assert clip([ok], norm=None) == -1
    for bad in (-1.0, float("nan"), float("inf")):
        assert clip([ok], max_norm=bad) == -1
    assert clip([ok], ws=None) == _lib.MOE_ERR_WORKSPACE
    assert clip([ok], ws_bytes=0) == _lib.MOE_ERR_WORKSPACE
    assert clip([ok, (None, FAKE, 8, 0)]) == -1
    assert clip([ok, (FAKE, FAKE, -1, 0)]) == -1
    assert clip([ok, (FAKE, FAKE, 8, 5)]) == _lib.MOE_ERR_UNSUPPORTED
    assert clip([ok, (FAKE + 2, FAKE, 8, 0)]) == -1      # misaligned float
    assert clip([ok, (FAKE, FAKE + 1, 8, 1)]) == -1
    assert clip([(FAKE, FAKE, 1 << 41, 1)]) == _lib.MOE_ERR_UNSUPPORTED
    assert _lib.lib().moe_clip_workspace_size(-1) == 0
    assert _lib.lib().moe_clip_workspace_size(0) > 0
    assert _lib.lib().moe_clip_workspace_size(1000) < 1 << 20


def test_binding_checks():
    d = moe.make_desc(4, 64, 2, 1, 64, torch.float32)
    r = moe.Routing(4, 2, 1, "cpu")
    x, rows = torch.zeros(4, 64), torch.zeros(4, 64)
    with pytest.raises(ValueError):
        moe.moe_dispatch_rows(d, r, x[:3], rows)
    with pytest.raises(ValueError):
        moe.moe_dispatch_rows(d, r, x, rows[:3])
    with pytest.raises(ValueError):
        moe.moe_dispatch_rows(d, r, x.bfloat16(), rows)
    with pytest.raises(ValueError):
        moe.moe_dispatch_rows(d, r, torch.zeros(64, 4).t(), rows)
    with pytest.raises(ValueError):      # routing of another token count
        moe.moe_dispatch_rows(d, moe.Routing(5, 2, 1, "cpu"), x, rows)
    with pytest.raises(ValueError):
        moe.moe_combine_rows_grad(d, r, x, rows, rows, torch.zeros(4, 2))
    with pytest.raises(ValueError):
        moe.Grads(d, "cpu", ("w4",))
    with pytest.raises(ValueError):
        moe.Grads(d, "cpu", (), w1=torch.zeros(2, 64, 63))
    g = moe.Grads(d, "cpu", ("x", "b1"), w2=torch.zeros(2, 64, 64))
    assert sorted(g.as_dict()) == ["b1", "w2", "x"]
    with pytest.raises(ValueError):
        moe.RouterWeights(torch.zeros(2, 64), torch.zeros(3))
    t, n = torch.zeros(8), torch.zeros(1)
    ws = torch.zeros(moe.moe_clip_workspace_size([t]), dtype=torch.uint8)
    for bad in ([t.double()], [t[::2]], [t, t]):
        with pytest.raises(ValueError):
            moe.moe_clip_grads(bad, 1.0, n, ws)
    for out in ([], [t.bfloat16()], [torch.zeros(7)]):
        with pytest.raises(ValueError):
            moe.moe_clip_grads([t], 1.0, n, ws, out=out)
    with pytest.raises(ValueError):
        moe.moe_clip_grads([t], 1.0, n, ws[:8])


@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu"])
@pytest.mark.parametrize("choice", [False, True])
def test_reference_gradient_against_differences(act, choice):
    """The float64 loss's autograd gradient (what the kernels are held to)
    against central differences of the same loss, the routing held."""
    g = torch.Generator().manual_seed(3)

    def n(*s, v=0.5):
        return torch.randn(*s, generator=g, dtype=torch.float64) * v

    T, d, E, F = 5, 4, 3, 4
    w = {"w_router": n(E, d), "b_router": n(E), "expert_bias": None,
         "w1": n(E, F, d), "b1": n(E, F), "w2": n(E, d, F), "b2": n(E, d),
         "ws1": n(F, d), "bs1": None, "ws2": n(d, F), "bs2": None}
    if act == "swiglu":
        w.update(w3=n(E, F, d), b3=n(E, F), ws3=n(F, d), bs3=None)
    x, dy = n(T, d), n(T, d)
    r = ref.route(x @ w["w_router"].t() + w["b_router"], 2,
                  2 if choice else 3, choice)
    leaves = {"x": x, **{k: v for k, v in w.items() if v is not None}}
    for v in leaves.values():
        v.requires_grad_()
    total = ref.loss(w, x, dy, r, act, choice, 1, 0.01, 0.7, 0.3)
    got = dict(zip(leaves, torch.autograd.grad(total, leaves.values())))
    h = 1e-5
    with torch.no_grad():
        for name, v in leaves.items():
            flat = v.view(-1)
            for i in range(0, flat.numel(), 3):
                old = float(flat[i])
                flat[i] = old + h
                up = ref.loss(w, x, dy, r, act, choice, 1, 0.01, 0.7, 0.3)
                flat[i] = old - h
                down = ref.loss(w, x, dy, r, act, choice, 1, 0.01, 0.7, 0.3)
                flat[i] = old
                diff = float(up - down) / (2 * h)
                # truncation h^2 f'''/6 and rounding 1e-16 / h, of values
                # of order 1
                assert abs(diff - float(got[name].view(-1)[i])) < 1e-8, name
