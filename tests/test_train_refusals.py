"""Outputs laid over inputs or over each other, and a misaligned workspace, are
refused before any HIP call (host without a GPU)."""
import ctypes

import pytest
import torch

import sparse_mixture_experts_50_amd as moe
import sparse_mixture_experts_50_amd.layer as layer_module
from sparse_mixture_experts_50_amd import _lib
from test_train_abi import desc

STEP = 1 << 40       # apart, and never dereferenced
W = {n: (100 + i) * STEP for i, (n, _) in enumerate(_lib.MoeWeights._fields_)
     if "scale" not in n}
R = {n: (200 + i) * STEP for i, (n, _) in enumerate(_lib.MoeRouting._fields_)}
OUT = [n for n, _ in _lib.MoeGrads._fields_]


def backward(grads, x=STEP, dy=2 * STEP, ws=3 * STEP, **kw):
    d = desc(n_shared=1, activation=2, **kw)
    w, r, g = _lib.MoeWeights(**W), _lib.MoeRouting(**R), \
        _lib.MoeGrads(**grads)
    return _lib.lib().moe_backward(
        ctypes.byref(d), x, ctypes.byref(w), ctypes.byref(r), dy, 1.0, 0.1,
        ctypes.byref(g), ws, 1 << 39, None)


def router(grads, x=STEP, dw=2 * STEP, dx_add=None, ws=3 * STEP):
    w, r, g = _lib.MoeWeights(**W), _lib.MoeRouting(**R), \
        _lib.MoeGrads(**grads)
    return _lib.lib().moe_router_grad(
        ctypes.byref(desc()), x, ctypes.byref(w), ctypes.byref(r), dw, dx_add,
        1.0, 0.1, ctypes.byref(g), ws, 1 << 39, None)


@pytest.mark.parametrize("name", OUT)
def test_backward_output_over_an_input(name):
    assert backward({name: STEP}) == -1                      # x
    assert backward({name: 2 * STEP}) == -1                  # dy
    for v in W.values():
        assert backward({name: v}) == -1
    for n in ("topk_idx", "topk_w", "offsets", "slot_of", "f"):
        assert backward({name: R[n]}) == -1
    assert backward({name: 3 * STEP}) == -1                  # the workspace


def test_backward_outputs_over_each_other():
    for i, a in enumerate(OUT):
        for b in OUT[:i]:
            assert backward({a: 300 * STEP, b: 300 * STEP}) == -1, (a, b)


@pytest.mark.parametrize("name", ["x", "w_router", "b_router"])
def test_router_grad_output_over_an_input(name):
    ins = [STEP, 2 * STEP, 3 * STEP, W["w_router"], W["b_router"],
           W["expert_bias"]] + [R[n] for n in ("topk_idx", "topk_w",
                                               "slot_of", "f")]
    for v in ins:
        assert router({name: v}) == -1
    if name != "x":
        assert router({name: 300 * STEP}, dx_add=300 * STEP) == -1
        assert router({name: 300 * STEP, "x": 300 * STEP}) == -1


def test_row_operators_output_over_an_input():
    L, d = _lib.lib(), desc(n_shared=1)

    def call(name, *args, **r):
        rr = _lib.MoeRouting(**{**R, **r})
        return getattr(L, name)(ctypes.byref(d), ctypes.byref(rr),
                                *[a * STEP for a in args], None)

    for name in ("moe_dispatch_rows", "moe_dispatch_rows_grad",
                 "moe_combine_rows"):
        assert call(name, 1, 1) == -1
        assert call(name, 1, 2, slot_of=2 * STEP) == -1
    assert call("moe_combine_rows", 1, 2, topk_w=2 * STEP) == -1
    for args in ((1, 2, 1, 4), (1, 2, 3, 1), (1, 2, 3, 2), (1, 2, 3, 3),
                 (1, 2, 2, 2)):
        assert call("moe_combine_rows_grad", *args) == -1
    for at in (3, 4):
        assert call("moe_combine_rows_grad", 1, 2, 3, 4,
                    slot_of=at * STEP) == -1
        assert call("moe_combine_rows_grad", 1, 2, 3, 4,
                    topk_w=at * STEP) == -1


def clip(items, norm, ws):
    arr = (_lib.MoeTensor * len(items))(*items)
    return _lib.lib().moe_clip_grads(len(items), arr, 1.0, norm, ws, 1 << 30,
                                     None)


def test_clip_norm_over_a_tensor():
    a, b = (STEP, STEP, 8, 0), (2 * STEP, 3 * STEP, 8, 1)
    for norm in (STEP, 2 * STEP, 3 * STEP, 4 * STEP):
        assert clip([a, b], norm, 4 * STEP) == -1


def test_clip_misaligned_workspace():
    for off in (1, 4, 8):
        assert clip([(STEP, STEP, 8, 0)], 2 * STEP, 3 * STEP + off) == \
            _lib.MOE_ERR_WORKSPACE


def test_clip_out_over_another_tensor(monkeypatch):
    """Each result goes to its own tensor or apart from all of them."""
    a, b, n = torch.ones(8), torch.ones(8), torch.zeros(1)
    ws = torch.zeros(moe.moe_clip_workspace_size([a, b]), dtype=torch.uint8)
    new = torch.empty(8)
    for src, out in (([a, b], [b, a]), ([a, b], [new, a]), ([a, b], [a, a]),
                     ([a, b], [b, new]), ([a, a], [a, new])):
        with pytest.raises(ValueError, match="twice|another"):
            moe.moe_clip_grads(src, 1.0, n, ws, out=out)
    sent = []
    monkeypatch.setattr(layer_module, "_run", lambda *args: sent.append(1))
    for src, out in (([a, b], [a, new]), ([a, b], [a, b]), ([a, a], [b, new]),
                     ([a, torch.empty(0)], [new, torch.empty(0)])):
        moe.moe_clip_grads(src, 1.0, n, ws, out=out)
    assert len(sent) == 4
