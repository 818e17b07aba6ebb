"""Dense layers beside the sparse one: linear layers with an epilogue
(moe_linear), the feed-forward block (moe_dense_*) and their gradients.

Shapes and layouts are those of include/moe.h: x [M][K], w and w3 [N][K],
y [M][N]; the block's w1 and w3 [d_ff][d], w2 [d][d_ff].  All tensors of a
call are contiguous, of one dtype (float32 or bfloat16) and on one GPU.
Activations: "none", "gelu", "silu", and gated "swiglu" (SiLU(x w^T + b) *
(x w3^T + b3)) and "geglu" (with GELU).
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _lib
from ._lib import (MoeDenseDesc, MoeDenseGrads, MoeDenseWeights,
                   MoeLinearDesc, MoeLinearGrads, MoeLinearWeights)
from .layer import (_DT, _TORCH, _capturing, _check, _grad_ws, _need, _opt,
                    _ptr, _run)

_ACT = {"gelu": _lib.MOE_ACT_GELU, "silu": _lib.MOE_ACT_SILU,
        "swiglu": _lib.MOE_ACT_SWIGLU, "none": _lib.MOE_ACT_NONE,
        "geglu": _lib.MOE_ACT_GEGLU}
_GATED = (_lib.MOE_ACT_SWIGLU, _lib.MOE_ACT_GEGLU)


def _type_and_act(dtype, activation):
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    if activation not in _ACT:
        raise ValueError(f"unknown activation {activation!r}")
    return _DT[dtype], _ACT[activation]


@functools.lru_cache(maxsize=1024)
def _size_of(name: str, kind, sizes: tuple) -> int:
    """A function of the descriptor's numbers alone."""
    desc = kind(*sizes)
    n = getattr(_lib.lib(), name)(ctypes.byref(desc))
    if n == 0:
        raise _lib.MoeError(name, _lib.MOE_ERR_INVALID_ARG)
    return n


def _linear_size(name: str, d) -> int:
    return _size_of(name, MoeLinearDesc,
                    (d.M, d.N, d.K, d.dtype, d.activation))


def _dense_size(name: str, d) -> int:
    return _size_of(name, MoeDenseDesc,
                    (d.T, d.d, d.d_ff, d.dtype, d.activation))


class _Weights:
    """Weight tensors by name; ``_struct``: the C struct of their pointers."""

    def _set(self, shapes: dict, required, **given):
        first = given[required[0]]
        self.dtype, self.device = first.dtype, first.device
        if self.dtype not in _DT:
            raise ValueError(f"unsupported dtype {self.dtype}")
        for name, t in given.items():
            (_need if name in required else _opt)(
                t, name, shapes[name], self.dtype, self.device)
            setattr(self, name, t)

    def struct(self):
        return self._struct(*[_ptr(getattr(self, n))
                              for n, _ in self._struct._fields_])


class LinearWeights(_Weights):
    """Weights of a linear layer: w [N][K], b [N]; gated: w3, b3 as well."""

    _struct = MoeLinearWeights

    def __init__(self, w, b=None, w3=None, b3=None):
        if w3 is None and b3 is not None:
            raise ValueError("b3 needs w3")
        self.N, self.K = w.shape
        self.gated = w3 is not None
        shapes = {"w": (self.N, self.K), "b": (self.N,),
                  "w3": (self.N, self.K), "b3": (self.N,)}
        self._set(shapes, ("w",), w=w, b=b, w3=w3, b3=b3)


class DenseWeights(_Weights):
    """Weights of the feed-forward block: w1 [d_ff][d], w2 [d][d_ff], biases
    b1 [d_ff] and b2 [d]; gated: w3 and b3 like w1 and b1."""

    _struct = MoeDenseWeights

    def __init__(self, w1, w2, w3=None, b1=None, b2=None, b3=None):
        if w3 is None and b3 is not None:
            raise ValueError("b3 needs w3")
        self.d_ff, self.d = w1.shape
        self.gated = w3 is not None
        F, d = self.d_ff, self.d
        shapes = {"w1": (F, d), "b1": (F,), "w2": (d, F), "b2": (d,),
                  "w3": (F, d), "b3": (F,)}
        self._set(shapes, ("w1", "w2"), w1=w1, w2=w2, w3=w3, b1=b1, b2=b2,
                  b3=b3)


class _Grads:
    """Gradient buffers by name, of the shapes and the type of what they are
    the gradients of; None: not wanted."""

    def _set(self, desc, shapes: dict, device, names, given):
        dt = _TORCH[desc.dtype]
        for name in (*names, *given):
            if name not in shapes:
                raise ValueError(f"unknown gradient {name!r}")
        for name, shape in shapes.items():
            t = given.get(name)
            if t is not None:
                _need(t, name, shape, dt, t.device)
            elif name in names:
                t = torch.empty(shape, dtype=dt, device=device)
            setattr(self, name, t)

    @classmethod
    def _of(cls, given: dict):
        """The buffers as they are (the call that uses them checks them)."""
        g = cls.__new__(cls)
        for n, _ in cls._struct._fields_:
            setattr(g, n, given.get(n))
        return g

    def as_dict(self) -> dict:
        """The wanted gradients by name."""
        return {n: getattr(self, n) for n, _ in self._struct._fields_
                if getattr(self, n) is not None}

    def struct(self):
        return self._struct(*[_ptr(getattr(self, n))
                              for n, _ in self._struct._fields_])

    def _check(self, shapes: dict, dtype, device):
        for name, t in self.as_dict().items():
            _check(t, "gradient " + name, shapes[name], dtype, device)


def _linear_shapes(desc) -> dict:
    N, K = desc.N, desc.K
    return {"x": (desc.M, K), "w": (N, K), "b": (N,), "w3": (N, K),
            "b3": (N,)}


def _dense_shapes(desc) -> dict:
    d, F = desc.d, desc.d_ff
    return {"x": (desc.T, d), "w1": (F, d), "b1": (F,), "w2": (d, F),
            "b2": (d,), "w3": (F, d), "b3": (F,)}


class LinearGrads(_Grads):
    """Gradients of a linear layer: ``names`` of "x", "w", "b", "w3", "b3"
    are allocated, buffers given by name (``w=...``) are used as they are."""

    _struct = MoeLinearGrads

    def __init__(self, desc: MoeLinearDesc, device, names=(), **given):
        self._set(desc, _linear_shapes(desc), device, names, given)


class DenseGrads(_Grads):
    """Gradients of the feed-forward block: ``names`` of "x", "w1", "b1",
    "w2", "b2", "w3", "b3" are allocated, buffers given by name are used."""

    _struct = MoeDenseGrads

    def __init__(self, desc: MoeDenseDesc, device, names=(), **given):
        self._set(desc, _dense_shapes(desc), device, names, given)


# ---------------------------------------------------------------- linear

def make_linear_desc(M: int, N: int, K: int, dtype: torch.dtype,
                     activation: str = "none") -> MoeLinearDesc:
    """M rows of K features to N features (multiples of 64)."""
    dt, act = _type_and_act(dtype, activation)
    return MoeLinearDesc(M, N, K, dt, act)


def moe_linear_workspace_size(desc: MoeLinearDesc) -> int:
    return _linear_size("moe_linear_workspace_size", desc)


def moe_linear_grad_workspace_size(desc: MoeLinearDesc) -> int:
    return _linear_size("moe_linear_grad_workspace_size", desc)


def _of_linear(desc, x, w, what):
    if (w.N, w.K) != (desc.N, desc.K) or _DT[w.dtype] != desc.dtype or \
            w.gated != (desc.activation in _GATED):
        raise ValueError(f"{what}: weights of another layer")
    _check(x, "x", (desc.M, desc.K), w.dtype, w.device)


def moe_linear(desc, x, w: LinearWeights, y, ws, residual=None) -> None:
    """y [M][N] = residual + act(x w^T + b), or the gated form.  ``ws`` of
    moe_linear_workspace_size(desc) bytes."""
    _of_linear(desc, x, w, "moe_linear")
    _check(y, "y", (desc.M, desc.N), w.dtype, w.device)
    if residual is not None:
        _check(residual, "residual", (desc.M, desc.N), w.dtype, w.device)
    p, n = _grad_ws(moe_linear_workspace_size(desc), ws, w.device)
    _run("moe_linear", w.device, ctypes.byref(desc), x.data_ptr(),
         ctypes.byref(w.struct()), _ptr(residual), y.data_ptr(), p, n)


def moe_linear_grad(desc, x, w: LinearWeights, dy, g: LinearGrads, ws,
                    dx_add=None) -> None:
    """Gradients of sum(dy * y) for dy [M][N] into the buffers of g (g.x plus
    ``dx_add``).  ``ws`` of moe_linear_grad_workspace_size(desc) bytes."""
    _of_linear(desc, x, w, "moe_linear_grad")
    _check(dy, "dy", (desc.M, desc.N), w.dtype, w.device)
    if dx_add is not None:
        _check(dx_add, "dx_add", (desc.M, desc.K), w.dtype, w.device)
    g._check(_linear_shapes(desc), w.dtype, w.device)
    p, n = _grad_ws(moe_linear_grad_workspace_size(desc), ws, w.device)
    _run("moe_linear_grad", w.device, ctypes.byref(desc), x.data_ptr(),
         ctypes.byref(w.struct()), dy.data_ptr(), _ptr(dx_add),
         ctypes.byref(g.struct()), p, n)


# ----------------------------------------------------------------- block

def make_dense_desc(T: int, d: int, d_ff: int, dtype: torch.dtype,
                    activation: str = "swiglu") -> MoeDenseDesc:
    """T tokens of a feed-forward block (d, d_ff multiples of 64)."""
    dt, act = _type_and_act(dtype, activation)
    return MoeDenseDesc(T, d, d_ff, dt, act)


def moe_dense_workspace_size(desc: MoeDenseDesc) -> int:
    return _dense_size("moe_dense_workspace_size", desc)


def moe_dense_grad_workspace_size(desc: MoeDenseDesc) -> int:
    return _dense_size("moe_dense_grad_workspace_size", desc)


def _of_dense(desc, x, w, what):
    if (w.d, w.d_ff) != (desc.d, desc.d_ff) or \
            _DT[w.dtype] != desc.dtype or \
            w.gated != (desc.activation in _GATED):
        raise ValueError(f"{what}: weights of another layer")
    _check(x, "x", (desc.T, desc.d), w.dtype, w.device)


def moe_dense_forward(desc, x, w: DenseWeights, y, ws,
                      residual=None) -> None:
    """y [T][d] = residual + W2 h + b2 with h = act(W1 x + b1), or the gated
    form.  ``ws`` of moe_dense_workspace_size(desc) bytes."""
    _of_dense(desc, x, w, "moe_dense_forward")
    shape = (desc.T, desc.d)
    _check(y, "y", shape, w.dtype, w.device)
    if residual is not None:
        _check(residual, "residual", shape, w.dtype, w.device)
    p, n = _grad_ws(moe_dense_workspace_size(desc), ws, w.device)
    _run("moe_dense_forward", w.device, ctypes.byref(desc), x.data_ptr(),
         ctypes.byref(w.struct()), _ptr(residual), y.data_ptr(), p, n)


def moe_dense_backward(desc, x, w: DenseWeights, dy, g: DenseGrads, ws,
                       dx_add=None) -> None:
    """Gradients of sum(dy * y) for dy [T][d] into the buffers of g (g.x plus
    ``dx_add``).  ``ws`` of moe_dense_grad_workspace_size(desc) bytes."""
    _of_dense(desc, x, w, "moe_dense_backward")
    shape = (desc.T, desc.d)
    _check(dy, "dy", shape, w.dtype, w.device)
    if dx_add is not None:
        _check(dx_add, "dx_add", shape, w.dtype, w.device)
    g._check(_dense_shapes(desc), w.dtype, w.device)
    p, n = _grad_ws(moe_dense_grad_workspace_size(desc), ws, w.device)
    _run("moe_dense_backward", w.device, ctypes.byref(desc), x.data_ptr(),
         ctypes.byref(w.struct()), dy.data_ptr(), _ptr(dx_add),
         ctypes.byref(g.struct()), p, n)


class DenseLayer:
    """The feed-forward block of a layer that is not sparse: weights plus a
    workspace.

    ``activation``: "gelu", "silu", or "swiglu" (the default when the weights
    carry w3) or "geglu".  ``forward(x, residual)`` returns y, ``backward``
    the gradients; nothing is kept between the two.  The calls of one layer
    share its workspace: run them one after the other."""

    def __init__(self, weights: DenseWeights,
                 activation: Optional[str] = None):
        if activation is None:
            activation = "swiglu" if weights.gated else "gelu"
        act = _type_and_act(weights.dtype, activation)[1]
        if activation == "none":
            raise ValueError("the block needs an activation")
        if (act in _GATED) != weights.gated:
            raise ValueError("a gated activation needs w3, and w3 needs one")
        self.w = weights
        self.activation = activation
        self._grads = None          # the weights' gradients
        self._ws = None             # what calls of every T share
        self._plans = {}            # (T, backward): descriptor, workspace
        self._captured = set()      # plans that a graph works in

    def _plan(self, T: int, backward: bool):
        """(descriptor, workspace) of calls of T tokens.  The workspace is
        replaced when a larger call needs more; calls that were captured into
        a graph keep theirs."""
        key = (T, backward)
        if key not in self._plans:
            w = self.w
            desc = make_dense_desc(T, w.d, w.d_ff, w.dtype, self.activation)
            need = (moe_dense_grad_workspace_size if backward
                    else moe_dense_workspace_size)(desc)
            old = self._ws
            if old is None or old.numel() < need:
                if old is not None:
                    need = max(need, old.numel() + old.numel() // 4)
                    if old.is_cuda:
                        old.record_stream(
                            torch.cuda.current_stream(old.device))
                    self._plans = {k: p for k, p in self._plans.items()
                                   if k in self._captured}
                self._ws = torch.empty(need, dtype=torch.uint8,
                                       device=w.device)
            self._plans[key] = (desc, self._ws)
        if _capturing(self.w.device):
            self._captured.add(key)
        return self._plans[key]

    def forward(self, x: torch.Tensor,
                residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        """residual + the block's output, of x's shape (T, d) or (B, S, d)."""
        shape = x.shape
        x = x.reshape(-1, shape[-1]).contiguous()
        if residual is not None:
            if residual.shape != shape:
                raise ValueError(f"residual: shape {tuple(residual.shape)} "
                                 f"!= {tuple(shape)}")
            residual = residual.reshape(x.shape).contiguous()
        desc, ws = self._plan(x.shape[0], False)
        y = torch.empty_like(x)
        moe_dense_forward(desc, x, self.w, y, ws, residual=residual)
        return y.view(shape)

    def backward(self, x: torch.Tensor, dy: torch.Tensor,
                 residual: bool = False) -> DenseGrads:
        """Gradients of sum(dy * y) of x and of every weight, for the forward
        that had this x.  ``residual``: x was its residual as well (dy is
        added to x's gradient).  The weights' gradients are the same buffers
        on every call: use or copy them before the next.  x's gradient is
        (T, d) also for a (B, S, d) input."""
        x = x.reshape(-1, x.shape[-1]).contiguous()
        dy = dy.reshape(-1, dy.shape[-1]).contiguous()
        desc, ws = self._plan(x.shape[0], True)
        if self._grads is None:
            self._grads = DenseGrads(desc, self.w.device, [
                n for n in ("w1", "b1", "w2", "b2", "w3", "b3")
                if getattr(self.w, n) is not None]).as_dict()
        g = DenseGrads._of({"x": torch.empty_like(x), **self._grads})
        moe_dense_backward(desc, x, self.w, dy, g, ws,
                           dx_add=dy if residual else None)
        return g
