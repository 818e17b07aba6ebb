"""torch-facing wrappers of the C ABI, with the C entry points' names.

Only argument checking and marshalling happens here; each call enqueues the
HIP kernels on torch's current stream for the tensors' device.  Shapes and
layouts are those of include/moe.h:
  x [T][d]; w_router [E][d]; w1 [E][d_ff][d]; w2 [E][d][d_ff];
  b1 [E][d_ff]; b2 [E][d]; shared expert ws1 [d_ff][d], ws2 [d][d_ff];
  b_router / expert_bias float32 [E].
FP8 expert matrices: uint8 (or float8_e4m3fn) tensors of the same shapes
holding OCP E4M3 codes, with float32 per-output-channel scales
w1_scale [E][d_ff], w2_scale [E][d], ws1_scale [d_ff], ws2_scale [d].
SwiGLU experts add the up projection w3 [E][d_ff][d], b3 [E][d_ff] (ws3,
bs3 for the shared expert; w3_scale, ws3_scale for FP8); W1 is the gate.
Expert-sorted rows are [R + n_shared * T][d]: R = T * k routed rows (E * C
for expert choice) in slot order, then the shared expert's, one per token.
"""
from __future__ import annotations

import collections
import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import MoeDesc, MoeGrads, MoeRouting, MoeWeights, check

_DT = {torch.float32: _lib.MOE_F32, torch.bfloat16: _lib.MOE_BF16}
_ROUTING = {"topk": _lib.MOE_ROUTE_TOPK,
            "expert_choice": _lib.MOE_ROUTE_EXPERT_CHOICE}
_ACT = {"gelu": _lib.MOE_ACT_GELU, "silu": _lib.MOE_ACT_SILU,
        "swiglu": _lib.MOE_ACT_SWIGLU}


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t: Optional[torch.Tensor], name: str, shape, dtype, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _opt(t, name, shape, dtype, device):
    if t is not None:
        _need(t, name, shape, dtype, device)


def make_desc(T: int, d: int, E: int, k: int, d_ff: int, dtype: torch.dtype,
              n_shared: int = 0, capacity: int = -1,
              aux_alpha: float = 0.01, routing: str = "topk",
              expert_fp8: bool = False, activation: str = "gelu") -> MoeDesc:
    """``routing`` is "topk" or "expert_choice" (then k must be E and
    capacity the tokens each expert picks); ``expert_fp8`` marks E4M3
    expert matrices; ``activation`` is "gelu", "silu" or "swiglu"."""
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}")
    if routing not in _ROUTING:
        raise ValueError(f"unknown routing {routing!r}")
    if activation not in _ACT:
        raise ValueError(f"unknown activation {activation!r}")
    return MoeDesc(T, d, E, k, d_ff, n_shared, _DT[dtype], capacity,
                   aux_alpha, _ROUTING[routing], int(bool(expert_fp8)),
                   _ACT[activation])


def moe_capacity(T: int, E: int, capacity_factor: Optional[float]) -> int:
    """floor(T / E * cf); -1 (no limit) when cf is None."""
    if capacity_factor is None:
        return -1
    c = _lib.lib().moe_capacity(T, E, float(capacity_factor))
    if c < -1:
        check("moe_capacity", c)
    return c


def moe_workspace_size(desc: MoeDesc) -> int:
    n = _lib.lib().moe_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise _lib.MoeError("moe_workspace_size", _lib.MOE_ERR_INVALID_ARG)
    return n


def moe_gemm_variant(desc: MoeDesc, up: bool) -> int:
    """Internal id of the grouped-GEMM kernel the up (or down) projection
    runs for this descriptor (diagnostics, benchmark reports)."""
    v = _lib.lib().moe_gemm_variant(ctypes.byref(desc), 1 if up else 0)
    check("moe_gemm_variant", min(v, 0))
    return v


def moe_gemm_tail_split(desc: MoeDesc, up: bool) -> int:
    """K ranges per half-height tile of the four-wave 256-row GEMM for the
    up (or down) projection (1: no split, or another kernel runs)."""
    v = _lib.lib().moe_gemm_tail_split(ctypes.byref(desc), 1 if up else 0)
    check("moe_gemm_tail_split", min(v, 0))
    return v


def _codes(t):
    """float8_e4m3fn tensors are passed as their uint8 codes."""
    if t is not None and t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)
    return t


class Weights:
    """Device weight tensors of one layer (see module docstring).  The
    expert matrices are FP8 when given as uint8 / float8_e4m3fn codes, and
    then need their scales."""

    def __init__(self, w_router, w1, w2, b_router=None, expert_bias=None,
                 b1=None, b2=None, ws1=None, bs1=None, ws2=None, bs2=None,
                 w1_scale=None, w2_scale=None, ws1_scale=None,
                 ws2_scale=None, w3=None, b3=None, ws3=None, bs3=None,
                 w3_scale=None, ws3_scale=None):
        w1, w2, ws1, ws2 = _codes(w1), _codes(w2), _codes(ws1), _codes(ws2)
        w3, ws3 = _codes(w3), _codes(ws3)
        self.w3, self.b3, self.ws3, self.bs3 = w3, b3, ws3, bs3
        self.w3_scale, self.ws3_scale = w3_scale, ws3_scale
        self.gated = w3 is not None
        self.w_router, self.w1, self.w2 = w_router, w1, w2
        self.b_router, self.expert_bias = b_router, expert_bias
        self.b1, self.b2 = b1, b2
        self.ws1, self.bs1, self.ws2, self.bs2 = ws1, bs1, ws2, bs2
        self.w1_scale, self.w2_scale = w1_scale, w2_scale
        self.ws1_scale, self.ws2_scale = ws1_scale, ws2_scale
        E, d_ff, d = w1.shape
        self.E, self.d, self.d_ff = E, d, d_ff
        self.dtype = w_router.dtype
        self.device = w1.device
        self.n_shared = 0 if ws1 is None else 1
        self.expert_fp8 = w1.dtype == torch.uint8
        dt, dev = self.dtype, self.device
        wdt = torch.uint8 if self.expert_fp8 else dt
        f32 = torch.float32
        _need(w_router, "w_router", (E, d), dt, dev)
        _need(w1, "w1", (E, d_ff, d), wdt, dev)
        _need(w2, "w2", (E, d, d_ff), wdt, dev)
        _opt(b_router, "b_router", (E,), f32, dev)
        _opt(expert_bias, "expert_bias", (E,), f32, dev)
        _opt(b1, "b1", (E, d_ff), dt, dev)
        _opt(b2, "b2", (E, d), dt, dev)
        if self.expert_fp8:
            _need(w1_scale, "w1_scale", (E, d_ff), f32, dev)
            _need(w2_scale, "w2_scale", (E, d), f32, dev)
        if self.gated:
            _need(w3, "w3", (E, d_ff, d), wdt, dev)
            _opt(b3, "b3", (E, d_ff), dt, dev)
            if self.expert_fp8:
                _need(w3_scale, "w3_scale", (E, d_ff), f32, dev)
        if self.n_shared:
            _need(ws1, "ws1", (d_ff, d), wdt, dev)
            _need(ws2, "ws2", (d, d_ff), wdt, dev)
            _opt(bs1, "bs1", (d_ff,), dt, dev)
            _opt(bs2, "bs2", (d,), dt, dev)
            if self.expert_fp8:
                _need(ws1_scale, "ws1_scale", (d_ff,), f32, dev)
                _need(ws2_scale, "ws2_scale", (d,), f32, dev)
            if self.gated:
                _need(ws3, "ws3", (d_ff, d), wdt, dev)
                _opt(bs3, "bs3", (d_ff,), dt, dev)
                if self.expert_fp8:
                    _need(ws3_scale, "ws3_scale", (d_ff,), f32, dev)

    @staticmethod
    def from_dict(inp: dict, device=None) -> "Weights":
        def g(key):
            t = inp.get(key)
            if t is None:
                return None
            return t.to(device).contiguous() if device is not None else t
        return Weights(g("wr"), g("w1"), g("w2"), b_router=g("br"),
                       expert_bias=g("ebias"), b1=g("b1"), b2=g("b2"),
                       ws1=g("ws1"), bs1=g("bs1"), ws2=g("ws2"),
                       bs2=g("bs2"), w1_scale=g("w1_scale"),
                       w2_scale=g("w2_scale"), ws1_scale=g("ws1_scale"),
                       ws2_scale=g("ws2_scale"), w3=g("w3"), b3=g("b3"),
                       ws3=g("ws3"), bs3=g("bs3"), w3_scale=g("w3_scale"),
                       ws3_scale=g("ws3_scale"))

    def struct(self) -> MoeWeights:
        return MoeWeights(*[_ptr(t) for t in (
            self.w_router, self.b_router, self.expert_bias, self.w1, self.b1,
            self.w2, self.b2, self.ws1, self.bs1, self.ws2, self.bs2,
            self.w1_scale, self.w2_scale, self.ws1_scale, self.ws2_scale,
            self.w3, self.b3, self.ws3, self.bs3, self.w3_scale,
            self.ws3_scale)])


class Routing:
    """Device buffers of the routing results and statistics (k = E for
    expert choice).  One that MoeLayer.forward returned stands for that call:
    once a later forward has filled the same buffers, the training operators
    refuse it (``clone()`` it before)."""

    _buffers = None      # the Routing whose buffers these are, and
    _call = None         # the forward that filled them

    def __init__(self, T: int, E: int, k: int, device,
                 slots: Optional[int] = None):
        """``slots``: length of slot_token, T*k by default (expert choice
        uses E*C)."""
        i32, f32 = torch.int32, torch.float32
        z = lambda *s, dt: torch.empty(s, dtype=dt, device=device)
        self.topk_idx = z(T, k, dt=i32)
        self.topk_w = z(T, k, dt=f32)
        self.counts = z(E, dt=i32)
        self.kept = z(E, dt=i32)
        self.offsets = z(E + 1, dt=i32)
        self.slot_token = z(T * k if slots is None else slots, dt=i32)
        self.slot_of = z(T, k, dt=i32)
        self.f = z(E, dt=f32)
        self.p = z(E, dt=f32)
        self.l_aux = z(1, dt=f32)
        # z-loss, entropy (bits), load imbalance, utilization, drop rate,
        # max share
        self.monitor = z(6, dt=f32)

    def clone(self) -> "Routing":
        """A copy that later forwards leave alone."""
        self.check_current()
        out = self._copy()
        out._buffers = out._call = None
        for n, _ in MoeRouting._fields_:
            setattr(out, n, getattr(self, n).clone())
        return out

    def check_current(self) -> None:
        """Raise ValueError if a later forward has filled the buffers."""
        if self._buffers is not None and \
                self._buffers._call is not self._call:
            raise ValueError(
                "routing of an earlier forward: its buffers hold a later "
                "one's of as many tokens (clone() the routing before that)")

    def _filled(self, captured: bool) -> "Routing":
        """These buffers as one forward's results.  What a graph fills again
        on every replay stands for no one call."""
        self._call = object()
        out = self._copy()
        out._buffers = None if captured else self
        return out

    def _copy(self) -> "Routing":
        out = Routing.__new__(Routing)
        out.__dict__.update(self.__dict__)
        return out

    def struct(self) -> MoeRouting:
        return MoeRouting(*[_ptr(getattr(self, n)) for n, _ in
                            MoeRouting._fields_])


def _ws(desc, ws: torch.Tensor):
    need = moe_workspace_size(desc)
    if ws.numel() * ws.element_size() < need or not ws.is_contiguous():
        raise ValueError(f"workspace needs {need} contiguous bytes")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def moe_router_topk(desc, x, w: Weights, r: Routing, ws) -> None:
    _need(x, "x", (desc.T, desc.d), w.dtype, w.device)
    p, n = _ws(desc, ws)
    rs, wsct = r.struct(), w.struct()
    check("moe_router_topk", _lib.lib().moe_router_topk(
        ctypes.byref(desc), x.data_ptr(), ctypes.byref(wsct),
        ctypes.byref(rs), p, n, _stream(x)))


def moe_permute(desc, r: Routing, ws) -> None:
    p, n = _ws(desc, ws)
    rs = r.struct()
    check("moe_permute", _lib.lib().moe_permute(
        ctypes.byref(desc), ctypes.byref(rs), p, n, _stream(ws)))


def moe_route_dispatch(desc, x, w: Weights, r: Routing, ws) -> None:
    """moe_router_topk + moe_permute (one launch for decode-sized steps)."""
    _need(x, "x", (desc.T, desc.d), w.dtype, w.device)
    p, n = _ws(desc, ws)
    rs, wsct = r.struct(), w.struct()
    check("moe_route_dispatch", _lib.lib().moe_route_dispatch(
        ctypes.byref(desc), x.data_ptr(), ctypes.byref(wsct),
        ctypes.byref(rs), p, n, _stream(x)))


def moe_grouped_ffn(desc, x, w: Weights, r: Routing, ws) -> None:
    _need(x, "x", (desc.T, desc.d), w.dtype, w.device)
    p, n = _ws(desc, ws)
    rs, wsct = r.struct(), w.struct()
    check("moe_grouped_ffn", _lib.lib().moe_grouped_ffn(
        ctypes.byref(desc), x.data_ptr(), ctypes.byref(wsct),
        ctypes.byref(rs), p, n, _stream(x)))


def moe_ffn_up(desc, x, w: Weights, r: Routing, ws) -> None:
    _need(x, "x", (desc.T, desc.d), w.dtype, w.device)
    p, n = _ws(desc, ws)
    rs, wsct = r.struct(), w.struct()
    check("moe_ffn_up", _lib.lib().moe_ffn_up(
        ctypes.byref(desc), x.data_ptr(), ctypes.byref(wsct),
        ctypes.byref(rs), p, n, _stream(x)))


def moe_ffn_down(desc, w: Weights, r: Routing, ws) -> None:
    p, n = _ws(desc, ws)
    rs, wsct = r.struct(), w.struct()
    check("moe_ffn_down", _lib.lib().moe_ffn_down(
        ctypes.byref(desc), ctypes.byref(wsct), ctypes.byref(rs), p, n,
        _stream(ws)))


def moe_combine(desc, r: Routing, y, ws) -> None:
    _need(y, "y", (desc.T, desc.d), y.dtype, ws.device)
    p, n = _ws(desc, ws)
    rs = r.struct()
    check("moe_combine", _lib.lib().moe_combine(
        ctypes.byref(desc), ctypes.byref(rs), y.data_ptr(), p, n,
        _stream(y)))


def moe_forward(desc, x, w: Weights, r: Routing, y, ws) -> None:
    _need(x, "x", (desc.T, desc.d), w.dtype, w.device)
    _need(y, "y", (desc.T, desc.d), w.dtype, w.device)
    p, n = _ws(desc, ws)
    rs, wsct = r.struct(), w.struct()
    check("moe_forward", _lib.lib().moe_forward(
        ctypes.byref(desc), x.data_ptr(), ctypes.byref(wsct),
        ctypes.byref(rs), y.data_ptr(), p, n, _stream(x)))


def moe_forward_noalloc(desc, x, w: Weights, r: Routing, y) -> None:
    """moe_forward with the library's static device scratch instead of a
    workspace (no allocation; raises MoeError with MOE_ERR_SCRATCH when the
    shape needs more than the static buffer)."""
    _need(x, "x", (desc.T, desc.d), w.dtype, w.device)
    _need(y, "y", (desc.T, desc.d), w.dtype, w.device)
    rs, wsct = r.struct(), w.struct()
    check("moe_forward_noalloc", _lib.lib().moe_forward_noalloc(
        ctypes.byref(desc), x.data_ptr(), ctypes.byref(wsct),
        ctypes.byref(rs), y.data_ptr(), _stream(x)))


def moe_bias_update(counts, target: float, gamma: float,
                    expert_bias) -> None:
    E = expert_bias.numel()
    if counts.dtype != torch.int32 or counts.numel() != E:
        raise ValueError("counts must be int32 [E]")
    if expert_bias.dtype != torch.float32 or not expert_bias.is_contiguous():
        raise ValueError("expert_bias must be contiguous float32 [E]")
    check("moe_bias_update", _lib.lib().moe_bias_update(
        E, counts.data_ptr(), float(target), float(gamma),
        expert_bias.data_ptr(), _stream(expert_bias)))


# ------------------------------------------------------------- training

class RouterWeights:
    """The router's weights alone, for moe_router_grad beside experts that
    are not this package's: w_router [E][d], b_router / expert_bias [E]
    float32 or None."""

    def __init__(self, w_router, b_router=None, expert_bias=None):
        E, d = w_router.shape
        self.E, self.d = E, d
        self.dtype, self.device = w_router.dtype, w_router.device
        self.w_router, self.b_router = w_router, b_router
        self.expert_bias = expert_bias
        f32 = torch.float32
        _need(w_router, "w_router", (E, d), self.dtype, self.device)
        _opt(b_router, "b_router", (E,), f32, self.device)
        _opt(expert_bias, "expert_bias", (E,), f32, self.device)

    def struct(self) -> MoeWeights:
        return MoeWeights(w_router=_ptr(self.w_router),
                          b_router=_ptr(self.b_router),
                          expert_bias=_ptr(self.expert_bias))


_TORCH = {v: k for k, v in _DT.items()}


def _grad_shapes(desc: MoeDesc) -> dict:
    T, d, E, F = desc.T, desc.d, desc.E, desc.d_ff
    return {"x": (T, d), "w_router": (E, d), "b_router": (E,),
            "w1": (E, F, d), "b1": (E, F), "w2": (E, d, F), "b2": (E, d),
            "ws1": (F, d), "bs1": (F,), "ws2": (d, F), "bs2": (d,),
            "w3": (E, F, d), "b3": (E, F), "ws3": (F, d), "bs3": (F,)}


class Grads:
    """Gradient buffers of a layer, of the shapes and types of what they
    are the gradients of (b_router float32).  ``names``: the wanted ones
    ("x", "w_router", "b_router", "w1", "b1", ... "bs3"); the others are
    None.  Buffers given by name (``w1=...``) are used as they are."""

    def __init__(self, desc: MoeDesc, device, names=(), **given):
        shapes = _grad_shapes(desc)
        dt = _TORCH[desc.dtype]
        for name in (*names, *given):
            if name not in shapes:
                raise ValueError(f"unknown gradient {name!r}")
        for name, shape in shapes.items():
            t = given.get(name)
            want = torch.float32 if name == "b_router" else dt
            if t is not None:
                _need(t, name, shape, want, t.device)
            elif name in names:
                t = torch.empty(shape, dtype=want, device=device)
            setattr(self, name, t)

    def as_dict(self) -> dict:
        """The wanted gradients by name."""
        return {n: getattr(self, n) for n, _ in MoeGrads._fields_
                if getattr(self, n) is not None}

    def struct(self) -> MoeGrads:
        return MoeGrads(*[_ptr(getattr(self, n))
                          for n, _ in MoeGrads._fields_])


def _routed(desc: MoeDesc) -> int:
    if desc.routing == _lib.MOE_ROUTE_EXPERT_CHOICE:
        return desc.E * desc.capacity
    return desc.T * desc.k


def _check(t, name, shape, dtype, device):
    """_need, quick for what is right."""
    if not (t.shape == shape and t.dtype is dtype and t.device == device
            and t.is_contiguous()):
        _need(t, name, shape, dtype, device)


def _tokens(desc, t, name, device):
    _check(t, name, (desc.T, desc.d), _TORCH[desc.dtype], device)


def _rows(desc, t, name, device):
    _check(t, name, (_routed(desc) + desc.n_shared * desc.T, desc.d),
           _TORCH[desc.dtype], device)


def _routing(desc, r: Routing, device):
    """The routing buffers of this descriptor's calls."""
    r.check_current()
    if r.slot_of.device != device:
        raise ValueError(f"routing on {r.slot_of.device}, expected {device}")
    if (r.slot_of.shape != (desc.T, desc.k) or
            r.slot_token.numel() != _routed(desc) or
            r.offsets.numel() != desc.E + 1):
        raise ValueError("routing buffers of another shape")


def _slots(r: Routing) -> MoeRouting:
    """The part of the routing that the row operators read."""
    rs = MoeRouting()
    rs.slot_of = r.slot_of.data_ptr()
    rs.topk_w = r.topk_w.data_ptr()
    return rs


# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(name: str, device: torch.device, *args) -> None:
    """Call an entry point on the device's current stream, with that device
    current (a stream handle of 0 means the current device's)."""
    fn = getattr(_lib.lib(), name)
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _run(name, device, *args)
    stream = (_raw_stream(index) if _raw_stream is not None
              else torch.cuda.current_stream(device).cuda_stream)
    check(name, fn(*args, stream))


def moe_dispatch_rows(desc, r: Routing, x, xs) -> None:
    """x [T][d] into expert-sorted rows xs; rows of dropped assignments are
    left as they were."""
    dev = x.device
    _tokens(desc, x, "x", dev)
    _rows(desc, xs, "xs", dev)
    _routing(desc, r, dev)
    _run("moe_dispatch_rows", dev, ctypes.byref(desc),
         ctypes.byref(_slots(r)), x.data_ptr(), xs.data_ptr())


def moe_dispatch_rows_grad(desc, r: Routing, dxs, dx) -> None:
    """dx [T][d]: the gradient of moe_dispatch_rows for row gradients dxs."""
    dev = dx.device
    _tokens(desc, dx, "dx", dev)
    _rows(desc, dxs, "dxs", dev)
    _routing(desc, r, dev)
    _run("moe_dispatch_rows_grad", dev, ctypes.byref(desc),
         ctypes.byref(_slots(r)), dxs.data_ptr(), dx.data_ptr())


def moe_combine_rows(desc, r: Routing, ys, y) -> None:
    """Expert-sorted rows ys back into token order, weighted: y [T][d]."""
    dev = y.device
    _tokens(desc, y, "y", dev)
    _rows(desc, ys, "ys", dev)
    _routing(desc, r, dev)
    _run("moe_combine_rows", dev, ctypes.byref(desc),
         ctypes.byref(_slots(r)), ys.data_ptr(), y.data_ptr())


def moe_combine_rows_grad(desc, r: Routing, dy, ys, dys, dw) -> None:
    """Gradients of moe_combine_rows for dy [T][d]: of the rows into dys
    (may be ys itself; rows of dropped assignments are left as they were),
    of the routing weights into dw [T][k] float32."""
    dev = dy.device
    _tokens(desc, dy, "dy", dev)
    _rows(desc, ys, "ys", dev)
    _rows(desc, dys, "dys", dev)
    _check(dw, "dw", (desc.T, desc.k), torch.float32, dev)
    _routing(desc, r, dev)
    _run("moe_combine_rows_grad", dev, ctypes.byref(desc),
         ctypes.byref(_slots(r)), dy.data_ptr(), ys.data_ptr(),
         dys.data_ptr(), dw.data_ptr())


def moe_router_grad_workspace_size(desc: MoeDesc) -> int:
    n = _lib.lib().moe_router_grad_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise _lib.MoeError("moe_router_grad_workspace_size",
                            _lib.MOE_ERR_INVALID_ARG)
    return n


def moe_grad_workspace_size(desc: MoeDesc) -> int:
    n = _lib.lib().moe_grad_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise _lib.MoeError(
            "moe_grad_workspace_size", _lib.MOE_ERR_UNSUPPORTED
            if desc.expert_fp8 else _lib.MOE_ERR_INVALID_ARG)
    return n


def _grad_ws(need: int, ws: torch.Tensor, device):
    if ws.device != device:
        raise ValueError(f"workspace on {ws.device}, expected {device}")
    n = ws.numel() * ws.element_size()
    if n < need or not ws.is_contiguous():
        raise ValueError(f"workspace needs {need} contiguous bytes")
    return ws.data_ptr(), n


def _check_grads(desc, g: Grads, device):
    shapes = _grad_shapes(desc)
    for name, t in g.as_dict().items():
        want = torch.float32 if name == "b_router" else _TORCH[desc.dtype]
        _need(t, "gradient " + name, shapes[name], want, device)


def _check_router(desc, x, w, r, what):
    _tokens(desc, x, "x", w.device)
    if (w.E, w.d) != (desc.E, desc.d) or w.dtype != x.dtype:
        raise ValueError(f"{what}: weights of another layer")
    _routing(desc, r, w.device)


def moe_router_grad(desc, x, w, r: Routing, dw, g: Grads, ws,
                    aux_scale: float = 0.0, z_scale: float = 0.0,
                    dx_add=None) -> None:
    """Gradient of the router for the gradient dw [T][k] of the routing
    weights and of aux_scale * l_aux + z_scale * z-loss, into g.x (plus
    ``dx_add``), g.w_router and g.b_router where wanted.  ``w``: Weights or
    RouterWeights; ``ws`` of moe_router_grad_workspace_size(desc) bytes."""
    _check_router(desc, x, w, r, "moe_router_grad")
    _need(dw, "dw", (desc.T, desc.k), torch.float32, w.device)
    if dx_add is not None:
        _tokens(desc, dx_add, "dx_add", w.device)
    _check_grads(desc, g, w.device)
    p, n = _grad_ws(moe_router_grad_workspace_size(desc), ws, w.device)
    rs, wsct, gs = r.struct(), w.struct(), g.struct()
    _run("moe_router_grad", x.device, ctypes.byref(desc), x.data_ptr(),
         ctypes.byref(wsct), ctypes.byref(rs), dw.data_ptr(), _ptr(dx_add),
         float(aux_scale), float(z_scale), ctypes.byref(gs), p, n)


def moe_backward(desc, x, w: Weights, r: Routing, dy, g: Grads, ws,
                 aux_scale: float = 0.0, z_scale: float = 0.0) -> None:
    """Gradient of the layer (moe_forward) for dy [T][d] and of
    aux_scale * l_aux + z_scale * z-loss, into the buffers of g.  x, w and r
    are the forward's; ``ws`` of moe_grad_workspace_size(desc) bytes."""
    _check_router(desc, x, w, r, "moe_backward")
    if (w.d_ff, w.n_shared, int(w.expert_fp8)) != (
            desc.d_ff, desc.n_shared, desc.expert_fp8):
        raise ValueError("moe_backward: weights of another layer")
    _tokens(desc, dy, "dy", w.device)
    _check_grads(desc, g, w.device)
    p, n = _grad_ws(moe_grad_workspace_size(desc), ws, w.device)
    rs, wsct, gs = r.struct(), w.struct(), g.struct()
    _run("moe_backward", x.device, ctypes.byref(desc), x.data_ptr(),
         ctypes.byref(wsct), ctypes.byref(rs), dy.data_ptr(),
         float(aux_scale), float(z_scale), ctypes.byref(gs), p, n)


def moe_clip_workspace_size(tensors) -> int:
    """Workspace bytes of moe_clip_grads for these tensors."""
    return _lib.lib().moe_clip_workspace_size(len(tensors))


def moe_clip_grads(tensors, max_norm: float, norm, ws, out=None) -> None:
    """Global norm of contiguous float32 / bfloat16 tensors into norm [1]
    (float32), and the tensors scaled by min(1, max_norm / (norm + 1e-6)),
    in place or into ``out`` (tensors of the same sizes and types, each its
    own gradient or apart from all of them).  ``ws`` of
    moe_clip_workspace_size(tensors) bytes."""
    device = norm.device
    _need(norm, "norm", (1,), torch.float32, device)
    out = tensors if out is None else out
    count = len(tensors)
    if len(out) != count:
        raise ValueError("out: as many tensors as there are gradients")
    same = out is tensors
    flat, seen, pairs = [], set(), []
    for t, o in zip(tensors, out):
        n, dtype = t.numel(), _DT.get(t.dtype)
        if dtype is None:
            raise ValueError(f"unsupported dtype {t.dtype}")
        if t.device != device or not (same or (
                o.device == device and o.dtype == t.dtype
                and o.numel() == n)):
            raise ValueError("tensors of one device; out of the same sizes "
                             "and types")
        if not (t.is_contiguous() and (same or o.is_contiguous())):
            raise ValueError("tensors must be contiguous")
        src = t.data_ptr()
        dst = src if same else o.data_ptr()
        if n:
            seen.add(dst)
            pairs.append((src, dst))
        # MoeTensor: two pointers, the count, the type (and padding)
        flat += (src, dst, n, dtype)
    if len(seen) != len(pairs):
        raise ValueError("a tensor is given twice")
    if not same and not seen.isdisjoint(s for s, _ in pairs):
        times = collections.Counter(s for s, _ in pairs)
        if any(times[d] > (s == d) for s, d in pairs):
            raise ValueError("out: a tensor is another's gradient")
    arr = (ctypes.c_int64 * (4 * count))(*flat)
    p, size = _grad_ws(moe_clip_workspace_size(tensors), ws, device)
    _run("moe_clip_grads", device, count,
         ctypes.cast(arr, ctypes.POINTER(_lib.MoeTensor)), float(max_norm),
         norm.data_ptr(), p, size)


def moe_grad_norm(tensors, norm, ws) -> None:
    """The norm of moe_clip_grads alone, into norm [1]; the tensors stay as
    they are (moe_clip_grads without outputs)."""
    device = norm.device
    _need(norm, "norm", (1,), torch.float32, device)
    flat = []
    for t in tensors:
        dtype = _DT.get(t.dtype)
        if dtype is None:
            raise ValueError(f"unsupported dtype {t.dtype}")
        if t.device != device:
            raise ValueError("tensors of one device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        flat += (t.data_ptr(), 0, t.numel(), dtype)
    arr = (ctypes.c_int64 * len(flat))(*flat)
    p, size = _grad_ws(moe_clip_workspace_size(tensors), ws, device)
    _run("moe_clip_grads", device, len(tensors),
         ctypes.cast(arr, ctypes.POINTER(_lib.MoeTensor)), 0.0,
         norm.data_ptr(), p, size)


def _capturing(device: torch.device) -> bool:
    """Whether the device's current stream is being captured into a graph."""
    if device.type != "cuda":
        return False
    if device.index == torch.cuda.current_device():
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(device):
        return torch.cuda.is_current_stream_capturing()


class MoeLayer:
    """One sparse MoE FFN layer on a GPU: weights plus reusable buffers.

    ``routing="topk"``: each token picks ``k`` experts, with an optional
    capacity floor(T/E * capacity_factor).  ``routing="expert_choice"``:
    each expert picks floor(T/E * capacity_factor) tokens (``k`` is then E
    and a capacity factor is required).  ``activation``: "gelu", "silu",
    or "swiglu" (the default when the weights carry w3).

    ``forward(x)`` returns ``(y, routing)``; the routing buffers are reused
    by the next call with the same T: ``routing.clone()`` keeps them, as a
    second forward before the first one's backward needs.  ``backward`` and
    the row operators refuse a routing that a later forward has overwritten;
    they do not see the replays of a captured one."""

    def __init__(self, weights: Weights, k: int,
                 capacity_factor: Optional[float] = None,
                 aux_alpha: float = 0.01, routing: str = "topk",
                 activation: Optional[str] = None):
        if routing not in _ROUTING:
            raise ValueError(f"unknown routing {routing!r}")
        if activation is None:
            activation = "swiglu" if weights.gated else "gelu"
        if (activation == "swiglu") != weights.gated:
            raise ValueError("swiglu needs w3, and w3 needs swiglu")
        self.activation = activation
        if routing == "expert_choice":
            if capacity_factor is None:
                raise ValueError("expert choice needs a capacity factor")
            k = weights.E
        self.w = weights
        self.k = k
        self.capacity_factor = capacity_factor
        self.aux_alpha = aux_alpha
        self.routing = routing
        self._bufs = {}
        self._grads = None          # the weights' gradients
        self._grad_mem = {}         # x's gradient and the workspace, flat
        self._grad_bufs = {}
        self._captured = set()      # token counts that a graph works in

    def desc(self, T: int) -> MoeDesc:
        w = self.w
        cap = moe_capacity(T, w.E, self.capacity_factor)
        if self.routing == "expert_choice":
            cap = min(cap, T)
        return make_desc(T, w.d, w.E, self.k, w.d_ff, w.dtype,
                         n_shared=w.n_shared, capacity=cap,
                         aux_alpha=self.aux_alpha, routing=self.routing,
                         expert_fp8=w.expert_fp8, activation=self.activation)

    def buffers(self, T: int):
        if T not in self._bufs:
            desc = self.desc(T)
            nbytes = moe_workspace_size(desc)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.w.device)
            slots = None
            if self.routing == "expert_choice":
                slots = self.w.E * desc.capacity
            r = Routing(T, self.w.E, self.k, self.w.device, slots=slots)
            y = torch.empty((T, self.w.d), dtype=self.w.dtype,
                            device=self.w.device)
            self._bufs[T] = (desc, r, ws, y)
        return self._bufs[T]

    def forward(self, x: torch.Tensor):
        if x.dim() == 3:                    # (B, S, H) -> (B*S, H)
            shape = x.shape
            y, r = self.forward(x.reshape(-1, shape[-1]))
            return y.reshape(shape), r
        desc, r, ws, y = self.buffers(x.shape[0])
        moe_forward(desc, x.contiguous(), self.w, r, y, ws)
        return y, r._filled(_capturing(self.w.device))

    def _grad_flat(self, name: str, n: int, dtype) -> torch.Tensor:
        """At least n elements that calls of every T share.  Where they are
        too few, a quarter more than before at least, so that token counts
        that creep up do not reallocate each time."""
        old = self._grad_mem.get(name)
        if old is None or old.numel() < n:
            if old is not None:
                n = max(n, old.numel() + old.numel() // 4)
                if old.is_cuda:
                    old.record_stream(torch.cuda.current_stream(old.device))
                # what a captured graph writes stays as it is
                self._grad_bufs = {T: b for T, b in self._grad_bufs.items()
                                   if T in self._captured}
            self._grad_mem[name] = torch.empty(n, dtype=dtype,
                                               device=self.w.device)
        return self._grad_mem[name]

    def grad_buffers(self, T: int):
        """(descriptor, Grads of x and every weight of the layer, gradient
        workspace) for calls of T tokens.  The weights' gradients are the
        same buffers for every T, and x's gradient and the workspace share
        their memory, which is replaced when a larger call needs more; a T
        that was captured into a graph keeps the buffers of its capture."""
        if T not in self._grad_bufs:
            desc, w = self.desc(T), self.w
            need = moe_grad_workspace_size(desc)
            if self._grads is None:
                self._grads = Grads(desc, w.device, [
                    n for n in _grad_shapes(desc)
                    if getattr(w, n, None) is not None]).as_dict()
            gx = self._grad_flat("x", T * w.d, w.dtype)
            ws = self._grad_flat("ws", need, torch.uint8)
            g = Grads(desc, w.device, x=gx[:T * w.d].view(T, w.d),
                      **self._grads)
            self._grad_bufs[T] = (desc, g, ws)
        if _capturing(self.w.device):
            self._captured.add(T)
        return self._grad_bufs[T]

    def backward(self, x: torch.Tensor, routing: Routing, dy: torch.Tensor,
                 aux_scale: float = 1.0, z_scale: float = 0.0) -> Grads:
        """Gradients of sum(dy * y) + aux_scale * l_aux + z_scale * z-loss
        for the forward that had this x and left this routing (the last one
        of as many tokens, or a clone() of its routing): of x and of every
        weight (FP8 experts have none).  The buffers are reused by the next
        backward, of any T: use or copy the gradients before it, and run the
        calls of a layer one after the other.  x's gradient is (T, H) also
        for a (B, S, H) input."""
        x = x.reshape(-1, x.shape[-1]).contiguous()
        dy = dy.reshape(-1, dy.shape[-1]).contiguous()
        desc, g, ws = self.grad_buffers(x.shape[0])
        moe_backward(desc, x, self.w, routing, dy, g, ws,
                     aux_scale=aux_scale, z_scale=z_scale)
        return g

    def bias_update(self, routing: Routing, gamma: float) -> None:
        """One aux-loss-free step on weights.expert_bias from the counts of
        the last forward: target is T*k/E."""
        if self.w.expert_bias is None:
            raise ValueError("layer has no expert_bias")
        T = routing.topk_idx.shape[0]
        moe_bias_update(routing.counts, T * self.k / self.w.E, gamma,
                        self.w.expert_bias)
