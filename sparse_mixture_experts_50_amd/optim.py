"""AdamW over many tensors in one call (moe_adamw_step), with its states.

The arithmetic runs in the HIP kernels; this module holds the states, checks
arguments and marshals the list.
"""
from __future__ import annotations

import ctypes
from array import array
from typing import Optional, Sequence

import torch

from . import _lib
from .layer import _DT, _capturing, _need, _run

BLOCK = 32           # elements of an 8-bit state that share a scale

_address, _index = torch.Tensor.data_ptr, torch.Tensor.get_device
_contiguous, _shape = torch.Tensor.is_contiguous, torch.Tensor.shape.__get__


class AdamW:
    """AdamW with decoupled weight decay over contiguous float32 / bfloat16
    tensors of one GPU, updated in place.

    ``lr``, ``betas``, ``eps``: attributes that may change between steps.
    ``weight_decay``: one number, or one for each parameter; fixed.
    ``state_bits``: 32 (float32 moments) or 8 (E4M3 codes in blocks of 32
    that share a power of two; the second moment as its square root, whose
    random rounding leaves the moment itself 2 to 5 % high in a long run).
    ``master``: keep a float32 copy of every bfloat16 parameter, on which the
    step is taken.  ``stochastic``: round bfloat16 parameters without such a
    copy at random instead of to nearest.  ``seed``: of the random roundings,
    which are the same for the same seed and step.
    ``device_steps``: count steps on the GPU, as a step that is captured into
    a graph needs.  ``lr_scale``: float32 [1] on the GPU that multiplies
    ``lr`` (a schedule that a graph's replays see), or None.

    The states are the lists ``m`` and ``v`` (float32, or float8_e4m3fn with
    ``m_scale`` and ``v_scale``: uint8 exponents + 127, one per block) and
    ``master`` (None where there is no copy); ``steps`` counts the steps done.
    A loaded checkpoint is copied into them or put in their place (tensors of
    the same shape and type, aligned to 16 bytes but for the scales), and
    parameters that are loaded into their master copies too.  Parameters stay
    where they are (a step refuses one that has moved), and so do the states
    once a step was captured into a graph."""

    def __init__(self, params: Sequence[torch.Tensor], lr: float,
                 betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 state_bits: int = 32, master: bool = False,
                 stochastic: bool = False, seed: int = 0,
                 device_steps: bool = False,
                 lr_scale: Optional[torch.Tensor] = None):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW: no parameters")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits {state_bits}: 8 or 32")
        self.device = self.params[0].device
        self.lr, self.betas, self.eps = lr, tuple(betas), eps
        self.state_bits, self.stochastic = state_bits, bool(stochastic)
        self.seed = seed
        count = len(self.params)
        if isinstance(weight_decay, (int, float)):
            weight_decay = [weight_decay] * count
        if len(weight_decay) != count:
            raise ValueError("weight_decay: one, or one for each parameter")
        self.weight_decay = [float(d) for d in weight_decay]
        if lr_scale is not None:
            _need(lr_scale, "lr_scale", (1,), torch.float32, self.device)
        self.lr_scale = lr_scale
        self._dev_steps = torch.zeros(
            1, dtype=torch.int64, device=self.device) if device_steps else None
        self._host_steps = 0
        self.m, self.v, self.master = [], [], []
        self.m_scale = [] if state_bits == 8 else None
        self.v_scale = [] if state_bits == 8 else None
        seen = set()
        for i, p in enumerate(self.params):
            if p.dtype not in _DT:
                raise ValueError(f"parameter {i}: unsupported dtype {p.dtype}")
            if p.device != self.device or not p.is_contiguous():
                raise ValueError(f"parameter {i}: contiguous tensors of one "
                                 "device")
            if p.numel() and p.data_ptr() in seen:
                raise ValueError(f"parameter {i} is given twice")
            seen.add(p.data_ptr())
            dt = torch.float32 if state_bits == 32 else torch.uint8
            for moments, scales in ((self.m, self.m_scale),
                                    (self.v, self.v_scale)):
                t = torch.zeros(p.shape, dtype=dt, device=self.device)
                if state_bits == 8:
                    t = t.view(torch.float8_e4m3fn)
                    scales.append(torch.zeros(
                        (p.numel() + BLOCK - 1) // BLOCK, dtype=torch.uint8,
                        device=self.device))
                moments.append(t)
            self.master.append(p.detach().float() if master and
                               p.dtype == torch.bfloat16 else None)
        self._build()

    def _build(self):
        """The list of moe_adamw_step, as its 64-bit words; a step fills in
        the gradients, the counts and the types."""
        count = len(self.params)
        self._list = (_lib.MoeAdamwTensor * count)()
        words = memoryview(self._list).cast("B").cast("q")
        self._grad_words, self._type_words = words[1::10], words[9::10]
        self._types = None           # of the gradients in the list
        self._captured = False       # whether a graph holds the addresses
        self._memory = []
        self._shapes = [p.shape for p in self.params]
        for e, p, decay in zip(self._list, self.params, self.weight_decay):
            e.param, e.weight_decay = p.data_ptr(), decay
        # what the entries of each list of states have to be
        self._states = {}
        for name in ("m", "v", "m_scale", "v_scale", "master"):
            own = getattr(self, name) or [None] * count
            if any(t is not None for t in own):
                self._states[name] = [None if t is None else (t.shape, t.dtype)
                                      for t in own]
        self._hold()

    def _all(self):
        """The tensors whose addresses the list holds, in a fixed order."""
        own = [*self.params, *self.m, *self.v]
        if self.state_bits == 8:
            own += (*self.m_scale, *self.v_scale)
        if "master" in self._states:
            own += [t for t in self.master if t is not None]
        return own

    def _hold(self):
        """Takes over the states' addresses.  They are held under other names
        too: while these live, no other memory gets one of the addresses.
        What was replaced is given back once the steps behind are done."""
        for name, want in self._states.items():
            own = getattr(self, name)
            if len(own) != len(want):
                raise ValueError(f"{name}: as many as there are parameters")
            for i, (t, need) in enumerate(zip(own, want)):
                if need is not None:
                    _need(t, f"{name} of parameter {i}", *need, self.device)
                elif t is not None:
                    raise ValueError(f"{name} of parameter {i}: there is none")
        places = [t.data_ptr() for t in self._all()]
        if len(set(places) - {0}) != sum(map(bool, places)):
            raise ValueError("a state is given twice")
        for name in self._states:
            for e, t in zip(self._list, getattr(self, name)):
                setattr(e, name, None if t is None else t.data_ptr())
        for t in self._memory:
            if t.is_cuda:
                t.record_stream(torch.cuda.current_stream(t.device))
        self._places, self._memory = places, [t.detach() for t in self._all()]

    def _check_places(self):
        """Refuses a parameter that has moved; takes over states that were put
        in others' place."""
        own = self._all()
        try:
            if list(map(_address, own)) == self._places:
                return
        except TypeError:            # not a tensor
            pass
        if len(self.params) != len(self._shapes):
            raise ValueError("parameters were added or taken away")
        for i, (p, at) in enumerate(zip(self.params, self._places)):
            if p.data_ptr() != at:
                raise ValueError(f"parameter {i} has moved")
        if self._captured:
            raise ValueError("a captured step keeps its states: copy into "
                             "them instead")
        self._hold()

    def _set_types(self, types):
        """The gradients' types (None: no gradient) into the list."""
        for i, t in enumerate(types):
            if t is not None and t not in _DT:
                raise ValueError(f"gradient {i}: unsupported dtype {t}")
        for i, (e, p, t) in enumerate(zip(self._list, self.params, types)):
            e.numel = 0 if t is None else self._shapes[i].numel()
            # the last word: the parameter's type, the gradient's above it
            if t is not None:
                self._type_words[i] = _DT[p.dtype] | _DT[t] << 32
        self._types = types

    @property
    def steps(self) -> int:
        """Steps done (with device_steps: waits for the GPU)."""
        if self._dev_steps is not None:
            return int(self._dev_steps)
        return self._host_steps

    @steps.setter
    def steps(self, n: int) -> None:
        if n < 0:
            raise ValueError("steps must not be negative")
        if self._dev_steps is not None:
            self._dev_steps.fill_(n)
        self._host_steps = n

    def step(self, grads, norm: Optional[torch.Tensor] = None,
             max_norm: float = 1.0) -> None:
        """One step with the gradients of the parameters, in their order: of
        their shapes, contiguous, float32 or bfloat16; None leaves a parameter
        and its states as they are.  ``norm``: float32 [1] as moe_grad_norm
        leaves it: the gradients are scaled by min(1, max_norm / (norm +
        1e-6)) on the way."""
        if len(grads) != len(self.params):
            raise ValueError("as many gradients as there are parameters")
        capturing = _capturing(self.device)
        if capturing and self._dev_steps is None:
            raise ValueError("a captured step needs device_steps=True")
        if norm is not None:
            _need(norm, "norm", (1,), torch.float32, self.device)
        if self.lr_scale is not None:
            _need(self.lr_scale, "lr_scale", (1,), torch.float32, self.device)
        self._check_places()
        self._captured = self._captured or capturing
        device = self.device
        try:                         # (20 tensors: 1 us less than the loop)
            right = (list(map(_shape, grads)) == self._shapes and
                     all(map(_contiguous, grads)) and
                     set(map(_index, grads)) == {device.index})
        except TypeError:            # a gradient is None
            right = False
        if not right:
            for i, (g, shape) in enumerate(zip(grads, self._shapes)):
                if g is not None:
                    _need(g, f"gradient {i}", shape, g.dtype, device)
        types = [None if g is None else g.dtype for g in grads]
        if types != self._types:
            self._set_types(types)
        self._grad_words[:] = array("q", [0 if g is None else g.data_ptr()
                                          for g in grads])
        h = _lib.MoeAdamw(
            self.lr, self.betas[0], self.betas[1], self.eps,
            self._host_steps + 1,
            None if self._dev_steps is None else self._dev_steps.data_ptr(),
            None if self.lr_scale is None else self.lr_scale.data_ptr(),
            None if norm is None else norm.data_ptr(), max_norm,
            self.state_bits, int(self.stochastic), self.seed & 0xFFFFFFFF)
        _run("moe_adamw_step", device, ctypes.byref(h), len(self.params),
             self._list)
        self._host_steps += 1
