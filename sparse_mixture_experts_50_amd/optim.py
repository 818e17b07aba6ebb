"""AdamW over many tensors in one call (moe_adamw_step), with its states.

The arithmetic runs in the HIP kernels; this module holds the states, checks
arguments and marshals the list.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from .layer import _DT, _capturing, _need, _run

BLOCK = 32           # elements of an 8-bit state that share a scale


class AdamW:
    """AdamW with decoupled weight decay over contiguous float32 / bfloat16
    tensors of one GPU, updated in place.

    ``lr``, ``betas``, ``eps``: attributes that may change between steps.
    ``weight_decay``: one number, or one for each parameter; fixed.
    ``state_bits``: 32 (float32 moments) or 8 (E4M3 codes in blocks of 32
    that share a power of two; the second moment as its square root).
    ``master``: keep a float32 copy of every bfloat16 parameter, on which the
    step is taken.  ``stochastic``: round bfloat16 parameters without such a
    copy at random instead of to nearest.  ``seed``: of the random roundings,
    which are the same for the same seed and step.
    ``device_steps``: count steps on the GPU, as a step that is captured into
    a graph needs.  ``lr_scale``: float32 [1] on the GPU that multiplies
    ``lr`` (a schedule that a graph's replays see).

    The states are the lists ``m`` and ``v`` (float32, or float8_e4m3fn with
    ``m_scale`` and ``v_scale``: uint8 exponents + 127, one per block) and
    ``master`` (None where there is no copy); ``steps`` counts the steps done.
    A loaded checkpoint is copied into them, and parameters that are loaded
    into their master copies too."""

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
        self._words = (ctypes.c_int64 * (10 * count)).from_buffer(self._list)
        self._of = []                # shape, place and size of each
        ptr = lambda t: None if t is None else t.data_ptr()
        for i, p in enumerate(self.params):
            e = self._list[i]
            e.param = p.data_ptr()
            e.m, e.v = ptr(self.m[i]), ptr(self.v[i])
            e.master = ptr(self.master[i])
            if self.state_bits == 8:
                e.m_scale = ptr(self.m_scale[i])
                e.v_scale = ptr(self.v_scale[i])
            e.weight_decay = self.weight_decay[i]
            # the last word: the parameter's type, the gradient's above it
            types = {t: _DT[p.dtype] | code << 32 for t, code in _DT.items()}
            self._of.append((p, p.shape, p.data_ptr(), p.numel(), types))

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
        if self._dev_steps is None and _capturing(self.device):
            raise ValueError("a captured step needs device_steps=True")
        if norm is not None:
            _need(norm, "norm", (1,), torch.float32, self.device)
        device, words, k = self.device, self._words, 0
        index = device.index
        for g, (p, shape, at, n, types) in zip(grads, self._of):
            if g is None:
                words[k + 7] = 0
                k += 10
                continue
            word = types.get(g.dtype)
            if word is None:
                raise ValueError(f"gradient {k // 10}: unsupported dtype "
                                 f"{g.dtype}")
            if g.get_device() != index or g.shape != shape or \
                    not g.is_contiguous():
                _need(g, f"gradient {k // 10}", shape, g.dtype, device)
            if p.data_ptr() != at:
                raise ValueError(f"parameter {k // 10} has moved")
            words[k + 1] = g.data_ptr()
            words[k + 7] = n
            words[k + 9] = word
            k += 10
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
