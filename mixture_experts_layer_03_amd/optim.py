"""AdamW over the tensors of a model, one launch for dozens of them.

``AdamW`` keeps the states and the step count of a list of parameters and
issues moe_adamw_step (include/moe.h has the arithmetic):

    opt = AdamW([w_r, w_gu, w_down], lr=1e-4, weight_decay=0.1, state_bits=8, seed=1)
    blk.backward(...)
    opt.step([blk.dw_r, blk.dw_gu, blk.dw_down], grad_scale=clip)

States are fp32, or 8 bits with a power of two for each 128 elements.  bf16
parameters are rounded at random (alike on all ranks that have the same seed),
unless ``masters`` keeps fp32 copies of them.
"""
from __future__ import annotations

import ctypes
from array import array
from collections import OrderedDict
from operator import attrgetter

import torch

from . import abi

_dtype, _shape, _index = attrgetter("dtype"), attrgetter("shape"), torch.Tensor.get_device
_contiguous, _pointer = torch.Tensor.is_contiguous, torch.Tensor.data_ptr


def state_shapes(numel: int, state_bits: int):
    """{name: (elements, dtype)} of one tensor's state."""
    if state_bits == 32:
        return {"m": (numel, torch.float32), "v": (numel, torch.float32)}
    blocks = -(-numel // 128)
    return {"m": (numel, torch.float8_e4m3fn), "v": (numel, torch.float8_e5m2),
            "m_scale": (blocks, torch.uint8), "v_scale": (blocks, torch.uint8)}


class States(OrderedDict):
    """{name: the tensors}: other tensors in their place would not reach the kernel, so none are taken.
    Pickled and copied it is an OrderedDict."""

    def _fixed(self, *args, **kw):
        raise TypeError("AdamW: states are loaded with load_state, or copied into in place")

    __setitem__ = __delitem__ = update = pop = popitem = clear = setdefault = __ior__ = _fixed

    def __init__(self, items):
        for name, tensors in items:
            super().__setitem__(name, tensors)

    def __reduce__(self):
        return OrderedDict, (), None, None, iter(self.items())


class AdamW:
    """params: contiguous bf16 or fp32 tensors, all of one type and on one device.

    masters: True for fp32 copies made here, or a list of them; state: a dict
    of lists of tensors (as ``self.state``) to go on from, with ``step`` its
    step count.  Given tensors are stepped in place; ``state`` and ``masters``
    show them, and load_state copies into them.  weight_decay: one number or one
    for each tensor.  capturable: the step count and the learning rate live on
    the device, so that a captured step() counts on when it is replayed;
    ``set_lr`` changes the rate."""

    def __init__(self, params, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits: int = 32, masters=None, seed: int = 0, step: int = 0, state=None,
                 capturable: bool = False):
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW: no parameters")
        if state_bits not in (8, 32):
            raise ValueError("AdamW: state_bits must be 8 or 32, not %r" % (state_bits,))
        self.dtype, self.device = self.params[0].dtype, self.params[0].device
        self.dcode = abi._dtype_code(self.params[0])
        for i, p in enumerate(self.params):
            self._need("parameter", i, p, p.numel(), self.dtype)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * len(self.params)
        if len(decay) != len(self.params):
            raise ValueError("AdamW: %d weight decays for %d parameters" % (len(decay), len(self.params)))
        self.lr, self.betas, self.eps, self.state_bits = float(lr), betas, eps, state_bits
        self.seed, self.steps = int(seed) & 0xFFFFFFFFFFFFFFFF, int(step)
        if masters is True:
            masters = [p.float() for p in self.params]
        # The kernel has the states' addresses: tensor objects of their own keep that memory, whatever
        # becomes of the caller's.
        self._masters = [t.detach() for t in masters] if masters else None
        if self._masters is not None and self.dtype != torch.bfloat16:
            raise ValueError("AdamW: only bf16 parameters have fp32 copies")
        names = state_shapes(0, state_bits)
        if state is None:
            state = {n: [] for n in names}
            for p in self.params:
                for n, (count, dt) in state_shapes(p.numel(), state_bits).items():
                    t = torch.zeros(count, dtype=dt, device=self.device)
                    state[n].append(t.fill_(127) if dt == torch.uint8 else t)
        self._state = {n: [t.detach() for t in state[n]] for n in names}
        for i, p in enumerate(self.params):
            for n, (count, dt) in state_shapes(p.numel(), state_bits).items():
                self._need(n, i, self._state[n][i], count, dt)
            if self._masters is not None:
                self._need("master", i, self._masters[i], p.numel(), torch.float32)
        self._table = (abi.AdamwTensor * len(self.params))()
        for i, p in enumerate(self.params):
            t = self._table[i]
            t.param, t.numel, t.weight_decay = p.data_ptr(), p.numel(), float(decay[i])
            t.m, t.v = self._state["m"][i].data_ptr(), self._state["v"][i].data_ptr()
            if state_bits == 8:
                t.m_scale, t.v_scale = self._state["m_scale"][i].data_ptr(), self._state["v_scale"][i].data_ptr()
            if self._masters is not None:
                t.master = self._masters[i].data_ptr()
        self._shapes = [p.shape for p in self.params]
        self._pointers = [p.data_ptr() for p in self.params]
        words = ctypes.sizeof(abi.AdamwTensor) // 8
        self._grad_column = memoryview(self._table).cast("B").cast("Q")[abi.AdamwTensor.grad.offset // 8::words]
        self.lr_dev = self.step_dev = None
        if capturable:
            self.lr_dev = torch.full((1,), self.lr, dtype=torch.float32, device=self.device)
            self.step_dev = torch.full((1,), self.steps, dtype=torch.int64, device=self.device)

    @property
    def state(self):
        """{name: a tensor for each parameter}; what is written into them is what the next step reads."""
        return States((n, tuple(t.detach() for t in ts)) for n, ts in self._state.items())

    @property
    def masters(self):
        """The fp32 copies, a tensor for each parameter, or None."""
        return None if self._masters is None else tuple(t.detach() for t in self._masters)

    def load_state(self, state, step: int, masters=None):
        """Goes on from a state (as ``state``) and masters of the same sizes, on any device, after `step` steps."""
        if (masters is None) != (self._masters is None):
            raise ValueError("AdamW: masters go with an optimizer that has them")
        pairs = [(n, ts, state.get(n, ())) for n, ts in self._state.items()]
        if masters is not None:
            pairs.append(("master", self._masters, masters))
        for what, to, given in pairs:
            if len(given) != len(to):
                raise ValueError("AdamW: %s of %d tensors for %d parameters" % (what, len(given), len(to)))
            for i, (t, f) in enumerate(zip(to, given)):
                if f.numel() != t.numel() or f.dtype != t.dtype:
                    raise ValueError("AdamW: %s %d must be %d of %s, not %d of %s"
                                     % (what, i, t.numel(), t.dtype, f.numel(), f.dtype))
        for _, to, given in pairs:
            for t, f in zip(to, given):
                t.copy_(f.reshape(t.shape))
        self.steps = int(step)
        if self.step_dev is not None:
            self.step_dev.fill_(self.steps)

    def _need(self, what, i, t, numel, dtype):
        if t.numel() != numel or t.dtype != dtype or t.device != self.device or not t.is_contiguous():
            raise ValueError("AdamW: %s %d must be contiguous, %d of %s on %s, not %s of %s on %s"
                             % (what, i, numel, dtype, self.device, tuple(t.shape), t.dtype, t.device))

    def set_lr(self, lr: float):
        self.lr = float(lr)
        if self.lr_dev is not None:
            self.lr_dev.fill_(self.lr)

    def step(self, grads, grad_scale=None, stream=None):
        """One step in place.  grads: a tensor for each parameter, all fp32 or (bf16 parameters)
        all bf16; grad_scale: an fp32 device tensor of one element that multiplies them, or None.
        Everything runs on `stream` (the current one); with capturable another one is refused,
        since the count is stepped on the current one (``step_dev``; ``steps`` counts calls, not replays)."""
        if len(grads) != len(self.params):
            raise ValueError("AdamW: %d gradients for %d parameters" % (len(grads), len(self.params)))
        if self.step_dev is not None and stream is not None and stream != abi._stream(None):
            raise ValueError("AdamW: a capturable step runs on the current stream, which steps its count")
        dtype, device = grads[0].dtype, self.device
        gcode = abi._dtype_code(grads[0])
        if device.type != "cuda" or device.index != torch.cuda.current_device():
            raise ValueError("AdamW: the parameters are on %s, not on the current device" % device)
        # over the lists at once: a loop over the tensors would take longer than their kernel
        if (list(map(_shape, grads)) != self._shapes or set(map(_dtype, grads)) != {dtype}
                or set(map(_index, grads)) != {device.index} or not all(map(_contiguous, grads))):
            for i, (g, p) in enumerate(zip(grads, self.params)):
                if g.shape != p.shape:
                    raise ValueError("AdamW: gradient %d is %s, its parameter %s" % (i, tuple(g.shape), tuple(p.shape)))
                self._need("gradient", i, g, p.numel(), dtype)
        if list(map(_pointer, self.params)) != self._pointers:
            raise ValueError("AdamW: a parameter has moved")
        self._grad_column[:] = memoryview(array("Q", map(_pointer, grads)))
        if grad_scale is not None:
            self._need("grad_scale", 0, grad_scale, 1, torch.float32)
        if self.step_dev is not None:
            self.step_dev.add_(1)
        try:
            abi.moe_adamw_step(self._table, len(self.params), self.dcode, gcode, self.state_bits,
                               self.lr, self.betas[0], self.betas[1], self.eps, self.steps + 1, self.seed,
                               grad_scale, self.lr_dev, self.step_dev, stream)
        except abi.MoeError:
            if self.step_dev is not None:
                self.step_dev.sub_(1)   # nothing was stepped
            raise
        self.steps += 1
