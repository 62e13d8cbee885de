"""Binding of the training step around the layer (include/mok.h): the gradient norm with its clip
factor, and AdamW over many tensors.

As in ``_native``: argument marshalling only, every step runs in the library's CUDA kernels, the
stream is PyTorch's current stream unless given, and there is no fallback.  ``GradNorm`` and
``AdamW`` are made once for a set of buffers that a training loop keeps (the parameters and the
gradient buffers that ``MoELayer.backward(out=...)`` writes); they hold references to them.  Making one
waits for the current stream, so that the buffers it fills (a workspace, first states, f32 copies) are
ready on every stream.
"""
from __future__ import annotations

import ctypes
from typing import Dict, List, Optional, Sequence

import torch

from ._native import _check, _settle, _stream, load

P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t

ELEM_TYPES = {torch.float32: 0, torch.bfloat16: 1}
STATE_F32, STATE_MX8 = 0, 1
GRAD_NORM_WS_BYTES = 16640


class GradTensor(ctypes.Structure):
    _fields_ = [("grad", P), ("n", ctypes.c_int64), ("grad_type", I32), ("reserved", I32)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("param", P), ("master", P), ("grad", P), ("m", P), ("v", P), ("m_scale", P), ("v_scale", P),
                ("n", ctypes.c_int64), ("counter", ctypes.c_uint64), ("lr", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("param_type", I32), ("grad_type", I32), ("state_type", I32),
                ("reserved", I32)]


class AdamWHyper(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


def _fn(name, argtypes):
    fn = getattr(load(), name)
    if fn.argtypes is None:
        fn.argtypes = argtypes
        fn.restype = I32
    return fn


def _grad_norm_fn():
    return _fn("mok_grad_norm", [ctypes.POINTER(GradTensor), I32, ctypes.c_float, P, P, SZ, P])


def _adamw_fn():
    return _fn("mok_adamw_step", [ctypes.POINTER(AdamWTensor), I32, ctypes.POINTER(AdamWHyper), P, P])


def _expect_tensor(t, name, dtypes, n=None):
    """The C ABI takes bare pointers, so types, sizes and layout are checked here, on the host."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise ValueError(f"{name}: expected a tensor of {' or '.join(map(str, dtypes))}, got "
                         f"{t.dtype if isinstance(t, torch.Tensor) else type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")


def _same_device(tensors):
    devices = {t.device for t in tensors}
    if len(devices) > 1:
        raise ValueError(f"all tensors must be on one device, got {sorted(map(str, devices))}")


def grad_tensors(grads: Sequence[torch.Tensor]):
    """The mok_grad_tensor array of f32 or bf16 CUDA tensors."""
    arr = (GradTensor * max(1, len(grads)))()
    for i, g in enumerate(grads):
        _expect_tensor(g, f"grads[{i}]", (torch.float32, torch.bfloat16))
        arr[i] = GradTensor(g.data_ptr(), g.numel(), ELEM_TYPES[g.dtype], 0)
    _same_device(grads)
    return arr


class GradNorm:
    """Global 2-norm of a set of gradient buffers and the factor that clips it to ``max_norm``
    (mok_grad_norm).  ``compute`` returns a float32 [2] CUDA tensor {norm, factor} that the next
    call overwrites; the factor (``result[1:]``) is what ``AdamW.step`` takes."""

    def __init__(self, grads: Sequence[torch.Tensor], max_norm: float):
        if not max_norm > 0:
            raise ValueError(f"max_norm must be positive, got {max_norm}")
        self.grads = list(grads)
        self.max_norm = float(max_norm)
        self._table = grad_tensors(self.grads)
        device = self.grads[0].device if self.grads else torch.device("cuda")
        self.result = torch.empty(2, dtype=torch.float32, device=device)
        self.ws = torch.zeros(GRAD_NORM_WS_BYTES, dtype=torch.uint8, device=device)
        _settle(device)
        self._call = _grad_norm_fn()
        self._out, self._ws = self.result.data_ptr(), self.ws.data_ptr()

    def compute(self, stream=None) -> torch.Tensor:
        code = self._call(self._table, len(self.grads), self.max_norm, self._out, self._ws, GRAD_NORM_WS_BYTES,
                          _stream(stream))
        if code:
            _check("mok_grad_norm", code)
        return self.result


class AdamW:
    """AdamW over many tensors at once (mok_adamw_step), in place.

    ``params`` are f32 or bf16 CUDA tensors, ``grads`` the f32 or bf16 buffers their gradients are
    written to before each ``step``.  ``state``: "f32", or "mx8" for E4M3 elements with one power of
    two per 32 (1.03 bytes an element each for m and sqrt(v)).  ``masters``: None (bf16 parameters are
    rounded at random with the mean unchanged), True (f32 copies are made here) or the copies.
    ``lr`` and ``weight_decay``: one number, or one for each tensor.  ``states``: {"m", "v"} (and
    {"m_scale", "v_scale"} for "mx8") lists of tensors to go on from, e.g. of a checkpoint, with
    ``step`` the number of steps done; zero otherwise.  ``counters``: the first rounding-bit counter of
    each tensor (multiples of 8, by default one range after the other).
    """

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], lr=1e-3, betas=(0.9, 0.999),
                 eps: float = 1e-8, weight_decay=0.0, state: str = "f32", masters=None, seed: int = 0, step: int = 0,
                 states: Optional[Dict[str, List[torch.Tensor]]] = None, counters: Optional[Sequence[int]] = None):
        params, grads = list(params), list(grads)
        if len(params) != len(grads):
            raise ValueError(f"{len(params)} params and {len(grads)} grads")
        if state not in ("f32", "mx8"):
            raise ValueError(f'state must be "f32" or "mx8", got {state!r}')
        beta1, beta2 = betas
        if not (0 <= beta1 < 1 and 0 <= beta2 < 1 and eps >= 0):
            raise ValueError(f"betas must be in [0, 1) and eps >= 0, got {betas}, {eps}")
        count = len(params)
        both = (torch.float32, torch.bfloat16)
        for i, (p, g) in enumerate(zip(params, grads)):
            _expect_tensor(p, f"params[{i}]", both)
            _expect_tensor(g, f"grads[{i}]", both, p.numel())
        self.params, self.grads, self.mx8 = params, grads, state == "mx8"
        if masters is True:
            masters = [p.float() if p.dtype == torch.bfloat16 else None for p in params]
        self.masters = [None] * count if masters is None else list(masters)
        made = states or self._zero_states()
        names = ("m", "v", "m_scale", "v_scale") if self.mx8 else ("m", "v")
        self.states = {n: list(made[n]) for n in names}
        lists = [self.masters, *self.states.values()]
        if any(len(x) != count for x in lists) or (counters is not None and len(counters) != count):
            raise ValueError("masters, states and counters need one entry for each parameter")
        element = torch.float8_e4m3fn if self.mx8 else torch.float32
        for i, p in enumerate(params):
            if self.masters[i] is not None:
                if p.dtype != torch.bfloat16:
                    raise ValueError(f"masters[{i}]: only bf16 parameters have a master")
                _expect_tensor(self.masters[i], f"masters[{i}]", (torch.float32,), p.numel())
            for n in ("m", "v"):
                _expect_tensor(self.states[n][i], f"states[{n!r}][{i}]", (element,), p.numel())
            for n in names[2:]:
                _expect_tensor(self.states[n][i], f"states[{n!r}][{i}]", (torch.uint8,), -(-p.numel() // 32))
        _same_device([t for x in [params, grads, *lists] for t in x if t is not None])
        if counters is None:
            counters, at = [], 0
            for p in params:
                counters.append(at)
                at += -(-p.numel() // 32) * 32
        each = lambda x, name: [float(x)] * count if isinstance(x, (int, float)) else [float(y) for y in x]  # noqa: E731
        lrs, decays = each(lr, "lr"), each(weight_decay, "weight_decay")
        if len(lrs) != count or len(decays) != count:
            raise ValueError("lr and weight_decay: one number, or one for each parameter")
        if params:
            _settle(params[0].device)
            self._device = params[0].get_device()
        self._table = (AdamWTensor * max(1, count))()
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        for i, p in enumerate(params):
            self._table[i] = AdamWTensor(
                ptr(p), ptr(self.masters[i]), ptr(grads[i]), ptr(self.states["m"][i]), ptr(self.states["v"][i]),
                ptr(self.states["m_scale"][i]) if self.mx8 else None,
                ptr(self.states["v_scale"][i]) if self.mx8 else None, p.numel(), counters[i], lrs[i], decays[i],
                ELEM_TYPES[p.dtype], ELEM_TYPES[grads[i].dtype], STATE_MX8 if self.mx8 else STATE_F32, 0)
        self._hyper = AdamWHyper(beta1, beta2, eps, step, seed & 0xFFFFFFFF, 0)
        self._hyper_ref = ctypes.byref(self._hyper)
        self._call = _adamw_fn()

    def _zero_states(self):
        if not self.mx8:
            return {n: [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in self.params]
                    for n in ("m", "v")}
        made = {n: [torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn)
                    for p in self.params] for n in ("m", "v")}
        for n in ("m_scale", "v_scale"):
            made[n] = [torch.full((-(-p.numel() // 32),), 1, dtype=torch.uint8, device=p.device) for p in self.params]
        return made

    @property
    def steps(self) -> int:
        """Steps done."""
        return self._hyper.step

    def set_lr(self, lr):
        """One learning rate for all tensors, or one for each."""
        lrs = [float(lr)] * len(self.params) if isinstance(lr, (int, float)) else [float(x) for x in lr]
        if len(lrs) != len(self.params):
            raise ValueError("lr: one number, or one for each parameter")
        for i, x in enumerate(lrs):
            self._table[i].lr = x

    def step(self, grad_scale: Optional[torch.Tensor] = None, stream=None):
        """One step on what the gradient buffers hold; ``grad_scale``: float32 [1] CUDA tensor, the
        factor on every gradient (a NaN skips the update; the step is counted all the same, since the
        host does not wait for the factor).  A captured graph repeats the step it was captured at,
        with its number, rates and rounding bits."""
        scale = None
        if grad_scale is not None:
            if not (grad_scale.dtype is torch.float32 and grad_scale.is_cuda and grad_scale.numel() == 1):
                _expect_tensor(grad_scale, "grad_scale", (torch.float32,), 1)
            if self.params and grad_scale.get_device() != self._device:
                raise ValueError(f"grad_scale is on {grad_scale.device}, the parameters are not")
            scale = grad_scale.data_ptr()
        self._hyper.step += 1
        code = self._call(self._table, len(self.params), self._hyper_ref, scale, _stream(stream))
        if code:
            self._hyper.step -= 1
            _check("mok_adamw_step", code)

    def state_values(self, i: int) -> Dict[str, torch.Tensor]:
        """m and v of tensor i as float32 values."""
        m, v = self.states["m"][i], self.states["v"][i]
        if not self.mx8:
            return {"m": m, "v": v}
        scale = lambda n: torch.exp2(self.states[n][i].float() - 127).repeat_interleave(32)[:m.numel()]  # noqa: E731
        return {"m": (m.float().flatten() * scale("m_scale")).view(m.shape),
                "v": (v.float().flatten() * scale("v_scale")).square().view(v.shape)}
