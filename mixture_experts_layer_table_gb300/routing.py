"""Binding of the group-limited routing (include/mok.h): expert selection from router logits, with the
load-balancing outputs, and its backward.

As in ``_native``: argument marshalling only, every step runs in the library's CUDA kernels, the
stream is PyTorch's current stream unless given, and there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import Dict, Optional

import torch

from ._native import _check, _expect, _settle, _stream, load

P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t

GROUP_MAX, GROUP_TOP2 = 0, 1
ROUTE_WS_BYTES = 98560
LOGIT_TYPES = {torch.float32: 0, torch.bfloat16: 1}


class RouteDesc(ctypes.Structure):
    _fields_ = [("T", I64), ("logits_stride", I64), ("E", I32), ("k", I32), ("router", I32), ("renorm", I32),
                ("route_scale", ctypes.c_float), ("n_group", I32), ("topk_group", I32), ("group_score", I32),
                ("logits_type", I32), ("balance_coef", ctypes.c_float), ("bias_rate", ctypes.c_float),
                ("reserved", I32)]


def make_route_desc(T, E, k, router, renorm, route_scale=1.0, n_group=1, topk_group=1, group_score=GROUP_TOP2,
                    balance_coef=0.0, bias_rate=0.0) -> RouteDesc:
    return RouteDesc(T, 0, E, k, router, int(bool(renorm)), route_scale, n_group, topk_group, group_score, 0,
                     balance_coef, bias_rate, 0)


def _route_fn():
    fn = load().mok_route
    if fn.argtypes is None:
        fn.argtypes = [ctypes.POINTER(RouteDesc)] + [P] * 11 + [SZ, P]
        fn.restype = I32
    return fn


def _route_backward_fn():
    fn = load().mok_route_backward
    if fn.argtypes is None:
        fn.argtypes = [ctypes.POINTER(RouteDesc)] + [P] * 5 + [I64, P, P]
        fn.restype = I32
    return fn


def _rows(t, T, E, dtype, name, device) -> int:
    """Row stride of a [T][E] CUDA tensor on this device whose rows are contiguous."""
    if t.shape != (T, E) or t.dtype != dtype:
        raise ValueError(f"{name}: expected ({T}, {E}) {dtype}, got {tuple(t.shape)} {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    _same_device(t, name, device)
    if T > 1 and (t.stride(1) != 1 and E > 1 or t.stride(0) < E) or T == 1 and E > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap, got strides {t.stride()}")
    return t.stride(0) if T > 1 else E


def _same_device(t, name, device):
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the router's buffers are not")


def _address(t, shape, dtype, name, device):
    """The address of a contiguous CUDA tensor of this shape and type on this device (its index)."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype and t.get_device() == device and
            t.is_contiguous()):
        _expect(t, shape, dtype, name)
        _same_device(t, name, device)
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


class Router:
    """One routing descriptor with its output buffers, which each call overwrites.  Making one with ``balance`` waits for
    the current stream, so that its zero-filled workspace is ready on every stream.

    ``forward`` returns {"topk_idx", "gates"}, with ``scores`` also "scores", and with ``balance``
    also "counts", "prob_sum", "loss", "dprob" and, where a bias is given, "bias_next"."""

    def __init__(self, desc: RouteDesc, dtype=torch.float32, balance: bool = False, scores: bool = False,
                 device="cuda"):
        if dtype not in LOGIT_TYPES:
            raise ValueError(f"logits are float32 or bfloat16, got {dtype}")
        # a descriptor of its own: the row stride is each call's
        self.desc = RouteDesc.from_buffer_copy(desc)
        self.desc.logits_type = LOGIT_TYPES[dtype]
        self.dtype, self.balance = dtype, balance
        T, E, k = desc.T, desc.E, desc.k
        new = lambda shape, dt=torch.float32: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        self.out = {"topk_idx": new((T, k), torch.int32), "gates": new((T, k))}
        if scores:
            self.out["scores"] = new((T, E))
        self.ws = None
        if balance:
            self.out |= {"counts": new((E,), torch.int32), "prob_sum": new((E,)), "loss": new((1,)), "dprob": new((E,))}
            self.ws = torch.zeros(ROUTE_WS_BYTES, dtype=torch.uint8, device=device)
            _settle(device)
        self.bias_next = new((E,)) if balance else None
        address = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._args = tuple(address(self.out.get(n))
                           for n in ("topk_idx", "gates", "scores", "counts", "prob_sum", "loss", "dprob"))
        self._ws = address(self.ws)
        self._shape, self._sel, self._experts = (T, E), (T, k), (E,)
        self._device = self.out["gates"].get_device() if self.out["gates"].is_cuda else None  # its index
        self.dlogits = None  # made by the first backward without `out`
        self._ref = ctypes.byref(self.desc)
        self._call = _route_fn()
        self._call_backward = _route_backward_fn()

    def forward(self, logits: torch.Tensor, bias: Optional[torch.Tensor] = None,
                bias_next: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
        """``bias_next``: where the moved bias goes (with ``balance`` and a bias), e.g. ``bias`` itself."""
        if bias_next is not None and (bias is None or not self.balance):
            raise ValueError("bias_next needs a bias and a router with balance")
        self._take_logits(logits)
        out, moved, b = self.out, None, None
        if bias is not None:
            b = _address(bias, self._experts, torch.float32, "bias", self._device)
            if self.balance:
                to = self.bias_next if bias_next is None else bias_next
                moved = _address(to, self._experts, torch.float32, "bias_next", self._device)
                out = dict(out, bias_next=to)
        code = self._call(self._ref, logits.data_ptr(), b, *self._args, moved, self._ws, ROUTE_WS_BYTES,
                          _stream(stream))
        if code:
            _check("mok_route", code)
        return out

    def backward(self, logits: torch.Tensor, topk_idx: Optional[torch.Tensor], dgates: Optional[torch.Tensor],
                 dprob: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Gradient with respect to the logits, in their type: ``out``, or a buffer of this object that its next
        ``backward`` without ``out`` overwrites.  ``device_status``: int32 [2] CUDA tensor."""
        self._take_logits(logits)
        idx = dg = dp = status = None
        if dgates is not None:
            dg = _address(dgates, self._sel, torch.float32, "dgates", self._device)
            idx = _address(topk_idx, self._sel, torch.int32, "topk_idx", self._device)
        if dprob is not None:
            dp = _address(dprob, self._experts, torch.float32, "dprob", self._device)
        if device_status is not None:
            status = _address(device_status, (2,), torch.int32, "device_status", self._device)
        stride = 0
        if out is None:  # 5 us of a call less than a new tensor
            if self.dlogits is None:
                self.dlogits = torch.empty(self._shape, dtype=self.dtype, device=logits.device)
            out = self.dlogits
        elif not (out.shape == self._shape and out.dtype is self.dtype and out.get_device() == self._device and
                  out.is_contiguous()):
            stride = _rows(out, *self._shape, self.dtype, "out", self._device)
        code = self._call_backward(self._ref, logits.data_ptr(), idx, dg, dp, out.data_ptr(), stride, status,
                                   _stream(stream))
        if code:
            _check("mok_route_backward", code)
        return out

    def _take_logits(self, logits):
        if (logits.shape == self._shape and logits.dtype is self.dtype and logits.get_device() == self._device and
                logits.is_contiguous()):
            self.desc.logits_stride = 0
        else:
            self.desc.logits_stride = _rows(logits, *self._shape, self.dtype, "logits", self._device)
