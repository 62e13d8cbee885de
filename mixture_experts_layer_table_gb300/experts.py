"""Binding of the operators for experts outside the layer (include/mok.h): rows moved by a schedule table
and back, and E4M3 operands with a scale for each block of 128: quantisers, grouped products, weight gradients.

As in ``_native``: argument marshalling only, every step runs in the library's CUDA kernels, the
stream is PyTorch's current stream unless given, and there is no fallback.  A tensor that a call makes belongs to the
stream of the call, as if that were the current one.  Tensors are on the current
device.  Rows (tokens, expert rows, E4M3 rows, scales) may be further apart than they are long; E4M3 rows start
at multiples of 16 bytes (``empty_e4m3``).

An expert's two products in training, with ``offsets``, ``src_of`` and ``row_of`` of ``schedule``:

    xq = fp8_quantize(x, src_of=src_of, k=k, offsets=offsets)              # sorted rows, both layouts
    hu = w13.matmul(xq["q"], xq["scale"], offsets)
    aq = fp8_quantize(hu, source="swiglu", offsets=offsets)
    y = merge_rows(w2.matmul(aq["q"], aq["scale"], offsets), row_of, k, gates)
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Dict, Optional

import torch

from ._native import _check, _settle, _stream, load

P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64

E4M3 = torch.float8_e4m3fn
ELEM_TYPES = {torch.float32: 0, torch.bfloat16: 1}
SOURCES = {"plain": 0, "swiglu": 1, "swiglu_grad": 2}


class RowsDesc(ctypes.Structure):
    _fields_ = [("T", I64), ("R", I64), ("H", I64), ("token_stride", I64), ("row_stride", I64), ("k", I32), ("type", I32)]


class Fp8QuantizeDesc(ctypes.Structure):
    _fields_ = [("R", I64), ("C", I64), ("T", I64), ("x_stride", I64), ("grad_stride", I64), ("q_stride", I64),
                ("scale_stride", I64), ("qt_stride", I64), ("E", I32), ("k", I32), ("source", I32), ("type", I32)]


class Fp8WeightsDesc(ctypes.Structure):
    _fields_ = [("N", I64), ("K", I64), ("q_stride", I64), ("qt_stride", I64), ("E", I32), ("type", I32)]


class Fp8MatmulDesc(ctypes.Structure):
    _fields_ = [("R", I64), ("N", I64), ("K", I64), ("x_stride", I64), ("x_scale_stride", I64), ("w_stride", I64),
                ("out_stride", I64), ("E", I32), ("out_type", I32)]


class Fp8WeightGradDesc(ctypes.Structure):
    _fields_ = [("R", I64), ("N", I64), ("H", I64), ("dy_stride", I64), ("x_stride", I64), ("E", I32), ("out_type", I32)]


_FNS: Dict[str, object] = {}


def _fn(name, desc, pointers):
    """The entry point `name`: a descriptor, `pointers` addresses and the stream."""
    fn = _FNS.get(name)
    if fn is None:
        fn = getattr(load(), name)
        fn.argtypes = [ctypes.POINTER(desc)] + [P] * (pointers + 1)
        fn.restype = I32
        _FNS[name] = fn
    return fn


# The current device's index and a device's current stream, without what torch.cuda adds to them (0.5 us of a call).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _device(t, name) -> int:
    """The index of the device that a CUDA tensor is on: the current one."""
    device = t.get_device() if isinstance(t, torch.Tensor) else -1
    if device < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_current_device()}")
    return device


def _expect(t, shape, dtype, name, device):
    if not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape) or t.dtype is not dtype:
        got = f"{tuple(t.shape)} {t.dtype}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {got}")
    if not t.is_cuda or t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{device}, got {t.device}")


def _packed(t, shape, dtype, name, device) -> int:
    """The address of a contiguous tensor of this shape and type."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _expect(t, shape, dtype, name, device)
    raise ValueError(f"{name} must be contiguous")


def _optional(t, shape, dtype, name, device) -> Optional[int]:
    return None if t is None else _packed(t, shape, dtype, name, device)


def _rows(t, shape, dtype, name, device, unit=1):
    """(address, row stride) of a [rows][width] tensor whose rows are contiguous, do not overlap and start at multiples
    of `unit` elements; a stride of 0 stands for the packed one."""
    try:
        if not (t.shape == shape and t.dtype is dtype and t.get_device() == device):
            _expect(t, shape, dtype, name, device)
    except AttributeError:
        _expect(t, shape, dtype, name, device)
    rows, width = shape
    if t.is_contiguous() and (unit == 1 or width % unit == 0):
        return t.data_ptr(), 0
    if (width > 1 and t.stride(1) != 1) or (rows > 1 and (t.stride(0) < width or t.stride(0) % unit)):
        raise ValueError(f"{name}: rows must be contiguous, must not overlap and must start at multiples of {unit} "
                         f"elements, got strides {t.stride()}")
    return t.data_ptr(), t.stride(0) if rows > 1 else 0


def _queue(stream, device):
    """The handle of the stream of a call: the device's current one unless given."""
    return _raw_stream(device) if stream is None and _raw_stream is not None else _stream(stream)


_HERE = contextlib.nullcontext()


def _on(stream):
    """The context in which a call makes its buffers: its stream's, whose allocator gives out no memory that another stream
    is still to write, and on which a fill comes in front of the kernel."""
    if stream is None:
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        # 0 and 1 both name the default stream, which is no external one to PyTorch
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def empty_e4m3(*shape, device="cuda") -> torch.Tensor:
    """An uninitialised E4M3 tensor whose rows (of the last dimension) start at multiples of 16 bytes."""
    width = shape[-1]
    return torch.empty((*shape[:-1], -(-width // 16) * 16), dtype=torch.uint8, device=device).view(E4M3)[..., :width]


def _blocks(n) -> int:
    return -(-n // 128)


# ------------------------------------------------------------------ rows by a schedule table

def _elem(t, name) -> int:
    """The mok_elem_type of a matrix."""
    kind = ELEM_TYPES.get(t.dtype) if isinstance(t, torch.Tensor) and t.dim() == 2 else None
    if kind is None:
        raise ValueError(f"{name}: expected a float32 or bfloat16 matrix, got "
                         f"{(tuple(t.shape), t.dtype) if isinstance(t, torch.Tensor) else type(t).__name__}")
    return kind


def gather_rows(x: torch.Tensor, src_of: torch.Tensor, k: int, gates: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Sorted rows [R][H] of tokens x [T][H] (mok_gather_rows): row r is gates[a] x[a / k], a = src_of[r]; zeros where
    src_of is -1.  ``device_status``: int32 [2] CUDA tensor for an index out of range."""
    kind, dtype = _elem(x, "x"), x.dtype
    device = _device(x, "x")
    T, H = x.shape
    R = src_of.shape[0] if isinstance(src_of, torch.Tensor) and src_of.dim() == 1 else -1
    if out is None:
        with _on(stream):
            out = torch.empty((max(0, R), H), dtype=dtype, device=x.device)
    xp, xs = _rows(x, (T, H), dtype, "x", device)
    op, os_ = _rows(out, (R, H), dtype, "out", device)
    d = RowsDesc(T, R, H, xs, os_, k, kind)
    code = _fn("mok_gather_rows", RowsDesc, 5)(
        d, xp, _packed(src_of, (R,), torch.int32, "src_of", device),
        _optional(gates, (T, k), torch.float32, "gates", device), op,
        _optional(device_status, (2,), torch.int32, "device_status", device), _queue(stream, device))
    if code:
        _check("mok_gather_rows", code)
    return out


def _tokens(row_of, k, name="row_of") -> int:
    if not isinstance(row_of, torch.Tensor) or row_of.dim() != 1 or k < 1 or row_of.shape[0] % k:
        raise ValueError(f"{name}: expected an int32 vector of T k = T {k} rows")
    return row_of.shape[0] // k


def merge_rows(o: torch.Tensor, row_of: torch.Tensor, k: int, gates: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Tokens [T][H] of sorted rows o [R][H] (mok_merge_rows): y[t] = sum_j gates[t][j] o[row_of[t k + j]], where
    row_of is -1 nothing.  Without gates the gradient of ``gather_rows``."""
    kind, dtype = _elem(o, "o"), o.dtype
    device = _device(o, "o")
    R, H = o.shape
    T = _tokens(row_of, k)
    if out is None:
        with _on(stream):
            out = torch.empty((T, H), dtype=dtype, device=o.device)
    rp, rs = _rows(o, (R, H), dtype, "o", device)
    yp, ys = _rows(out, (T, H), dtype, "out", device)
    d = RowsDesc(T, R, H, ys, rs, k, kind)
    code = _fn("mok_merge_rows", RowsDesc, 5)(
        d, rp, _packed(row_of, (T * k,), torch.int32, "row_of", device),
        _optional(gates, (T, k), torch.float32, "gates", device), yp,
        _optional(device_status, (2,), torch.int32, "device_status", device), _queue(stream, device))
    if code:
        _check("mok_merge_rows", code)
    return out


def merge_rows_backward(dy: torch.Tensor, o: torch.Tensor, row_of: torch.Tensor, gates: Optional[torch.Tensor] = None,
                        out: Optional[Dict[str, torch.Tensor]] = None, device_status: Optional[torch.Tensor] = None,
                        stream=None) -> Dict[str, torch.Tensor]:
    """Gradient of ``merge_rows`` (mok_merge_rows_backward): {"do": [R][H], "dgates": f32 [T][k]}.  Rows of "do" that
    no assignment names are left as they were (zeros where it is made here).  ``out``: buffers, without "dgates" where
    that is not wanted."""
    kind, dtype = _elem(dy, "dy"), dy.dtype
    device = _device(dy, "dy")
    T, H = dy.shape
    if gates is not None and (not isinstance(gates, torch.Tensor) or gates.dim() != 2):
        raise ValueError("gates: expected a float32 matrix")
    if gates is not None:
        k = gates.shape[1]
    else:
        if not isinstance(row_of, torch.Tensor) or row_of.dim() != 1 or (row_of.shape[0] % T if T else row_of.shape[0]):
            raise ValueError(f"row_of: expected an int32 vector of T k = {T} k rows")
        k = row_of.shape[0] // T if T else 1
    R = o.shape[0] if isinstance(o, torch.Tensor) and o.dim() == 2 else -1
    yp, ys = _rows(dy, (T, H), dtype, "dy", device)
    rp, rs = _rows(o, (R, H), dtype, "o", device)
    if out is None:  # rows as far apart as those of o
        with _on(stream):
            out = {"do": torch.zeros((R, rs or H), dtype=dtype, device=dy.device)[:, :H],
                   "dgates": torch.empty((T, k), dtype=torch.float32, device=dy.device)}
    elif "do" not in out:
        raise ValueError('out: expected "do", and "dgates" where it is wanted')
    dp, ds = _rows(out["do"], (R, H), dtype, 'out["do"]', device)
    if ds != rs and (ds or H) != (rs or H):
        raise ValueError(f'out["do"]: rows {ds or H} elements apart, those of o {rs or H}')
    d = RowsDesc(T, R, H, ys, rs, k, kind)
    code = _fn("mok_merge_rows_backward", RowsDesc, 7)(
        d, yp, rp, _packed(row_of, (T * k,), torch.int32, "row_of", device),
        _optional(gates, (T, k), torch.float32, "gates", device), dp,
        _optional(out.get("dgates"), (T, k), torch.float32, 'out["dgates"]', device),
        _optional(device_status, (2,), torch.int32, "device_status", device), _queue(stream, device))
    if code:
        _check("mok_merge_rows_backward", code)
    return out


# ------------------------------------------------------------------ E4M3 in blocks of 128

def fp8_columns(R: int, E: int) -> int:
    """Columns P of the transposed layout of R rows in E groups: 128 (R / 128 + E)."""
    return 128 * (R // 128 + E)


def fp8_quantize(x: torch.Tensor, source: str = "plain", grad: Optional[torch.Tensor] = None,
                 src_of: Optional[torch.Tensor] = None, k: int = 1, gates: Optional[torch.Tensor] = None,
                 offsets: Optional[torch.Tensor] = None, rows: bool = True,
                 out: Optional[Dict[str, torch.Tensor]] = None, device_status: Optional[torch.Tensor] = None,
                 stream=None) -> Dict[str, torch.Tensor]:
    """E4M3 rows with f32 scales for each 128 elements (mok_fp8_quantize).

    ``source``: "plain" (x [R][C], or with ``src_of`` the gathered rows of tokens x [T][C], times ``gates`` where
    given), "swiglu" (silu(h) u of x = h | u [R][2C]) or "swiglu_grad" (dh | du of x = h | u [R][C] and ``grad`` = da
    [R][C/2]).  Returns {"q" [R][C], "scale" [C/128][R]} (without ``rows`` neither) and, with the groups' ``offsets``
    [E+1], {"qt" [C][P], "qt_scale" [P/128][C]}: along each group's rows, for ``fp8_weight_grad``.  ``out``: buffers
    for the pairs that are wanted."""
    kind, dtype = _elem(x, "x"), x.dtype
    device = _device(x, "x")
    if source not in SOURCES:
        raise ValueError(f"source must be one of {', '.join(SOURCES)}, got {source!r}")
    T, width = x.shape
    R = T
    if src_of is not None:
        R = src_of.shape[0] if isinstance(src_of, torch.Tensor) and src_of.dim() == 1 else -1
    if source == "swiglu" and width % 2:
        raise ValueError(f"x: h | u has an even width, got {width}")
    C = width // 2 if source == "swiglu" else width
    E = 0
    if offsets is not None:
        E = offsets.shape[0] - 1 if isinstance(offsets, torch.Tensor) and offsets.dim() == 1 else 0
        if E < 1:
            raise ValueError("offsets: expected an int32 vector of E + 1 row offsets")
    if out is None:
        new = lambda *s: torch.empty(s, dtype=torch.float32, device=x.device)  # noqa: E731
        out = {}
        with _on(stream):
            if rows:
                out |= {"q": empty_e4m3(max(0, R), C, device=x.device), "scale": new(_blocks(C), max(0, R))}
            if E:
                out |= {"qt": empty_e4m3(C, fp8_columns(R, E), device=x.device), "qt_scale": new(R // 128 + E, C)}
    for elements, scale in (("q", "scale"), ("qt", "qt_scale")):
        if (elements in out) != (scale in out):
            raise ValueError(f'out: "{elements}" and "{scale}" come together')
    if "q" in out and not rows:
        raise ValueError('out["q"] is given, but no rows are wanted')
    d = Fp8QuantizeDesc(R, C, T, 0, 0, 0, 0, 0, E, k, SOURCES[source], kind)
    xp, d.x_stride = _rows(x, (T, width), dtype, "x", device)
    gp = qp = sp = tp = tsp = None
    if grad is not None:
        gp, d.grad_stride = _rows(grad, (R, C // 2), dtype, "grad", device)
    if "q" in out:
        qp, d.q_stride = _rows(out["q"], (R, C), E4M3, 'out["q"]', device, 16)
        sp, d.scale_stride = _rows(out["scale"], (_blocks(C), R), torch.float32, 'out["scale"]', device)
    if "qt" in out:
        if not E:
            raise ValueError('out["qt"] needs the groups\' offsets')
        tp, d.qt_stride = _rows(out["qt"], (C, fp8_columns(R, E)), E4M3, 'out["qt"]', device, 16)
        tsp = _packed(out["qt_scale"], (R // 128 + E, C), torch.float32, 'out["qt_scale"]', device)
    code = _fn("mok_fp8_quantize", Fp8QuantizeDesc, 10)(
        d, xp, gp, _optional(src_of, (R,), torch.int32, "src_of", device),
        _optional(gates, (T, k), torch.float32, "gates", device),
        _optional(offsets, (E + 1,), torch.int32, "offsets", device), qp, sp, tp, tsp,
        _optional(device_status, (2,), torch.int32, "device_status", device), _queue(stream, device))
    if code:
        _check("mok_fp8_quantize", code)
    return out


class Fp8Weights:
    """Weights [E][N][K] (or [N][K]) in E4M3 with an f32 scale for each 128 x 128.

    ``q`` [E][N][K] and ``scale`` [E][N/128][K/128] serve ``matmul``; with ``transposed`` there are ``qt`` [E][K][N] and
    ``qt_scale`` too, for ``matmul_transposed``.  ``device_status`` (int32 [2]) receives what goes wrong on the
    device.  Making one waits for the current stream."""

    def __init__(self, w: torch.Tensor, transposed: bool = False):
        if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
            raise ValueError("w: expected [E][N][K] or [N][K]")
        shape = (1, *w.shape) if w.dim() == 2 else tuple(w.shape)
        self._make(*shape, transposed, w.device)
        self.quantize(w)
        _settle(w.device)

    @classmethod
    def empty(cls, E: int, N: int, K: int, transposed: bool = False, device="cuda") -> "Fp8Weights":
        """Room for weights that ``quantize`` fills."""
        self = cls.__new__(cls)
        self._make(E, N, K, transposed, device)
        _settle(self.q.device)
        return self

    @classmethod
    def of(cls, q: torch.Tensor, scale: torch.Tensor, qt: Optional[torch.Tensor] = None,
           qt_scale: Optional[torch.Tensor] = None) -> "Fp8Weights":
        """Weights in hand, e.g. of a checkpoint: E4M3 elements (rows at multiples of 16 bytes) and scales."""
        if not isinstance(q, torch.Tensor) or q.dim() not in (2, 3):
            raise ValueError("q: expected [E][N][K] or [N][K]")
        if (qt is None) != (qt_scale is None):
            raise ValueError("qt and qt_scale come together")
        for t, name in ((scale, "scale"), (qt, "qt"), (qt_scale, "qt_scale")):
            if t is not None and not isinstance(t, torch.Tensor) or name == "scale" and t is None:
                raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")
        if q.dim() == 2:
            q, scale = q.unsqueeze(0), scale.unsqueeze(0)
            qt, qt_scale = (None, None) if qt is None else (qt.unsqueeze(0), qt_scale.unsqueeze(0))
        self = cls.__new__(cls)
        self.shape = tuple(q.shape)
        self.q, self.scale, self.qt, self.qt_scale = q, scale, qt, qt_scale
        self._finish()
        _settle(self.q.device)
        return self

    def _make(self, E, N, K, transposed, device):
        self.shape = (E, N, K)
        new = lambda *s: torch.empty(s, dtype=torch.float32, device=device)  # noqa: E731
        self.q, self.scale = empty_e4m3(E, N, K, device=device), new(E, _blocks(N), _blocks(K))
        self.qt = empty_e4m3(E, K, N, device=device) if transposed else None
        self.qt_scale = new(E, _blocks(K), _blocks(N)) if transposed else None
        self._finish()

    def _finish(self):
        E, N, K = self.shape
        self._index = _device(self.q, "q")
        self._q = self._elements(self.q, (E, N, K), "q")
        self._scale = _packed(self.scale, (E, _blocks(N), _blocks(K)), torch.float32, "scale", self._index)
        self._qt, self._qt_scale = (None, 0), None
        if self.qt is not None:
            self._qt = self._elements(self.qt, (E, K, N), "qt")
            self._qt_scale = _packed(self.qt_scale, (E, _blocks(K), _blocks(N)), torch.float32, "qt_scale", self._index)
        self.device_status = torch.zeros(2, dtype=torch.int32, device=self.q.device)
        self._status = self.device_status.data_ptr()

    def _elements(self, t, shape, name):
        """(address, bytes between rows) of [E][rows][width] elements, one row after the other."""
        _expect(t, shape, E4M3, name, self._index)
        E, rows, width = shape
        ld = t.stride(1) if rows > 1 else t.stride(0) if E > 1 else -(-width // 16) * 16
        if (width > 1 and t.stride(2) != 1) or ld % 16 or ld < width or (E > 1 and t.stride(0) != rows * ld):
            raise ValueError(f"{name}: rows must be contiguous, evenly apart and start at multiples of 16 bytes, got "
                             f"strides {t.stride()}")
        return t.data_ptr(), ld

    def quantize(self, w: torch.Tensor, stream=None) -> "Fp8Weights":
        """Takes new weights (f32 or bf16, contiguous) into the buffers (mok_fp8_quantize_weights)."""
        E, N, K = self.shape
        _device(w, "w")
        if w.dtype not in ELEM_TYPES:
            raise ValueError("w: expected float32 or bfloat16 weights")
        shape = (N, K) if w.dim() == 2 and E == 1 else self.shape
        d = Fp8WeightsDesc(N, K, self._q[1], self._qt[1], E, ELEM_TYPES[w.dtype])
        code = _fn("mok_fp8_quantize_weights", Fp8WeightsDesc, 5)(
            d, _packed(w, shape, w.dtype, "w", self._index), self._q[0], self._scale, self._qt[0], self._qt_scale,
            _queue(stream, self._index))
        if code:
            _check("mok_fp8_quantize_weights", code)
        return self

    def matmul(self, x: torch.Tensor, x_scale: torch.Tensor, offsets: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """x W^T (mok_fp8_matmul): rows x [R][K] ("q" and "scale" of ``fp8_quantize``) of each group with its
        weights -> [R][N], bf16 or f32.  ``offsets``: int32 [E+1]; without, one group of all rows.  Rows of no group
        are left as they were."""
        E, N, K = self.shape
        return self._matmul(x, x_scale, offsets, out, dtype, stream, N, K, self._q, self._scale)

    def matmul_transposed(self, x: torch.Tensor, x_scale: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
        """x W: rows x [R][N] -> [R][K], e.g. the gradient of ``matmul`` with respect to its rows."""
        if self.qt is None:
            raise ValueError("made without transposed weights")
        E, N, K = self.shape
        return self._matmul(x, x_scale, offsets, out, dtype, stream, K, N, self._qt, self._qt_scale)

    def _matmul(self, x, x_scale, offsets, out, dtype, stream, N, K, w, w_scale):
        device = self._index
        if device != _current_device():
            raise ValueError(f"the weights are on cuda:{device}, not on the current device")
        E = self.shape[0]
        if offsets is None and E != 1:
            raise ValueError(f"{E} groups need their offsets")
        R = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() == 2 else -1
        if out is None:
            with _on(stream):
                out = torch.empty((max(0, R), N), dtype=dtype, device=self.q.device)
        elif isinstance(out, torch.Tensor):
            dtype = out.dtype
        if dtype not in ELEM_TYPES:
            raise ValueError(f"out is float32 or bfloat16, got {dtype}")
        d = Fp8MatmulDesc(R, N, K, 0, 0, w[1], 0, E, ELEM_TYPES[dtype])
        xp, d.x_stride = _rows(x, (R, K), E4M3, "x", device, 16)
        sp, d.x_scale_stride = _rows(x_scale, (_blocks(K), R), torch.float32, "x_scale", device)
        op, d.out_stride = _rows(out, (R, N), dtype, "out", device)
        code = _fn("mok_fp8_matmul", Fp8MatmulDesc, 7)(
            d, xp, sp, w[0], w_scale, _optional(offsets, (E + 1,), torch.int32, "offsets", device), op, self._status,
            _queue(stream, device))
        if code:
            _check("mok_fp8_matmul", code)
        return out

    def status(self):
        """(code, site) of the first error on the device since the last call; waits for the work of all of its streams."""
        return _read_status(self.device_status)


_STATUS: Dict[int, torch.Tensor] = {}  # of each device, for calls that bring no status word


def _status_of(t, device) -> Optional[int]:
    """The address of the device's status word, made by the first call that needs it.  Not under capture, whose memory is the
    graph's: there is none then."""
    word = _STATUS.get(device)
    if word is None:
        if torch.cuda.is_current_stream_capturing():
            return None
        word = torch.zeros(2, dtype=torch.int32, device=t.device)
        _settle(t.device)
        word = _STATUS.setdefault(device, word)  # another thread's, if that was first
    return word.data_ptr()


def _read_status(word):
    torch.cuda.synchronize(word.device)
    code, site = word.tolist()
    if code:
        word.zero_()
        _settle(word.device)
    return code, site


def fp8_status(device=None):
    """(code, site) of the first error on the device (the current one) of ``fp8_weight_grad`` calls without a
    ``device_status``, since the last call; waits for the work of all of its streams."""
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"device: expected a CUDA device, got {device}")
    index = device.index
    word = _STATUS.get(_current_device() if index is None else index)
    return (0, 0) if word is None else _read_status(word)


def fp8_weight_grad(dy: torch.Tensor, dy_scale: torch.Tensor, x: torch.Tensor, x_scale: torch.Tensor,
                    offsets: torch.Tensor, out: Optional[torch.Tensor] = None, dtype=torch.float32,
                    device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dW = dy^T x over each group's rows (mok_fp8_weight_grad): dy [N][P] and x [H][P] with their scales ("qt" and
    "qt_scale" of ``fp8_quantize`` with the same offsets) -> [E][N][H], f32 or bf16; zeros for a group without rows.
    A wait on the device that ran out (which leaves part of the gradient unwritten) goes to ``device_status``, or without
    one to what ``fp8_status`` reads (under capture only after a first call outside of one)."""
    try:
        (N, columns), (H, _), (E,) = dy.shape, x.shape, offsets.shape
    except (AttributeError, ValueError):
        raise ValueError("dy and x: expected matrices; offsets: expected a vector") from None
    device, E = _device(dy, "dy"), E - 1
    if E < 1 or columns % 128 or columns < 128 * E:
        raise ValueError(f"dy: expected 128 (R / 128 + E) columns, got {columns} with {E} groups")
    if out is None:
        with _on(stream):
            out = torch.empty((E, N, H), dtype=dtype, device=dy.device)
    elif isinstance(out, torch.Tensor):
        dtype = out.dtype
    if dtype not in ELEM_TYPES:
        raise ValueError(f"out is float32 or bfloat16, got {dtype}")
    # the most rows with that many columns
    d = Fp8WeightGradDesc(columns - 128 * E + 127, N, H, 0, 0, E, ELEM_TYPES[dtype])
    yp, d.dy_stride = _rows(dy, (N, columns), E4M3, "dy", device, 16)
    xp, d.x_stride = _rows(x, (H, columns), E4M3, "x", device, 16)
    code = _fn("mok_fp8_weight_grad", Fp8WeightGradDesc, 7)(
        d, yp, _packed(dy_scale, (columns // 128, N), torch.float32, "dy_scale", device), xp,
        _packed(x_scale, (columns // 128, H), torch.float32, "x_scale", device),
        _packed(offsets, (E + 1,), torch.int32, "offsets", device),
        _packed(out, (E, N, H), dtype, "out", device),
        _status_of(dy, device) if device_status is None else
        _packed(device_status, (2,), torch.int32, "device_status", device), _queue(stream, device))
    if code:
        _check("mok_fp8_weight_grad", code)
    return out
