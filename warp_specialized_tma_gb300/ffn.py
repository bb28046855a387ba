"""bf16 operators of a feed-forward block, over the C ABI of ``include/ffn_ops.h``.

    linear             act(x @ weight.T + bias) + residual, in one kernel
    linear_backward    its gradients
    gated              act(x @ w_gate.T) * (x @ w_up.T), in one kernel, with both projections
                       kept for the backward pass in bf16 or in 8 bits
    gated_backward     gradients of gated() and of the product with w_down that follows it
    device_status      whether a kernel's watchdog ran out

Matrices are bf16 CUDA tensors with contiguous rows, at any pitch and offset; sums are fp32, and
each result is rounded once.  Results that are not given have rows at multiples of 128 bytes, as
the quantisers' have: the next product reads them fastest.  Their pitch is above their width where
that is no multiple of 64.  Operands whose rows do not start at multiples of 16 bytes are copied
first, and large ones whose rows do not at multiples of 128, in every call: weights that are used
again and again are better laid out so once.

What gated() saves in 8 bits is in fp8's format: codes (float8_e4m3fn) and scales
(float8_e8m0fnu), a power of two for each row and block of 128 columns.

Every function enqueues its work on ``stream`` (default: the current stream of the tensors'
device) and returns without waiting.  The work is done by ``libffn_ops.so``; there is no
fallback.  Nothing is recorded for autograd: tensors that require a gradient are refused while
gradients are recorded, and tensors with a forward-mode tangent while tangents are; the backward
passes are called by name (as ``feedforward`` does).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import fp8

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libffn_ops.so")

# status codes (ffn_status)
OK = 0
ERR_INVALID_ARG = -1
ERR_ALIGNMENT = -2
ERR_WORKSPACE = -3
ERR_CUDA = -4
ERR_TENSORMAP = -5
ERR_DEVICE_TIMEOUT = -6
ERR_UNSUPPORTED = -7

# activations (ffn_activation)
ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

# how gated() keeps its projections
SAVES = {None: 0, "bf16": 1, "e4m3": 2}

# settings of a thread's products (ffn_option)
OPTIONS = {
    "cta_group": 1,
    "transposed": 2,
    "width": 3,
    "split": 4,
    "watchdog_ns": 5,
    "fault_skip_load": 6,
    "raster_group": 7,
    "repack": 8,
    "stream": 9,
    "together": 10,
}

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_SIGNATURES = {
    "ffn_strerror": (ctypes.c_char_p, [_I]),
    "ffn_version": (ctypes.c_char_p, []),
    "ffn_set_option": (_I, [_I, _L]),
    "ffn_get_option": (_I, [_I, ctypes.POINTER(_L)]),
    "ffn_plan_info": (_I, [_P]),
    "ffn_device_status": (_I, [ctypes.POINTER(ctypes.c_uint32)]),
}
for _name in ("linear", "linear_backward", "gated", "gated_backward"):
    _SIGNATURES[f"ffn_{_name}_workspace"] = (_I, [_P, ctypes.POINTER(_L)])
    _SIGNATURES[f"ffn_{_name}"] = (_I, [_P, _P, _L, _P])


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("tiles", ctypes.c_int64),
        ("k_blocks", ctypes.c_int64),
        ("grid_ctas", ctypes.c_int32),
        ("cta_group", ctypes.c_int32),
        ("transposed", ctypes.c_int32),
        ("width", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("split_tiles", ctypes.c_int32),
        ("cluster", ctypes.c_int32),
        ("packed", ctypes.c_int32),
        ("products", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class Matrix(ctypes.Structure):
    _fields_ = [("data", _P), ("ld", _L)]


class Quantized(ctypes.Structure):
    _fields_ = [("codes", _P), ("ld", _L), ("scales", _P)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("M", _L), ("N", _L), ("K", _L), ("x", Matrix), ("weight", Matrix), ("bias", _P),
                ("bias_type", ctypes.c_int32), ("activation", ctypes.c_int32), ("residual", Matrix), ("y", Matrix),
                ("y_type", ctypes.c_int32), ("reserved", ctypes.c_int32), ("z", Matrix)]


class LinearBackwardArgs(ctypes.Structure):
    _fields_ = [("M", _L), ("N", _L), ("K", _L), ("dy", Matrix), ("x", Matrix), ("weight", Matrix), ("z", Matrix),
                ("activation", ctypes.c_int32), ("dweight_type", ctypes.c_int32), ("dx", Matrix), ("dweight", Matrix),
                ("dbias", _P)]


class GatedArgs(ctypes.Structure):
    _fields_ = [("M", _L), ("F", _L), ("C", _L), ("x", Matrix), ("w_gate", Matrix), ("w_up", Matrix),
                ("activation", ctypes.c_int32), ("reserved", ctypes.c_int32), ("h", Matrix), ("g", Matrix),
                ("u", Matrix), ("qg", Quantized), ("qu", Quantized)]


class GatedBackwardArgs(ctypes.Structure):
    _fields_ = [("M", _L), ("F", _L), ("C", _L), ("N", _L), ("dy", Matrix), ("x", Matrix), ("g", Matrix),
                ("u", Matrix), ("qg", Quantized), ("qu", Quantized), ("w_gate", Matrix), ("w_up", Matrix),
                ("w_down", Matrix), ("activation", ctypes.c_int32), ("dweight_type", ctypes.c_int32), ("dx", Matrix),
                ("dw_gate", Matrix), ("dw_up", Matrix), ("dw_down", Matrix)]


class FfnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {load().ffn_strerror(status).decode()} (status {status})")


_lib = None
_lock = threading.Lock()


def load() -> ctypes.CDLL:
    """Loads libffn_ops.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is missing: build it with "
                                  "`python -m warp_specialized_tma_gb300.build` (needs nvcc)")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
        return _lib


def version() -> str:
    return load().ffn_version().decode()


_bind = None


def _ops():
    """The compiled tensor entry points (raises if they were not built)."""
    global _bind
    if _bind is None:
        load()
        mod = fp8._ops()
        mod.ffn_set_error(FfnError)
        _bind = mod
    return _bind


def _check(st: int, what: str) -> None:
    if st != OK:
        raise FfnError(st, what)


def _choice(table: dict, key, what: str) -> int:
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{what} must be one of {', '.join(map(repr, table))} (got {key!r})") from None


def _stream(stream, tensor):
    return contextlib.nullcontext() if stream is None else fp8._on(stream, tensor.device)


@contextlib.contextmanager
def options(**values):
    """Settings of this thread's products inside the block, any of OPTIONS by name (0: the plan's choice)."""
    lib = load()
    before = {}
    try:
        for name, value in values.items():
            old = _L()
            _check(lib.ffn_get_option(OPTIONS[name], ctypes.byref(old)), f"get_option({name})")
            _check(lib.ffn_set_option(OPTIONS[name], int(value)), f"set_option({name}={value})")
            before[name] = old.value
        yield
    finally:
        for name, value in before.items():
            lib.ffn_set_option(OPTIONS[name], value)


def plan_info() -> dict:
    """The plan of this thread's last product."""
    info = PlanInfo()
    _check(load().ffn_plan_info(ctypes.byref(info)), "ffn_plan_info")
    return info.as_dict()


def device_status(device=None):
    """(status, detail word) of the watchdog over every call on a CUDA device (default: the current one).

    Waits for the device.  ERR_DEVICE_TIMEOUT if, since the last query, a wait inside a kernel
    ran out (two seconds and more, where none should take a millisecond): that call's result is
    wrong.
    """
    if isinstance(device, int) and device < 0:
        raise ValueError(f"no such device: {device}")
    dev = torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        raise ValueError(f"{dev} is no CUDA device")
    if not torch.cuda.is_available():
        raise FfnError(ERR_CUDA, "ffn_device_status")
    word = ctypes.c_uint32()
    with torch.cuda.device(dev):
        st = load().ffn_device_status(ctypes.byref(word))
    return st, word.value


def linear(x, weight, bias=None, activation=None, residual=None, save: bool = False, out=None,
           out_dtype=None, stream=None):
    """act(x @ weight.T + bias) + residual: M x N in bf16 or fp32 (``out_dtype``: out's, or else bf16).

    x: M x K, weight: N x K, residual: M x N; bias: N values, bf16 or fp32.  With ``save`` returns
    (y, z), z being x @ weight.T + bias in bf16, which linear_backward() needs for an activation.
    ``out`` may be the residual itself, but not part of it nor over what else is read.
    """
    act = _choice(ACTIVATIONS, activation, "activation")
    with _stream(stream, x):
        return (_bind or _ops()).ffn_linear(x, weight, bias, act, residual, save, out, out_dtype)


def linear_backward(dy, x, weight, z=None, activation=None, bias: bool = False, grad_dtype=torch.bfloat16, stream=None):
    """Gradients of linear() from dy, the gradient of its result: (dx, dweight, dbias).

    dz = dy * act'(z) is rounded to bf16, in which the products take it; dx is bf16, dweight of
    grad_dtype (bf16 or fp32); both are always computed.  dbias, with ``bias``, is fp32 (else None).  The residual's gradient is
    dy itself.
    """
    act = _choice(ACTIVATIONS, activation, "activation")
    with _stream(stream, dy):
        return (_bind or _ops()).ffn_linear_backward(dy, x, weight, z, act, bias, grad_dtype)


def gated(x, w_gate, w_up, activation="silu", save=None, stream=None):
    """h = act(x @ w_gate.T) * (x @ w_up.T): M x F in bf16.

    With ``save`` returns (h, saved), what gated_backward() needs: "bf16" keeps both
    projections in bf16, as (g, u); "e4m3" in 8 bits, as (g codes, g scales, u codes, u scales),
    a quarter of the bytes of fp32 and half of bf16's.
    """
    act, how = _choice(ACTIVATIONS, activation, "activation"), _choice(SAVES, save, "save")
    with _stream(stream, x):
        out = (_bind or _ops()).ffn_gated(x, w_gate, w_up, act, how)
    return (out[0], out[1:]) if how else out


def gated_backward(dy, x, saved, w_gate, w_up, w_down, activation="silu", grad_dtype=torch.bfloat16, stream=None):
    """Gradients of y = h @ w_down.T with h = gated(x, w_gate, w_up), from dy: (dx, dw_gate, dw_up, dw_down).

    ``saved`` is what gated() saved; h is made again from it.  dg, du and h are rounded to bf16,
    in which the products take them.  All four gradients are always computed.
    """
    act = _choice(ACTIVATIONS, activation, "activation")
    with _stream(stream, dy):
        return (_bind or _ops()).ffn_gated_backward(dy, x, tuple(saved), w_gate, w_up, w_down, act, grad_dtype)
