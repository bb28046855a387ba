"""8-bit operators of a pre-norm projection, over the C ABI of ``include/fp8_ops.h``.

    gemm                D = A @ B.T of two quantised matrices
    device_status       whether a product's watchdog ran out
    quantize            codes and scales of a matrix's rows
    quantize_columns    ... of its columns (a transposed result)
    quantize_both       ... of both, from one read
    rmsnorm             residual addition, root-mean-square norm, quantised output
    rmsnorm_backward    its gradients

A quantised matrix of R rows and K columns is a pair of tensors: ``codes``
(float8_e4m3fn, R x K, rows at a multiple of 16 bytes) and ``scales``
(float8_e8m0fnu, ceil(K / 512) x R x 4, contiguous): byte j of ``scales[i, r]`` is the
power-of-two scale of row r's block 4 i + j of 128 columns, and an element's value
is its code times its block's scale.  The quantisers here make rows that start
at multiples of 128 bytes.

Every function takes CUDA tensors, enqueues its work on ``stream`` (default: the
current stream of the tensors' device) and returns without waiting.  The work is
done by ``libfp8_ops.so``; ``_fp8_bind.so`` checks and marshals tensors, and the
handle's settings go through ctypes.  There is no fallback.  Nothing is recorded for
autograd: tensors that require a gradient are refused while gradients are
recorded, and rmsnorm_backward is called by name (as ``prenorm`` does).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfp8_ops.so")
BIND_PATH = os.path.join(PKG, "_fp8_bind.so")

# status codes (fp8_status)
OK = 0
ERR_INVALID_ARG = -1
ERR_ALIGNMENT = -2
ERR_NOT_PLANNED = -3
ERR_CUDA = -4
ERR_TENSORMAP = -5
ERR_DEVICE_TIMEOUT = -6
ERR_UNSUPPORTED = -7

# element types (fp8_type)
TYPES = {torch.bfloat16: 0, torch.float32: 1}

# options of the product (fp8_gemm_option)
OPTIONS = {
    "cta_group": 1,
    "transposed": 2,
    "width": 3,
    "split": 4,
    "watchdog_ns": 5,
    "fault_skip_load": 6,
    "raster_group": 7,
}

NORM_MAX_COLUMNS = 32768

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_SIGNATURES = {
    "fp8_strerror": (ctypes.c_char_p, [_I]),
    "fp8_version": (ctypes.c_char_p, []),
    "fp8_gemm_create": (_I, [_I, ctypes.POINTER(_P)]),
    "fp8_gemm_destroy": (_I, [_P]),
    "fp8_gemm_set_option": (_I, [_P, _I, _L]),
    "fp8_gemm_get_option": (_I, [_P, _I, ctypes.POINTER(_L)]),
    "fp8_gemm_check_problem": (_I, [_L] * 6 + [_I]),
    "fp8_gemm_plan": (_I, [_P] + [_L] * 6 + [_I]),
    "fp8_gemm_plan_info": (_I, [_P, _P]),
    "fp8_gemm_run": (_I, [_P] * 7),
    "fp8_gemm_workspace": (_I, [_P, ctypes.POINTER(_L)]),
    "fp8_gemm_run_in": (_I, [_P] * 7 + [_L, _P]),
    "fp8_gemm_device_status": (_I, [_P, ctypes.POINTER(ctypes.c_uint32)]),
    "fp8_quantize": (_I, [_P, _I, _L, _L, _L, _I, _P, _P, _I, _P, _L, _P, _P, _L, _P, _P]),
    "fp8_rmsnorm": (_I, [_P, _L, _P, _L, _P, _I, _L, _L, ctypes.c_float, _P, _L, _P, _L, _P, _P, _P]),
    "fp8_rmsnorm_backward_workspace": (_I, [_L, _L, ctypes.POINTER(_L)]),
    "fp8_rmsnorm_backward": (_I, [_P, _L, _P, _L, _P, _I, _P, _P, _L, _P, _L, _P, _L, _L, _P, _L, _P]),
}


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
        ("smem_bytes", ctypes.c_int32),
        ("regs_per_thread", ctypes.c_int32),
        ("cluster", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class Fp8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {load().fp8_strerror(status).decode()} (status {status})")


_lib = None
_lock = threading.Lock()


def load() -> ctypes.CDLL:
    """Loads libfp8_ops.so (raises if it was not built)."""
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
    return load().fp8_version().decode()


_bind = None


def _ops():
    """The compiled tensor entry points (raises if they were not built)."""
    global _bind
    if _bind is None:
        load()
        if not os.path.exists(BIND_PATH):
            raise ImportError(f"{BIND_PATH} is missing: build it with `python -m warp_specialized_tma_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("_fp8_bind", BIND_PATH)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fp8_bind", loader))
        loader.exec_module(mod)
        mod.set_error(Fp8Error)
        _bind = mod
    return _bind


def _check(st: int, what: str) -> None:
    if st != OK:
        raise Fp8Error(st, what)


def _on(stream, device):
    """Context in which `stream` (a torch stream or a raw handle) is the current one: what a call
    allocates then belongs to the stream that it runs on."""
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        if handle in (0, 1):  # the default stream (cudaStreamLegacy), of which torch makes no ExternalStream
            stream = torch.cuda.default_stream(device)
        else:
            stream = torch.cuda.ExternalStream(handle, device=device)
            if stream.cuda_stream != handle:
                raise ValueError(f"stream {handle:#x} is none that torch can run on")
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def empty_quantized(rows: int, cols: int, device="cuda"):
    """Uninitialised (codes, scales) for a rows x cols matrix, rows at multiples of 128 bytes."""
    codes = torch.empty_strided((rows, cols), (-(-cols // 128) * 128, 1), dtype=torch.float8_e4m3fn, device=device)
    return codes, torch.empty((-(-cols // 512), rows, 4), dtype=torch.float8_e8m0fnu, device=device)


# ------------------------------------------------------------------ product
def _status(handle):
    w = ctypes.c_uint32()
    st = load().fp8_gemm_device_status(handle, ctypes.byref(w))
    return st, w.value


class Gemm:
    """One handle of the product, for its options and its plan.

    ``Gemm(device=0, width=128, ...)`` takes any option of OPTIONS as a keyword.
    A call's workspace comes from torch's allocator for its stream, and from a
    graph's memory where the call is captured, so calls may overlap.
    """

    def __init__(self, device: int = -1, **options):
        h = _P()
        _check(load().fp8_gemm_create(int(device), ctypes.byref(h)), "fp8_gemm_create")
        self.h = h
        self.device = int(device) if device >= 0 else torch.cuda.current_device()
        for k, v in options.items():
            self.set_option(k, v)

    def set_option(self, name: str, value: int) -> None:
        _check(load().fp8_gemm_set_option(self.h, OPTIONS[name], int(value)), f"set_option({name}={value})")

    def get_option(self, name: str) -> int:
        v = _L()
        _check(load().fp8_gemm_get_option(self.h, OPTIONS[name], ctypes.byref(v)), f"get_option({name})")
        return v.value

    def plan(self, M, N, K, lda=None, ldb=None, ldd=None, out_dtype=torch.bfloat16) -> dict:
        pitch = -(-K // 128) * 128
        _check(load().fp8_gemm_plan(self.h, M, N, K, pitch if lda is None else lda, pitch if ldb is None else ldb,
                                    N if ldd is None else ldd, TYPES[out_dtype]), "fp8_gemm_plan")
        return self.info()

    def info(self) -> dict:
        """The plan of the last plan() or run()."""
        info = PlanInfo()
        _check(load().fp8_gemm_plan_info(self.h, ctypes.byref(info)), "fp8_gemm_plan_info")
        return info.as_dict()

    def run(self, a, a_scales, b, b_scales, out=None, out_dtype=torch.bfloat16, stream=None):
        """a @ b.T (asynchronous), planned first if this handle does not remember a plan for it."""
        if a.device.type == "cuda" and a.device.index != self.device:
            raise ValueError(f"tensors must be on cuda:{self.device}, the handle's device (got {a.device})")
        if stream is not None:
            with _on(stream, a.device):
                return self.run(a, a_scales, b, b_scales, out, out_dtype)
        return (_bind or _ops()).gemm(self.h.value, a, a_scales, b, b_scales, out, out_dtype)

    def device_status(self):
        """(status, detail word) of the watchdog over this handle's launches; waits for the device."""
        return _status(self.h)

    def close(self) -> None:
        if getattr(self, "h", None) is not None:
            load().fp8_gemm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


def gemm(a, a_scales, b, b_scales, out=None, out_dtype=torch.bfloat16, stream=None):
    """a @ b.T for quantised a (M x K) and b (N x K): bf16 or fp32, M x N, summed in fp32.

    Runs on a handle kept for the device.  A call's workspace comes from torch's
    allocator for its stream, and from a graph's memory where the call is
    captured: calls on different streams, and graphs, share none.  A wait inside the
    kernel that runs out is reported by device_status().
    """
    if stream is not None:
        with _on(stream, a.device):
            return gemm(a, a_scales, b, b_scales, out, out_dtype)
    return (_bind or _ops()).gemm(0, a, a_scales, b, b_scales, out, out_dtype)


def device_status(device=None):
    """(status, detail word) of the watchdog over every gemm() on a CUDA device (default: the current one).

    Waits for the device.  ERR_DEVICE_TIMEOUT if, since the last call, a wait inside a
    product ran out (two seconds and more, where none should take a millisecond): that
    call's result is wrong.
    """
    index = device
    if not isinstance(device, int):
        dev = torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError(f"{dev} is no CUDA device")
        index = torch.cuda.current_device() if dev.index is None else dev.index
    return _status(_P(_ops().kept_handle(index)))


# ------------------------------------------------------------------ quantiser
def _quantize(x, tile, rows, columns, row_factor, column_factor, stream):
    if stream is not None:
        with _on(stream, x.device):
            return (_bind or _ops()).quantize(x, tile, rows, columns, row_factor, column_factor)
    return (_bind or _ops()).quantize(x, tile, rows, columns, row_factor, column_factor)


def quantize(x, tile: bool = False, row_factor=None, column_factor=None, stream=None):
    """(codes, scales) of x's rows, with one scale per 128 columns (or, with ``tile``, per 128 x 128 tile).

    x: bf16 or fp32; each element is first multiplied by its row's factor (fp32)
    and its column's (bf16 or fp32), where given.
    """
    return _quantize(x, tile, True, False, row_factor, column_factor, stream)


def quantize_columns(x, tile: bool = False, row_factor=None, column_factor=None, stream=None):
    """(codes, scales) of x's transpose: C rows of R codes, with one scale per 128 rows of x."""
    return _quantize(x, tile, False, True, row_factor, column_factor, stream)


def quantize_both(x, tile: bool = False, row_factor=None, column_factor=None, stream=None):
    """quantize(x) + quantize_columns(x) from one read of x: (codes, scales, codes_t, scales_t)."""
    return _quantize(x, tile, True, True, row_factor, column_factor, stream)


# ------------------------------------------------------------------ norm
def rmsnorm(x, weight, residual=None, eps: float = 1e-6, out_h=None, stream=None):
    """h = x + residual, normalised by its root mean square, times weight, quantised along the rows.

    x, residual: bf16 matrices; weight: bf16 or fp32.  Returns (codes, scales, h,
    rstd): h is the updated residual stream in bf16 (x itself without a residual;
    written to ``out_h``, which may be x or residual but not part of them, where given), rstd the rows'
    1 / rms in fp32 for the backward pass.
    """
    if stream is not None:
        with _on(stream, x.device):
            return (_bind or _ops()).rmsnorm(x, weight, residual, eps, out_h)
    return (_bind or _ops()).rmsnorm(x, weight, residual, eps, out_h)


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None, stream=None):
    """Gradients of rmsnorm from dy, the gradient of its output: (dx, dweight).

    dx (bf16) is the gradient of both x and residual, with ``dresidual``, the
    gradient that reaches h directly, added; dweight is fp32.
    """
    if stream is not None:
        with _on(stream, dy.device):
            return (_bind or _ops()).rmsnorm_backward(dy, h, weight, rstd, dresidual)
    return (_bind or _ops()).rmsnorm_backward(dy, h, weight, rstd, dresidual)
