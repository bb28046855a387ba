"""8-bit operators of a pre-norm projection, over the C ABI of ``include/fp8_ops.h``.

    gemm                D = A @ B.T of two quantised matrices
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
current stream of the tensors' device) and returns without waiting.  Argument
marshalling only: the work is done by ``libfp8_ops.so``, and there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libfp8_ops.so")

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


def _check(st: int, what: str) -> None:
    if st != OK:
        raise Fp8Error(st, what)


def _device_of(first, *others):
    """The CUDA device that all tensors are on; raises otherwise."""
    dev = first.device
    if dev.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device (got {dev})")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors must be on one device ({dev} and {t.device})")
    return dev


def _ld(t, what: str) -> int:
    """Elements from one row of t to the next."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be a matrix with contiguous rows")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"{what}: its rows overlap")
    return ld


def _codes_ld(t, what: str) -> int:
    if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"{what} must be float8_e4m3fn (or its bytes)")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be a matrix with contiguous rows")
    if t.shape[1] == 0:
        return 0
    # a single row has no pitch that matters: any that the library accepts
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 16) * 16


def _need_scales(t, codes, what: str) -> None:
    if t.dtype not in (torch.float8_e8m0fnu, torch.uint8):
        raise TypeError(f"{what} must be float8_e8m0fnu (or its bytes)")
    if t.shape != (-(-codes.shape[1] // 512), codes.shape[0], 4) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous ceil(K / 512) x rows x 4 tensor")


class _Nothing:
    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_NOTHING = _Nothing()


def _place(stream, device):
    """(raw handle of the stream to use, context in which its outputs and workspace are allocated).

    Memory allocated for a call belongs to the stream that the call runs on, so
    the allocator does not hand it on while that stream still uses it.
    """
    if stream is None:
        ctx = _NOTHING if torch.cuda.current_device() == device.index else torch.cuda.device(device)
        return torch.cuda.current_stream(device).cuda_stream, ctx
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return stream.cuda_stream, torch.cuda.stream(stream)


def empty_quantized(rows: int, cols: int, device):
    """Uninitialised (codes, scales) for a rows x cols matrix, rows at multiples of 128 bytes."""
    pitch = -(-cols // 128) * 128
    codes = torch.empty((rows, pitch), dtype=torch.float8_e4m3fn, device=device)
    scales = torch.empty((-(-cols // 512), rows, 4), dtype=torch.float8_e8m0fnu, device=device)
    return (codes if pitch == cols else codes[:, :cols]), scales


# ------------------------------------------------------------------ product
class Gemm:
    """One handle of the product: plan a problem, run it on tensors.

    ``Gemm(device=0, width=128, ...)`` takes any option of OPTIONS as a keyword.
    Launches of one handle share its workspace: order them (one stream).
    """

    def __init__(self, device: int = -1, **options):
        h = _P()
        _check(load().fp8_gemm_create(int(device), ctypes.byref(h)), "fp8_gemm_create")
        self.h = h
        self.device = int(device) if device >= 0 else torch.cuda.current_device()
        self.shape = None
        for k, v in options.items():
            self.set_option(k, v)

    def set_option(self, name: str, value: int) -> None:
        _check(load().fp8_gemm_set_option(self.h, OPTIONS[name], int(value)), f"set_option({name}={value})")
        self.shape = None

    def get_option(self, name: str) -> int:
        v = _L()
        _check(load().fp8_gemm_get_option(self.h, OPTIONS[name], ctypes.byref(v)), f"get_option({name})")
        return v.value

    def plan(self, M, N, K, lda=None, ldb=None, ldd=None, out_dtype=torch.bfloat16) -> dict:
        lda = -(-K // 128) * 128 if lda is None else lda
        ldb = -(-K // 128) * 128 if ldb is None else ldb
        self._plan((M, N, K, lda, ldb, N if ldd is None else ldd, TYPES[out_dtype]))
        return self.info()

    def _plan(self, shape) -> None:
        self.shape = None
        _check(load().fp8_gemm_plan(self.h, *shape), "fp8_gemm_plan")
        self.shape = shape

    def info(self) -> dict:
        info = PlanInfo()
        _check(load().fp8_gemm_plan_info(self.h, ctypes.byref(info)), "fp8_gemm_plan_info")
        return info.as_dict()

    def run(self, a, a_scales, b, b_scales, out=None, out_dtype=torch.bfloat16, stream=None):
        """out = a @ b.T (asynchronous); plans the problem if the last one was another."""
        M, K = a.shape
        N = b.shape[0]
        if b.shape[1] != K:
            raise ValueError(f"a and b contract over {K} and {b.shape[1]} columns")
        dev = _device_of(a, a_scales, b, b_scales, out)
        if dev.index != self.device:
            raise ValueError(f"tensors must be on cuda:{self.device}, the handle's device (got {dev})")
        _need_scales(a_scales, a, "a_scales")
        _need_scales(b_scales, b, "b_scales")
        st, ctx = _place(stream, dev)
        if out is None:
            if out_dtype not in TYPES:
                raise TypeError("out_dtype must be bf16 or fp32")
            with ctx:
                out = torch.empty((M, N), dtype=out_dtype, device=dev)
        elif out.shape != (M, N):
            raise ValueError(f"out must be {M} x {N}")
        if out.dtype not in TYPES:
            raise TypeError("out must be bf16 or fp32")
        shape = (M, N, K, _codes_ld(a, "a"), _codes_ld(b, "b"), _ld(out, "out"), TYPES[out.dtype])
        if shape != self.shape:
            self._plan(shape)
        _check(load().fp8_gemm_run(self.h, a.data_ptr(), a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(),
                                   out.data_ptr(), st), "fp8_gemm_run")
        return out

    def device_status(self):
        """(status, detail word) of the device watchdog; synchronises the last stream."""
        w = ctypes.c_uint32()
        st = load().fp8_gemm_device_status(self.h, ctypes.byref(w))
        return st, w.value

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


_handles: dict = {}


def gemm(a, a_scales, b, b_scales, out=None, out_dtype=torch.bfloat16, stream=None):
    """a @ b.T for quantised a (M x K) and b (N x K): bf16 or fp32, M x N, summed in fp32.

    Runs on a handle kept for the device and stream, so calls on different
    streams share no workspace.
    """
    dev = _device_of(a)
    key = (dev.index, torch.cuda.current_stream(dev).cuda_stream if stream is None
           else int(getattr(stream, "cuda_stream", stream)))
    g = _handles.get(key)
    if g is None:
        g = _handles[key] = Gemm(dev.index)
    return g.run(a, a_scales, b, b_scales, out, out_dtype, stream)


# ------------------------------------------------------------------ quantiser
def _quantize(x, tile, rows, columns, row_factor, column_factor, stream):
    if x.dtype not in TYPES:
        raise TypeError("x must be bf16 or fp32")
    ldx = _ld(x, "x")
    R, C = x.shape
    dev = _device_of(x, row_factor, column_factor)
    if row_factor is not None and (row_factor.dtype != torch.float32 or row_factor.shape != (R,)
                                   or not row_factor.is_contiguous()):
        raise ValueError(f"row_factor must be a contiguous fp32 vector of {R}")
    if column_factor is not None and (column_factor.dtype not in TYPES or column_factor.shape != (C,)
                                      or not column_factor.is_contiguous()):
        raise ValueError(f"column_factor must be a contiguous bf16 or fp32 vector of {C}")
    out = ()
    q = s = qt = st = None
    sh, ctx = _place(stream, dev)
    with ctx:
        if rows:
            q, s = empty_quantized(R, C, dev)
            out += (q, s)
        if columns:
            qt, st = empty_quantized(C, R, dev)
            out += (qt, st)
        _check(load().fp8_quantize(
            x.data_ptr(), TYPES[x.dtype], ldx, R, C, int(tile),
            None if row_factor is None else row_factor.data_ptr(),
            None if column_factor is None else column_factor.data_ptr(),
            0 if column_factor is None else TYPES[column_factor.dtype],
            q.data_ptr() if rows else None, _pitch(C), s.data_ptr() if rows else None,
            qt.data_ptr() if columns else None, _pitch(R), st.data_ptr() if columns else None,
            sh), "fp8_quantize")
    return out


def _pitch(cols: int) -> int:
    return -(-cols // 128) * 128


def quantize(x, tile: bool = False, row_factor=None, column_factor=None, stream=None):
    """(codes, scales) of x's rows, with one scale per 128 columns (or, with ``tile``, per 128 x 128 tile).

    x: bf16 or fp32; each element is first multiplied by its row's and its column's
    factor, where given.
    """
    return _quantize(x, tile, True, False, row_factor, column_factor, stream)


def quantize_columns(x, tile: bool = False, row_factor=None, column_factor=None, stream=None):
    """(codes, scales) of x's transpose: C rows of R codes, with one scale per 128 rows of x."""
    return _quantize(x, tile, False, True, row_factor, column_factor, stream)


def quantize_both(x, tile: bool = False, row_factor=None, column_factor=None, stream=None):
    """quantize(x) + quantize_columns(x) from one read of x: (codes, scales, codes_t, scales_t)."""
    return _quantize(x, tile, True, True, row_factor, column_factor, stream)


# ------------------------------------------------------------------ norm
def _need_weight(weight, C: int) -> int:
    if weight.dtype not in TYPES or weight.shape != (C,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous bf16 or fp32 vector of {C}")
    return TYPES[weight.dtype]


def _need_bf16(t, shape, what: str) -> int:
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{what} must be bf16")
    if t.shape != shape:
        raise ValueError(f"{what} must be {tuple(shape)}")
    return _ld(t, what)


def rmsnorm(x, weight, residual=None, eps: float = 1e-6, out_h=None, stream=None):
    """h = x + residual, normalised by its root mean square, times weight, quantised along the rows.

    Returns (codes, scales, h, rstd): h is the updated residual stream in bf16 (x
    itself without a residual; written to ``out_h``, which may be x or residual,
    where given), rstd the rows' 1 / rms in fp32 for the backward pass.
    """
    if x.dim() != 2:
        raise ValueError("x must be a matrix")
    R, C = x.shape
    ldx = _need_bf16(x, (R, C), "x")
    wt = _need_weight(weight, C)
    dev = _device_of(x, weight, residual, out_h)
    ldr = ldh = 0
    h = x
    if residual is None and out_h is not None:
        raise ValueError("out_h needs a residual: without one, h is x")
    sh, ctx = _place(stream, dev)
    with ctx:
        if residual is not None:
            ldr = _need_bf16(residual, (R, C), "residual")
            h = torch.empty((R, C), dtype=torch.bfloat16, device=dev) if out_h is None else out_h
            ldh = _need_bf16(h, (R, C), "out_h")
        codes, scales = empty_quantized(R, C, dev)
        rstd = torch.empty((R,), dtype=torch.float32, device=dev)
        _check(load().fp8_rmsnorm(
            x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, weight.data_ptr(), wt, R, C,
            eps, None if residual is None else h.data_ptr(), ldh, codes.data_ptr(), _pitch(C), scales.data_ptr(),
            rstd.data_ptr(), sh), "fp8_rmsnorm")
    return codes, scales, h, rstd


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None, stream=None):
    """Gradients of rmsnorm from dy, the gradient of its output: (dx, dweight).

    dx (bf16) is the gradient of both x and residual, with ``dresidual``, the
    gradient that reaches h directly, added; dweight is fp32.
    """
    if dy.dim() != 2:
        raise ValueError("dy must be a matrix")
    R, C = dy.shape
    lddy = _need_bf16(dy, (R, C), "dy")
    ldh = _need_bf16(h, (R, C), "h")
    wt = _need_weight(weight, C)
    lddr = 0 if dresidual is None else _need_bf16(dresidual, (R, C), "dresidual")
    if rstd.dtype != torch.float32 or rstd.shape != (R,) or not rstd.is_contiguous():
        raise ValueError(f"rstd must be a contiguous fp32 vector of {R}")
    dev = _device_of(dy, h, weight, rstd, dresidual)
    st, ctx = _place(stream, dev)
    with ctx:
        dx = torch.empty((R, C), dtype=torch.bfloat16, device=dev)
        dw = torch.empty((C,), dtype=torch.float32, device=dev)
        need = _L()
        _check(load().fp8_rmsnorm_backward_workspace(R, C, ctypes.byref(need)), "fp8_rmsnorm_backward_workspace")
        work = torch.empty((need.value,), dtype=torch.uint8, device=dev)
        _check(load().fp8_rmsnorm_backward(
            dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), wt, rstd.data_ptr(),
            None if dresidual is None else dresidual.data_ptr(), lddr, dx.data_ptr(), C, dw.data_ptr(), R, C,
            work.data_ptr(), need.value, st), "fp8_rmsnorm_backward")
    return dx, dw
