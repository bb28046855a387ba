"""64-bit references of the 8-bit operators, on the CPU, written from the
definitions: no code of the package, exact arithmetic where the format allows it."""
from __future__ import annotations

import numpy as np
import torch


def scale_exponents(amax: np.ndarray) -> np.ndarray:
    """Biased exponent of the least power of two s >= 2^-127 with amax / s <= 448."""
    amax = np.asarray(amax, np.float64)
    e = np.full(amax.shape, -127.0)
    pos = amax > 0
    e[pos] = np.maximum(np.ceil(np.log2(amax[pos] / 448.0)), -127.0)
    up = pos & (amax > 448.0 * np.exp2(e))  # log2's own rounding
    e[up] += 1
    down = pos & (e > -127) & (amax <= 448.0 * np.exp2(e - 1))
    e[down] -= 1
    return e + 127


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even, of values at most 448 in magnitude; NaN stays."""
    a = np.abs(v)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0)
    step = np.exp2(e - 3)
    return np.rint(v / step) * step


def block_amax(y: np.ndarray, tile: bool) -> np.ndarray:
    """R x ceil(C / 128) maxima of the finite magnitudes of y's row blocks (or of its tiles)."""
    R, C = y.shape
    kb, rb = -(-C // 128), -(-R // 128)
    full = np.zeros((rb * 128, kb * 128))
    full[:R, :C] = np.where(np.isfinite(y), np.abs(y), 0.0)
    m = full.reshape(rb * 128, kb, 128).max(2)
    if tile:
        m = np.repeat(m.reshape(rb, 128, kb).max(1), 128, 0)
    return m[:R]


def quantize(y: np.ndarray, tile: bool = False):
    """(code values, R x ceil(C / 128) biased exponents) of y's rows, in 64 bits."""
    y = np.asarray(y, np.float64)
    e = scale_exponents(block_amax(y, tile))
    s = np.repeat(np.exp2(e - 127), 128, 1)[:, : y.shape[1]]
    v = np.where(np.isinf(y), np.nan, y) / s
    return e4m3_round(v), e


def scale_bytes(scales: torch.Tensor, K: int):
    """(R x ceil(K / 128) bytes, padding bytes) of a packed scale tensor."""
    b = scales.view(torch.uint8).cpu().numpy()
    kt, R, _ = b.shape
    flat = b.transpose(1, 0, 2).reshape(R, kt * 4)
    kb = -(-K // 128)
    return flat[:, :kb].astype(np.float64), flat[:, kb:]


def values(codes: torch.Tensor, scales: torch.Tensor) -> np.ndarray:
    """The elements a quantised matrix stands for."""
    K = codes.shape[1]
    e, _ = scale_bytes(scales, K)
    return codes.cpu().float().numpy().astype(np.float64) * np.repeat(np.exp2(e - 127), 128, 1)[:, :K]


def pack_scales(e: np.ndarray) -> torch.Tensor:
    """R x ceil(K / 128) biased exponents -> the packed scale tensor."""
    R, kb = e.shape
    kt = -(-kb // 4)
    full = np.full((R, kt * 4), 127, np.uint8)
    full[:, :kb] = e
    return torch.from_numpy(full.reshape(R, kt, 4).transpose(1, 0, 2).copy()).view(torch.float8_e8m0fnu)


def rmsnorm(h: np.ndarray, w: np.ndarray, eps: float):
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_backward(dy, h, w, rstd, dres=None):
    n = h * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    return (dx if dres is None else dx + dres), (dy * n).sum(0)
