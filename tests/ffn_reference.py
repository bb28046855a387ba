"""64-bit references of the feed-forward operators, on the CPU, written from the definitions,
and what their fp32 kernels may be off by."""
from __future__ import annotations

import math

import numpy as np
import torch

import fp8_reference as fp8ref

HALF_STEP = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}

# An MMA adds 16 products to the accumulator; each such addition loses at most a unit of the
# accumulator's last place (2^-23 of it), which is at most the sum of magnitudes.  Pieces that
# meet, a bias and a residual add a few more; 16 stands for them.
def sum_error(K: int) -> float:
    return (math.ceil(K / 16) + 16) * 2.0**-23


# The activations' fp32 arithmetic: some ten roundings, exp2 and 1/x to 2 units, the argument of
# exp to 2^-22 of itself.  Up to an argument of 32 that is 2^-17 of the result.  Beyond it the result
# and the kernel's both are below |z| exp(-32), which is 2^-46 |z| (32 / ln 2 = 46.2): with an argument
# of 88, the last before the result is 0, 2^-22 of it is 2.1e-5 of the result.
ACT_ERROR = 2.0**-17


def act_error(z, y):
    return ACT_ERROR * y.abs() + 2.0**-46 * z.abs()


def act(name, z):
    if name is None:
        return z.clone()
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)))


def slope(name, z):
    if name is None:
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    if name == "gelu":
        return torch.special.erfc(-z / math.sqrt(2)) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z**3))
    return (1 + t) / 2 + z * (1 - t * t) / 2 * a * (1 + 3 * 0.044715 * z * z)


def product(a, b):
    """a @ b.T in 64 bits, and the same of magnitudes."""
    a, b = a.double(), b.double()
    return a @ b.T, a.abs() @ b.abs().T


def linear(x, w, bias=None, activation=None, residual=None):
    """(y, z, bound of y, bound of z), before the results' rounding."""
    z, mag = product(x, w)
    ez = sum_error(x.shape[1]) * mag
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0**-22 * (mag + bias.double().abs())
    y = act(activation, z)
    # |act'| is at most 1.13
    ey = 1.13 * ez + (act_error(z, y) if activation else 0)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0**-23 * y.abs()
    return y, z, ey, ez


def gated(x, wg, wu, activation):
    """(h, g, u, bounds of the three)."""
    g, mg = product(x, wg)
    u, mu = product(x, wu)
    eg, eu = sum_error(x.shape[1]) * mg, sum_error(x.shape[1]) * mu
    a = act(activation, g)
    ea = 1.13 * eg + act_error(g, a)
    h = a * u
    return h, g, u, ea * u.abs() + eu * a.abs() + ea * eu + 2.0**-23 * h.abs(), eg, eu


def close(got, want, bound, dtype=torch.bfloat16):
    """Whether `got`, rounded once to dtype, is `want` to within `bound` before the rounding."""
    got, want = got.double().cpu(), want.double()
    limit = bound + HALF_STEP[dtype] * (want.abs() + bound)
    same = torch.isnan(got) & torch.isnan(want) | (got == want)
    return bool((same | ((got - want).abs() <= limit)).all())


def close_rms(got, want, dtype=torch.bfloat16, extra=0.0):
    """Gradients whose operands were rounded to bf16 on the way, some of them to the other side than
    in the reference: off by the result's own rounding (each value by at most half a step, so their
    root mean square too) and by `extra` of the root mean square."""
    got, want = got.double().cpu(), want.double()
    if want.numel() == 0:
        return got.shape == want.shape
    return float((got - want).norm()) <= (HALF_STEP[dtype] + extra) * float(want.norm()) + 1e-30


def checkpoint(v):
    """What v stands for once it is held in 8 bits with a scale per row and block of 128."""
    codes, e = fp8ref.quantize(v.numpy())
    return torch.from_numpy(codes * np.repeat(np.exp2(e - 127), 128, 1)[:, : v.shape[1]])


def bf16(v):
    return v.to(torch.bfloat16).double()


def gated_backward(dy, x, g, u, wg, wu, wd, activation):
    """(dx, dw_gate, dw_up, dw_down) with dg, du and h in bf16, as the operator defines them."""
    dy, x, g, u, wg, wu, wd = (t.double() for t in (dy, x, g, u, wg, wu, wd))
    dh = dy @ wd
    dg, du, h = bf16(dh * u * slope(activation, g)), bf16(dh * act(activation, g)), bf16(act(activation, g) * u)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ h


def linear_backward(dy, x, w, z, activation):
    """(dx, dweight, dbias) with dz in bf16 for the products."""
    dz = dy.double() * (slope(activation, z.double()) if activation else 1.0)
    held = bf16(dz)
    return held @ w.double(), held.T @ x.double(), dz.sum(0)
