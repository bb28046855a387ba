"""A pre-norm projection in 8-bit floating point, served and trained with fp8's operators.

    h = x + residual
    y = (h / rms(h) * norm_weight) @ weight.T

``PreNormLinear`` keeps bf16 master weights and their quantised forms, laid out once
per update: the weight for the forward product and its transpose for the input
gradient, both from one read, with one scale per 128 x 128 tile.  The forward pass is
two launches (norm, product), for one token or many; the backward pass quantises
the output gradient both ways, recomputes the normed input into its transpose, and
takes the weight gradient with fp32 sums.

    python -m warp_specialized_tma_gb300.prenorm [--tokens 4096] [--width 4096] [--steps 20]

trains one on random data against a fixed target, then times its steps and the
decoding of single tokens from a CUDA graph.
"""
from __future__ import annotations

import argparse
import json
import sys

import torch

from . import fp8


class PreNormLinear:
    """norm_weight: bf16 or fp32, C values; weight: bf16, N x C."""

    def __init__(self, norm_weight, weight, eps: float = 1e-6):
        if weight.shape[1] != norm_weight.shape[0]:
            raise ValueError(f"weight must be N x {norm_weight.shape[0]}")
        self.norm_weight, self.weight, self.eps = norm_weight, weight, eps
        self.requantize()

    def requantize(self) -> None:
        """Lays the quantised weights out again after an update."""
        self.q, self.s, self.qt, self.st = fp8.quantize_both(self.weight, tile=True)

    def forward(self, x, residual=None):
        """(y, h, saved): saved is what backward() needs."""
        q, s, h, rstd = fp8.rmsnorm(x, self.norm_weight, residual, self.eps)
        return fp8.gemm(q, s, self.q, self.s), h, (h, rstd)

    def backward(self, dy, saved, dh=None):
        """(dx, dnorm_weight, dweight) from dy and dh, the gradients of y and h; dx is also the residual's."""
        h, rstd = saved
        dq, ds, dqt, dst = fp8.quantize_both(dy)
        dn = fp8.gemm(dq, ds, self.qt, self.st)
        nt, nst = fp8.quantize_columns(h, row_factor=rstd, column_factor=self.norm_weight)
        dweight = fp8.gemm(dqt, dst, nt, nst, out_dtype=torch.float32)
        dx, dnorm = fp8.rmsnorm_backward(dn, h, self.norm_weight, rstd, dh)
        return dx, dnorm, dweight


def _event_ms(fn, n: int) -> float:
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    a.record()
    for _ in range(n):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.3)
    args = ap.parse_args(argv)
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    C, T = args.width, args.tokens
    layer = PreNormLinear(torch.ones(C, device="cuda"), (rand(C, C) / C**0.5).to(torch.bfloat16))
    x, res = rand(T, C).to(torch.bfloat16), rand(T, C).to(torch.bfloat16)
    master = layer.weight.float()
    target = (rand(T, 64) @ rand(64, C) / 8).to(torch.bfloat16)
    losses = []
    for _ in range(args.steps):
        y, _, saved = layer.forward(x, res)
        dy = y - target
        losses.append(float(dy.float().square().mean()))
        _, dnorm, dweight = layer.backward(dy, saved)
        master -= args.lr / T * dweight
        layer.norm_weight -= args.lr / (T * C) * dnorm
        layer.weight = master.to(torch.bfloat16)
        layer.requantize()

    def step():
        y, _, saved = layer.forward(x, res)
        layer.backward(y, saved)

    one, one_res = x[:1].clone(), res[:1].clone()
    layer.forward(one, one_res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(one, one_res)
    out = {"tokens": T, "width": C, "loss_first": losses[0], "loss_last": losses[-1],
           "forward_backward_ms": _event_ms(step, 20), "decode_us": 1e3 * _event_ms(graph.replay, 200)}
    print(json.dumps(out))
    return 0 if losses[-1] < losses[0] and fp8.device_status()[0] == fp8.OK else 1


if __name__ == "__main__":
    sys.exit(main())
