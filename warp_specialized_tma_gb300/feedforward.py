"""A feed-forward block in bf16, served and trained with ffn's operators.

    y = (act(x @ w_gate.T) * (x @ w_up.T)) @ w_down.T + residual        GatedFeedForward
    y = act(x @ w_up.T + b_up) @ w_down.T + b_down + residual           FeedForward

Forward is two launches for a token or many.  Between the passes a gated block keeps its two
projections, in bf16 or in 8 bits (``save``), and the other one its pre-activation and its
hidden values; the backward passes return every gradient.

    python -m warp_specialized_tma_gb300.feedforward [--tokens 4096] [--width 2048] [--hidden 8192]
                                                     [--steps 20] [--save bf16|e4m3]

trains a gated block on random data against a fixed target, then times its steps and the
decoding of single tokens from a CUDA graph.
"""
from __future__ import annotations

import argparse
import json
import sys

import torch

from . import ffn


class GatedFeedForward:
    """w_gate, w_up: F x C; w_down: N x F; bf16.  ``save`` is how forward_train() keeps the projections: "bf16" or
    "e4m3", or None for a block that only serves."""

    def __init__(self, w_gate, w_up, w_down, activation="silu", save="bf16"):
        if w_gate.shape != w_up.shape or w_down.shape[1] != w_gate.shape[0]:
            raise ValueError("w_gate and w_up must be F x C, w_down N x F")
        ffn._choice(ffn.SAVES, save, "save")
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        self.activation, self.save = activation, save

    def forward(self, x, residual=None):
        """y alone, with nothing kept."""
        h = ffn.gated(x, self.w_gate, self.w_up, self.activation)
        return ffn.linear(h, self.w_down, residual=residual)

    def forward_train(self, x, residual=None):
        """(y, saved): saved is what backward() needs."""
        if self.save is None:
            raise ValueError("this block keeps nothing for a backward pass: save must be 'bf16' or 'e4m3'")
        h, kept = ffn.gated(x, self.w_gate, self.w_up, self.activation, save=self.save)
        return ffn.linear(h, self.w_down, residual=residual), (x, kept)

    def backward(self, dy, saved):
        """(dx, dw_gate, dw_up, dw_down); the residual's gradient is dy."""
        x, kept = saved
        return ffn.gated_backward(dy, x, kept, self.w_gate, self.w_up, self.w_down, self.activation)


class FeedForward:
    """w_up: F x C, w_down: N x F, bf16; biases of F and N values (bf16 or fp32), or None."""

    def __init__(self, w_up, w_down, b_up=None, b_down=None, activation="gelu"):
        if w_down.shape[1] != w_up.shape[0]:
            raise ValueError("w_up must be F x C, w_down N x F")
        self.w_up, self.w_down, self.b_up, self.b_down, self.activation = w_up, w_down, b_up, b_down, activation

    def forward(self, x, residual=None):
        """y alone, with nothing kept."""
        h = ffn.linear(x, self.w_up, self.b_up, self.activation)
        return ffn.linear(h, self.w_down, self.b_down, residual=residual)

    def forward_train(self, x, residual=None):
        """(y, saved): saved is what backward() needs."""
        h, z = ffn.linear(x, self.w_up, self.b_up, self.activation, save=True)
        return ffn.linear(h, self.w_down, self.b_down, residual=residual), (x, z, h)

    def backward(self, dy, saved):
        """(dx, dw_up, db_up, dw_down, db_down), biases' None where there are none; the residual's is dy."""
        x, z, h = saved
        dh, dw_down, db_down = ffn.linear_backward(dy, h, self.w_down, bias=self.b_down is not None)
        dx, dw_up, db_up = ffn.linear_backward(dh, x, self.w_up, z, self.activation, bias=self.b_up is not None)
        return dx, dw_up, db_up, dw_down, db_down


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
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.05)
    ap.add_argument("--save", choices=("bf16", "e4m3"), default="bf16")
    args = ap.parse_args(argv)
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    T, C, F = args.tokens, args.width, args.hidden
    masters = [rand(F, C) / C**0.5, rand(F, C) / C**0.5, rand(C, F) / F**0.5]
    block = GatedFeedForward(*(w.to(torch.bfloat16) for w in masters), save=args.save)
    x, res = rand(T, C).to(torch.bfloat16), rand(T, C).to(torch.bfloat16)
    target = res + (rand(T, 16) @ rand(16, C) / 4).to(torch.bfloat16)
    losses = []
    for _ in range(args.steps):
        y, saved = block.forward_train(x, res)
        dy = y - target
        losses.append(float(dy.float().square().mean()))
        grads = block.backward(dy, saved)[1:]
        for w, g in zip(masters, grads):
            w -= args.lr / T * g.float()
        block.w_gate, block.w_up, block.w_down = (w.to(torch.bfloat16) for w in masters)

    def step():
        y, saved = block.forward_train(x, res)
        block.backward(y, saved)

    one, one_res = x[:1].clone(), res[:1].clone()
    block.forward(one, one_res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(one, one_res)
    out = {"tokens": T, "width": C, "hidden": F, "save": args.save, "loss_first": losses[0], "loss_last": losses[-1],
           "forward_backward_ms": _event_ms(step, 20), "decode_us": 1e3 * _event_ms(graph.replay, 200)}
    print(json.dumps(out))
    return 0 if all(map(torch.isfinite, map(torch.tensor, losses))) and ffn.device_status()[0] == ffn.OK else 1


if __name__ == "__main__":
    sys.exit(main())
