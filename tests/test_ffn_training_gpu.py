"""The command's training, step by step against the same training in 64 bits: its first loss is that of its
data, its last that of its gradients' steps."""
from __future__ import annotations

import json

import pytest
import torch

from warp_specialized_tma_gb300 import feedforward

pytestmark = pytest.mark.gpu
bf = torch.bfloat16
T, C, F, STEPS, LR = 256, 128, 384, 3, 0.05


def exact_losses():
    """The losses before each step, and what the first one's roundings may change it by."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    held = lambda t: t.to(bf).double()  # noqa: E731
    masters = [t.double() for t in (rand(F, C) / C**0.5, rand(F, C) / C**0.5, rand(C, F) / F**0.5)]
    x, res = rand(T, C).to(bf).double(), rand(T, C).to(bf)
    target = (res + (rand(T, 16) @ rand(16, C) / 4).to(bf)).double()
    res, losses, off = res.double(), [], 0.0
    rms = lambda t: float(t.square().mean().sqrt())  # noqa: E731
    for _ in range(STEPS):
        wg, wu, wd = (held(m) for m in masters)
        g, u = x @ wg.T, x @ wu.T
        s = torch.sigmoid(g)
        h = g * s * u
        y = h @ wd.T + res
        d = y - target
        losses.append(float(d.square().mean()))
        # y, d and h are rounded to bf16, each value by at most 2^-8 of itself: d is off by `part`, and its
        # square's mean by twice the product of both at most
        part = 2.0**-8 * (rms(y) + rms(d) + rms(h @ wd.T))
        off = max(off, 2 * rms(d) * part + part**2)
        dh = d @ wd
        for m, grad in zip(masters, ((dh * u * (s + g * s * (1 - s))).T @ x, (dh * g * s).T @ x, d.T @ h)):
            m -= LR / T * grad
    return losses, off


@pytest.mark.parametrize("save", ["bf16", "e4m3"])
def test_the_command_trains_as_in_64_bits(save, capsys):
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    assert feedforward.main(["--tokens", str(T), "--width", str(C), "--hidden", str(F), "--steps", str(STEPS), "--lr", str(LR),
                             "--save", save]) == 0
    got = json.loads(capsys.readouterr().out.splitlines()[-1])
    want, off = exact_losses()
    assert abs(got["loss_first"] - want[0]) <= off
    # a gradient off by a share of its size (see test_gated_block: roundings of dg, du, h, g and u) changes a step's
    # effect on the loss by that share to first order; and as much again for what is of second order
    share = 2.0**-8 * 4 + (2.0**-4 if save == "e4m3" else 2.0**-8) * 2.4
    assert abs(got["loss_last"] - want[-1]) <= off + 2 * share * (want[0] - want[-1])
    # gradients of no effect, or of the other sign, would be found
    assert want[0] - want[-1] > off + 2 * share * (want[0] - want[-1])
