"""The feed-forward operators run together, as feedforward does: served, trained, captured, and their
gradients against the formula's and against differences of the 64-bit loss."""
from __future__ import annotations

import pytest
import torch

import ffn_reference as ref
from warp_specialized_tma_gb300 import feedforward, ffn

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)
    yield
    assert ffn.device_status() == (ffn.OK, 0)


def randn(*shape, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(bf)


def gated_weights(C, F, N):
    return randn(F, C, seed=1, scale=C**-0.5), randn(F, C, seed=2, scale=C**-0.5), randn(N, F, seed=3, scale=F**-0.5)


def directions(t, seed):
    return torch.randn(t.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("T,C,F", [(1, 136, 200), (70, 96, 257), (300, 264, 520)])
@pytest.mark.parametrize("save", ["bf16", "e4m3"])
def test_gated_block(T, C, F, save):
    wg, wu, wd = gated_weights(C, F, C)
    x, r, dy = randn(T, C, seed=4), randn(T, C, seed=5), randn(T, C, seed=6)
    block = feedforward.GatedFeedForward(wg.cuda(), wu.cuda(), wd.cuda(), save=save)
    y, saved = block.forward_train(x.cuda(), r.cuda())
    served = block.forward(x.cuda(), r.cuda())
    h, g, u, *_ = ref.gated(x, wg, wu, "silu")
    want = ref.bf16(h) @ wd.double().T + r.double()
    # some of h round to the other side, by 2^-7 of their value: fewer than one in sixty of a row
    for got in (y, served):
        assert ref.close_rms(got, want, extra=2.0**-10)
    grads = block.backward(dy.cuda(), saved)
    gs, us = (ref.bf16(g), ref.bf16(u)) if save == "bf16" else (ref.checkpoint(g), ref.checkpoint(u))
    formula = ref.gated_backward(dy, x, gs, us, wg, wu, wd, "silu")
    # some of g and u round to the other side, by a step: 2^-7 of few bf16, 2^-3 of few e4m3
    for a, b in zip(grads, formula):
        assert ref.close_rms(a, b, extra=2.0**-9)

    def loss(x, wg, wu, wd):
        return float(((ref.act("silu", x @ wg.T) * (x @ wu.T)) @ wd.T * dy.double()).sum())

    args = [t.double() for t in (x, wg, wu, wd)]
    # the gradient differs from the formula's of unrounded values by the roundings of its operands:
    # at most 2^-8 each of dg (du, h), of g and of u (which the slope turns into 1.2 of it), and of the
    # result; in 8 bits 2^-4 for g and u
    tol = 2.0**-8 * 4 + (2.0**-4 if save == "e4m3" else 2.0**-8) * 2.4
    for i, grad in enumerate(grads):
        v, eps = directions(args[i], 10 + i), 1e-4
        moved = [[a + s * eps * v if j == i else a for j, a in enumerate(args)] for s in (1, -1)]
        num = (loss(*moved[0]) - loss(*moved[1])) / (2 * eps)
        assert abs(num - float((grad.cpu().double() * v).sum())) <= tol * float(grad.double().norm()) * float(v.norm())


@pytest.mark.parametrize("T,C,F,N", [(1, 136, 200, 136), (70, 96, 257, 40), (300, 264, 520, 264)])
@pytest.mark.parametrize("activation", ["gelu", "relu"])
@pytest.mark.parametrize("bias", [torch.float32, bf, None])
def test_block_with_biases(T, C, F, N, activation, bias):
    wu, wd = randn(F, C, seed=1, scale=C**-0.5), randn(N, F, seed=2, scale=F**-0.5)
    bu, bd = (None, None) if bias is None else (randn(F, seed=3).to(bias), randn(N, seed=4).to(bias))
    x, r, dy = randn(T, C, seed=5), randn(T, N, seed=6), randn(T, N, seed=7)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    block = feedforward.FeedForward(c(wu), c(wd), c(bu), c(bd), activation)
    y, saved = block.forward_train(c(x), c(r))
    assert y.equal(block.forward(c(x), c(r)))
    dx, dwu, dbu, dwd, dbd = block.backward(c(dy), saved)
    assert (dbu is None) == (dbd is None) == (bias is None)

    def forward(x, wu, wd, bu, bd):
        z = x @ wu.T + (0 if bu is None else bu)
        return ref.act(activation, z) @ wd.T + (0 if bd is None else bd) + r.double()

    args = [None if t is None else t.double() for t in (x, wu, wd, bu, bd)]
    want = forward(*args)
    assert ref.close_rms(y, want, extra=2.0**-8)  # h's rounding
    grads = (dx, dwu, dwd, dbu, dbd)
    # roundings on the way: h or z, dh, dz, and the result's; where a relu's z is within its rounding
    # of 0 the slope is another's
    tol = 2.0**-8 * 5
    for i, grad in enumerate(grads):
        if grad is None:
            continue
        v, eps = directions(args[i], 20 + i), 1e-5
        moved = [[a + s * eps * v if j == i else a for j, a in enumerate(args)] for s in (1, -1)]
        num = float(((forward(*moved[0]) - forward(*moved[1])) * dy.double()).sum()) / (2 * eps)
        assert abs(num - float((grad.cpu().double() * v).sum())) <= tol * float(grad.double().norm()) * float(v.norm())


def test_tokens_decoded_from_a_graph_are_the_prompts():
    C, F = 256, 520
    wg, wu, wd = (w.cuda() for w in gated_weights(C, F, C))
    block = feedforward.GatedFeedForward(wg, wu, wd)
    x, r = randn(9, C, seed=4).cuda(), randn(9, C, seed=5).cuda()
    one, res = x[:1].clone(), r[:1].clone()
    block.forward(one, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.forward(one, res)
    whole = block.forward(x, r)
    for i in range(9):
        one.copy_(x[i:i + 1])
        res.copy_(r[i:i + 1])
        graph.replay()
        # the same values, summed in another order and h rounded: a step of bf16 now and then
        assert ref.close_rms(y, whole[i:i + 1].cpu(), extra=2.0**-8)


@pytest.mark.parametrize("save", ["bf16", "e4m3"])
def test_the_command_runs(save, capsys):
    assert feedforward.main(["--tokens", "256", "--width", "128", "--hidden", "384", "--steps", "3", "--save", save]) == 0
    assert '"decode_us"' in capsys.readouterr().out
