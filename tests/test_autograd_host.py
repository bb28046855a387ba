"""What autograd would lose without a word is refused: gradients and forward-mode tangents of operands.
No kernel runs here: a call that is not refused for its tangents goes on to ask for a CUDA device."""
from __future__ import annotations

import pytest
import torch
from torch.autograd import forward_ad

from warp_specialized_tma_gb300 import build as libbuild
from warp_specialized_tma_gb300 import ffn, fp8

bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()


def cpu(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


# calls by the operand that carries a tangent
CALLS = {
    "linear x": lambda d: ffn.linear(d(4, 8), cpu(16, 8)),
    "linear weight": lambda d: ffn.linear(cpu(4, 8), d(16, 8)),
    "linear bias": lambda d: ffn.linear(cpu(4, 8), cpu(16, 8), bias=d(16)),
    "linear residual": lambda d: ffn.linear(cpu(4, 8), cpu(16, 8), residual=d(4, 16)),
    "linear out": lambda d: ffn.linear(cpu(4, 8), cpu(16, 8), out=d(4, 16)),
    "linear_backward dy": lambda d: ffn.linear_backward(d(4, 16), cpu(4, 8), cpu(16, 8)),
    "linear_backward z": lambda d: ffn.linear_backward(cpu(4, 16), cpu(4, 8), cpu(16, 8), z=d(4, 16), activation="silu"),
    "gated w_up": lambda d: ffn.gated(cpu(4, 8), cpu(16, 8), d(16, 8)),
    "gated_backward w_down": lambda d: ffn.gated_backward(cpu(4, 8), cpu(4, 8), (cpu(4, 16), cpu(4, 16)), cpu(16, 8),
                                                          cpu(16, 8), d(8, 16)),
    "rmsnorm x": lambda d: fp8.rmsnorm(d(4, 8), cpu(8)),
    "quantize x": lambda d: fp8.quantize(d(4, 8)),
}
calls = pytest.mark.parametrize("call", CALLS.values(), ids=CALLS.keys())


def dual(*shape):
    return forward_ad.make_dual(cpu(*shape), torch.ones(*shape, dtype=bf))


@calls
def test_tangents_are_refused(call):
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            call(dual)
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
            call(dual)
        with pytest.raises(ValueError, match="CUDA device|one device"):
            call(lambda *shape: forward_ad.unpack_dual(dual(*shape)).primal)
    with pytest.raises(ValueError, match="CUDA device|one device"):
        call(cpu)


def test_a_function_with_a_jvp_may_call():
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            return ffn.linear(x, w)

        @staticmethod
        def jvp(ctx, dx, dw):
            raise AssertionError("not reached here")

    with forward_ad.dual_level(), pytest.raises(ValueError, match="CUDA device"):
        Linear.apply(dual(4, 8), cpu(16, 8))
