"""Results written into the caller's tensors are known to autograd: the tensor's version rises, so that a
backward pass which saved it before refuses to use what is now in it."""
from __future__ import annotations

import pytest
import torch

from warp_specialized_tma_gb300 import ffn, fp8

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)


def rand(*shape):
    return torch.randn(*shape, device="cuda").to(bf)


def into_residual(t):
    ffn.linear(rand(16, 64), rand(t.shape[1], 64), residual=t, out=t)


def into_apart(t):
    ffn.linear(rand(16, 64), rand(t.shape[1], 64), out=t)


def into_gemm(t):
    fp8.gemm(*fp8.quantize(rand(16, 64)), *fp8.quantize(rand(t.shape[1], 64)), out=t)


def into_norm(t):
    fp8.rmsnorm(rand(16, t.shape[1]), rand(t.shape[1]), residual=t, out_h=t)


writers = pytest.mark.parametrize("write", [into_residual, into_apart, into_gemm, into_norm])


@writers
def test_a_saved_tensor_may_not_be_overwritten(write):
    x = torch.randn(16, 128, device="cuda", requires_grad=True)
    h = rand(16, 128)
    loss = (x * h).sum()  # saves h
    before = h._version
    write(h)
    assert h._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@writers
def test_a_view_counts_for_its_base(write):
    base = rand(16, 256)
    before = base._version
    write(base[:, :128])
    assert base._version == before + 1


@writers
def test_tensors_of_inference_mode_may_be_written(write):
    with torch.inference_mode():
        h = rand(16, 128)
        was = h.clone()
        write(h)
    write(h)
    assert not h.equal(was)


def test_operands_keep_their_version():
    x, w, b, r = rand(16, 64), rand(128, 64), rand(128), rand(16, 128)
    ts = (x, w, b, r)
    before = [t._version for t in ts]
    y, z = ffn.linear(x, w, b, "gelu", r, save=True)
    ffn.linear_backward(y, x, w, z, "gelu", bias=True)
    assert [t._version for t in ts] == before and y._version == z._version == 0
