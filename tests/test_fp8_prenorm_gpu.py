"""The 8-bit operators together: a pre-norm projection's forward and backward pass
against the same layer in 64 bits, and offsets past 32 bits.

Rounding to e4m3 moves each operand's elements by at most 2^-4 of their value (or half
the least step of their block), so an entry of a product of two quantised operands is
off by at most about 2^-3 of the sum of its terms' magnitudes, and typically by
2^-5 of their root of squares.  The whole outputs are held to 2^-4 of their norm: the
rounding of two operands to 3 bits has a root mean square of 2^-3 / sqrt(12) = 0.036
of a value at most for each, 0.051 together, and e4m3's other roundings are below."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_reference as ref
from warp_specialized_tma_gb300 import fp8
from warp_specialized_tma_gb300.prenorm import PreNormLinear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def off(got: torch.Tensor, want: np.ndarray) -> float:
    return float(np.linalg.norm(got.cpu().double().numpy() - want) / np.linalg.norm(want))


@pytest.mark.parametrize("tokens,width,out", [(1, 512, 768), (37, 1000, 520), (600, 512, 384)])
def test_prenorm_linear(tokens, width, out):
    gen = torch.Generator().manual_seed(tokens)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, res = rand(tokens, width).to(torch.bfloat16), rand(tokens, width).to(torch.bfloat16)
    g = (1 + 0.1 * rand(width)).to(torch.bfloat16)
    w = (rand(out, width) * 0.05).to(torch.bfloat16)
    dy, dh = rand(tokens, out).to(torch.bfloat16), rand(tokens, width).to(torch.bfloat16)
    layer = PreNormLinear(g.cuda(), w.cuda())
    y, h, saved = layer.forward(x.cuda(), res.cuda())
    dx, dnorm, dweight = layer.backward(dy.cuda(), saved, dh.cuda())

    hn = (x.float() + res.float()).to(torch.bfloat16).double().numpy()
    gn, wn, dyn, dhn = (t.double().numpy() for t in (g, w, dy, dh))
    n, rstd = ref.rmsnorm(hn, gn, 1e-6)
    assert np.array_equal(h.cpu().double().numpy(), hn)
    assert off(y, n @ wn.T) < 2.0**-4
    dn = dyn @ wn
    want_x, want_g = ref.rmsnorm_backward(dn, hn, gn, rstd, dhn)
    assert off(dweight, dyn.T @ n) < 2.0**-4
    assert off(dx, want_x) < 2.0**-4
    assert off(dnorm, want_g) < 2.0**-4


def test_prenorm_decode_from_a_graph():
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(1024, 1024, generator=gen, device="cuda") * 0.03).to(torch.bfloat16)
    layer = PreNormLinear(torch.ones(1024, device="cuda"), w)
    x = torch.randn(1, 1024, generator=gen, device="cuda").to(torch.bfloat16)
    res = torch.randn(1, 1024, generator=gen, device="cuda").to(torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, _ = layer.forward(x, res)
    for k in range(3):
        x.copy_(torch.randn(1, 1024, generator=gen, device="cuda"))
        graph.replay()
        want, want_h, _ = layer.forward(x, res)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(h, want_h)


def test_training_lowers_the_loss():
    from warp_specialized_tma_gb300 import prenorm
    assert prenorm.main(["--tokens", "512", "--width", "512", "--steps", "8"]) == 0


# ---------------------------------------------------------------- offsets past 32 bits
def test_gemm_output_past_4g_elements():
    M, N, K = 65600, 65536, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, sa = fp8.quantize(torch.randn(M, K, generator=gen, device="cuda"))
    b, sb = fp8.quantize(torch.randn(N, K, generator=gen, device="cuda"))
    d = fp8.gemm(a, sa, b, sb)
    last = slice(M - 200, M)
    want = fp8.gemm(a[last], sa[:, last].contiguous(), b, sb)
    assert torch.equal(d[last], want)
    assert torch.equal(d[:200], fp8.gemm(a[:200], sa[:, :200].contiguous(), b, sb))


def test_quantize_past_4g_elements():
    R, C = 65600, 65536
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x.normal_(generator=gen)
    q, s = fp8.quantize(x)
    last = slice(R - 64, R)
    q2, s2 = fp8.quantize(x[last])
    assert torch.equal(q[last].view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s[:, last].view(torch.uint8), s2.view(torch.uint8))
    del q
    qt, st = fp8.quantize_columns(x)
    # 65536 rows are whole blocks: the last 64 are a block of their own
    q2, s2 = fp8.quantize_columns(x[R - 64:])
    assert torch.equal(qt[:, R - 64:].view(torch.uint8), q2.view(torch.uint8))
    kb = (R - 64) // 128
    assert torch.equal(st[kb // 4, :, kb % 4].view(torch.uint8), s2[0, :, 0].view(torch.uint8))


def test_norm_rows_past_4g_elements_apart():
    C, ld = 1000, 2**30 + 8
    big = torch.zeros(4 * ld + C, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(5, C, generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn(5, C, generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randn(C, generator=gen, device="cuda")
    far = big.as_strided((5, C), (ld, 1))
    far.copy_(x)
    got, want = fp8.rmsnorm(far, w), fp8.rmsnorm(x, w)
    for one, two in zip(got, want):
        assert torch.equal(one.contiguous().view(torch.uint8), two.contiguous().view(torch.uint8))
    g1, g2 = fp8.rmsnorm_backward(dy, far, w, got[3]), fp8.rmsnorm_backward(dy, x, w, got[3])
    assert torch.equal(g1[0], g2[0]) and torch.equal(g1[1], g2[1])
