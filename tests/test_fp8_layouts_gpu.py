"""The 8-bit operators on rows that lie differently from one array to the next, in place, and in
every way that the kernels share rows out; long sums in 32 bits.  References in 64 bits on the
CPU, tolerances as in test_fp8_gpu.py."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import fp8_reference as ref
from test_fp8_gpu import U, check_near, check_quantized, norm_inputs, norm_rel, spread_matrix
from warp_specialized_tma_gb300 import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


class Placed:
    """A matrix whose rows are `extra` elements further apart than long, `first` into a buffer of sevens."""

    def __init__(self, rows: torch.Tensor, extra: int, first: int):
        R, C = rows.shape
        self.buf = torch.full(((R + 1) * (C + extra) + first,), 7.0, dtype=rows.dtype, device="cuda")
        self.view = self.buf.as_strided((R, C), (C + extra, 1), first)
        self.view.copy_(rows)

    def rest_is_untouched(self) -> bool:
        kept = self.view.clone()
        self.view.fill_(7.0)
        rest = bool((self.buf == 7.0).all())
        self.view.copy_(kept)
        return rest


def ptr(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------- norm
# a row to a warp with 1, 2 and 4 vectors of 8 columns a lane, to a CTA with 1, 2 and 4
# a thread, and as wide as rows may be
FORWARD = [(400, 75), (400, 301), (400, 901), (400, 1501), (400, 3001), (400, 6634), (5, 700), (3, 32765)]


@pytest.mark.parametrize("out", ["own", "x", "residual"])
@pytest.mark.parametrize("shape", FORWARD, ids=lambda s: "x".join(map(str, s)))
def test_rmsnorm_rows_that_lie_differently(shape, out):
    R, C = shape
    x, res, w = norm_inputs(R, C, R + 3 * C, torch.float32, True)
    px, pr = Placed(x, 5, 3), Placed(res, 8, 1)
    ph = {"own": Placed(torch.zeros_like(x), 3, 2), "x": px, "residual": pr}[out]
    q, s, h, rstd = fp8.rmsnorm(px.view, w.cuda(), residual=pr.view, eps=1e-5, out_h=ph.view)
    kept = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(h.cpu(), kept) and h.data_ptr() == ph.view.data_ptr()
    assert px.rest_is_untouched() and pr.rest_is_untouched() and ph.rest_is_untouched()
    y, want = ref.rmsnorm(kept.double().numpy(), w.double().numpy(), 1e-5)
    rel = norm_rel(C)
    assert (np.abs(rstd.cpu().double().numpy() - want) <= rel * want).all()
    check_near(q, s, y, rel)


@pytest.mark.parametrize("shape", FORWARD, ids=lambda s: "x".join(map(str, s)))
def test_rmsnorm_without_residual_at_an_offset(shape):
    R, C = shape
    x, _, w = norm_inputs(R, C, R + 5 * C, torch.bfloat16, False)
    q, s, _, rstd = fp8.rmsnorm(Placed(x, 3, 5).view, w.cuda(), eps=1e-5)
    y, want = ref.rmsnorm(x.double().numpy(), w.double().numpy(), 1e-5)
    assert (np.abs(rstd.cpu().double().numpy() - want) <= norm_rel(C) * want).all()
    check_near(q, s, y, norm_rel(C))


def test_rmsnorm_refuses_rows_written_over_part_of_rows_read():
    C = 300
    buf = torch.zeros(40, 2 * C + 8, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(C, device="cuda")
    x, apart = buf[:20, :C], buf[:20, C:2 * C]  # rows between rows: apart
    res = torch.zeros(20, C, dtype=torch.bfloat16, device="cuda")
    fp8.rmsnorm(x, w, residual=res, out_h=apart)
    for over in (buf[:20, 1:C + 1], buf[1:21, :C], buf[:40:2, :C]):
        with pytest.raises(ValueError, match="out_h lies over"):
            fp8.rmsnorm(x, w, residual=res, out_h=over)
        with pytest.raises(ValueError, match="out_h lies over"):
            fp8.rmsnorm(res, w, residual=x, out_h=over)


# ---------------------------------------------------------------- norm gradient
# groups of a CTA's threads, a CTA's rows with 1, 2 and 4 vectors a thread through the ring, and
# rows beyond it; several rows to each
BACKWARD = [(6000, 75), (3000, 901), (1000, 4001), (700, 4500), (500, 6634), (470, 9001), (500, 16387), (400, 20001),
            (320, 24576)]


def backward_inputs(R, C, residual):
    h, _, w = norm_inputs(R, C, R * C + 5, torch.float32, False)
    gen = torch.Generator().manual_seed(R * C + 6)
    dy = (torch.randn(R, C, generator=gen) * 0.01).to(torch.bfloat16)
    dres = (torch.randn(R, C, generator=gen) * 0.01).to(torch.bfloat16) if residual else None
    rstd = (1.0 / (h.double().square().mean(1) + 1e-6).sqrt()).float()
    return dy, h, w, rstd, dres


def check_backward(dx, dw, dy, h, w, rstd, dres):
    R, C = h.shape
    hn, wn, dyn, rn = (t.double().numpy() for t in (h, w, dy, rstd))
    want, want_w = ref.rmsnorm_backward(dyn, hn, wn, rn, None if dres is None else dres.double().numpy())
    n, g = hn * rn[:, None], dyn * wn
    size = rn[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    tol = 2.0**-8 * np.abs(want) + (C + 16) * 2 * U * size
    assert (np.abs(dx.cpu().double().numpy() - want) <= tol).all()
    assert (np.abs(dw.cpu().double().numpy() - want_w) <= (R + 16) * 2 * U * np.abs(dyn * n).sum(0)).all()


def backward_into(dx, dy, h, w, rstd, dres):
    """fp8_rmsnorm_backward with a dx of the caller's; returns (status, dweight)."""
    lib, (R, C) = fp8.load(), h.shape
    need = ctypes.c_int64()
    assert lib.fp8_rmsnorm_backward_workspace(R, C, ctypes.byref(need)) == fp8.OK
    work, dw = torch.empty(need.value, dtype=torch.uint8, device="cuda"), torch.empty(C, device="cuda")
    st = lib.fp8_rmsnorm_backward(ptr(dy), dy.stride(0), ptr(h), h.stride(0), ptr(w), fp8.TYPES[w.dtype], ptr(rstd),
                                  ptr(dres), 0 if dres is None else dres.stride(0), ptr(dx), dx.stride(0), ptr(dw), R, C,
                                  ptr(work), need.value, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return st, dw


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("shape", BACKWARD, ids=lambda s: "x".join(map(str, s)))
def test_rmsnorm_backward_rows_that_lie_differently(shape, residual):
    dy, h, w, rstd, dres = backward_inputs(*shape, residual)
    py, ph = Placed(dy, 3, 1), Placed(h, 8, 5)
    pr = Placed(dres, 1, 2) if residual else None
    px = Placed(torch.zeros_like(dy), 7, 3)
    wg, rg = w.cuda(), rstd.cuda()
    dx, dw = fp8.rmsnorm_backward(py.view, ph.view, wg, rg, pr.view if residual else None)
    check_backward(dx, dw, dy, h, w, rstd, dres)
    st, dw2 = backward_into(px.view, py.view, ph.view, wg, rg, pr.view if residual else None)
    assert st == fp8.OK and torch.equal(px.view, dx) and torch.equal(dw2, dw)
    assert px.rest_is_untouched()


@pytest.mark.parametrize("shape", BACKWARD, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("extra,first", [(0, 0), (3, 1)], ids=["contiguous", "placed"])
def test_rmsnorm_backward_in_place(shape, extra, first):
    dy, h, w, rstd, dres = backward_inputs(*shape, True)
    wg, rg = w.cuda(), rstd.cuda()
    for which in (0, 1):
        py, ph, pr = Placed(dy, extra, first), Placed(h, 0, 0), Placed(dres, extra, first)
        px = (py, pr)[which]
        st, dw = backward_into(px.view, py.view, ph.view, wg, rg, pr.view)
        assert st == fp8.OK and px.rest_is_untouched()
        check_backward(px.view, dw, dy, h, w, rstd, dres)


def test_rmsnorm_backward_refuses_rows_written_over_part_of_rows_read():
    dy, h, w, rstd, dres = (t.cuda() for t in backward_inputs(20, 300, True))
    for k in range(3):
        given = [dy, h, dres]
        buf = torch.zeros(30 * 300, dtype=torch.bfloat16, device="cuda")
        given[k] = buf[:6000].view(20, 300)
        for over in (buf[1:6001].view(20, 300), buf[300:6300].view(20, 300)):
            assert backward_into(over, given[0], given[1], w, rstd, given[2])[0] == fp8.ERR_INVALID_ARG


# ---------------------------------------------------------------- quantiser
@pytest.mark.parametrize("shape", [(300, 1001), (129, 640), (700, 5999)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("extra,first", [(0, 0), (3, 1), (4, 2), (8, 8)])
def test_quantize_placed_with_factors(shape, extra, first):
    R, C = shape
    gen = torch.Generator().manual_seed(R + C)
    x = torch.randn(R, C, generator=gen).to(torch.bfloat16)
    f, w = torch.rand(R, generator=gen) + 0.1, torch.randn(C, generator=gen).to(torch.bfloat16)
    y = x.double().numpy() * f.double().numpy()[:, None] * w.double().numpy()
    q, s, qt, st = fp8.quantize_both(Placed(x, extra, first).view, row_factor=f.cuda(), column_factor=w.cuda())
    check_near(q, s, y, 4 * U)
    check_near(qt, st, y.T, 4 * U)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tile", [False, True], ids=["rows", "tiles"])
@pytest.mark.parametrize("extra,first", [(3, 1), (2, 6), (1, 7)])
def test_quantize_placed(extra, first, tile, dtype):
    x = spread_matrix(400, 1001, extra, dtype)
    q, s, qt, st = fp8.quantize_both(Placed(x, extra, first).view, tile=tile)
    check_quantized(q, s, x.double().numpy(), tile)
    check_quantized(qt, st, x.double().numpy().T, tile)


# ---------------------------------------------------------------- long sums
@pytest.mark.parametrize("options", [{}, {"cta_group": 1, "width": 192}, {"cta_group": 2, "width": 192, "split": 0}],
                         ids=["planned", "one-sm", "pairs"])
def test_gemm_long_sums_are_as_exact_as_short_ones(options):
    # The accumulator takes 4096 products, 32 at a time, and the sums of 8 such segments are
    # added in fp32: 136 additions in a row, each off by a unit in the last place (2 U of the
    # sum) at most, where one accumulator would take 1024.  As independent errors they come to
    # 2 U sqrt(136) = 1.4e-6 of the sum, root of mean squares.
    M, N, K = 256, 384, 32768
    gen = torch.Generator(device="cuda").manual_seed(12)
    a, sa = fp8.quantize(torch.randn(M, K, generator=gen, device="cuda") * 1e-3)
    b, sb = fp8.quantize(torch.randn(N, K, generator=gen, device="cuda"))
    want = ref.values(a, sa) @ ref.values(b, sb).T
    with fp8.Gemm(0, **options) as g:
        d = g.run(a, sa, b, sb, out_dtype=torch.float32)
    off = np.linalg.norm(d.cpu().double().numpy() - want) / np.linalg.norm(want)
    assert off <= 2 * U * np.sqrt(4096 / 32 + K / 4096)
