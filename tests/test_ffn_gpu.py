"""The feed-forward operators on the GPU against 64-bit references (ffn_reference): every kernel
variant, types, odd sizes, layouts, empty sums, values that are not finite, streams, graphs, workspaces
and launches that give up.  Integer operands whose sums fp32 holds must give the reference's bits."""
from __future__ import annotations

import ctypes
import itertools

import pytest
import torch

import ffn_reference as ref
import fp8_reference as fp8ref
from warp_specialized_tma_gb300 import ffn, fp8

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


def ints(*shape, seed=0, top=2):
    return torch.randint(-top, top + 1, shape, generator=torch.Generator().manual_seed(seed)).to(bf)


def gpu(*ts):
    out = [None if t is None else t.cuda() for t in ts]
    return out if len(out) > 1 else out[0]


# one SM and pairs, either side, whole tiles, tiles split through global memory and among clusters
VARIANTS = {
    "one": dict(cta_group=1, transposed=1, split=0),
    "pair": dict(cta_group=2, transposed=1, split=0),
    "one-t": dict(cta_group=1, transposed=2, split=0),
    "pair-t": dict(cta_group=2, transposed=2, split=0),
    "ranges": dict(cta_group=1, transposed=1, split=2),
    "ranges-t": dict(cta_group=1, transposed=2, split=2),
    "pair-ranges": dict(cta_group=2, transposed=1, split=2),
    "pair-ranges-t": dict(cta_group=2, transposed=2, split=2),
    "clusters": dict(cta_group=1, transposed=1, split=1),
    "clusters-t": dict(cta_group=1, transposed=2, split=1),
    "auto": dict(),
}
variants = pytest.mark.parametrize("variant", VARIANTS.values(), ids=VARIANTS.keys())

# a gradient's products one after the other, in each of these, or in one launch
GRADIENTS = {k: dict(v, together=2, stream=2) for k, v in VARIANTS.items()}
GRADIENTS |= {
    "together": dict(together=1, stream=2),
    "together-one": dict(together=1, cta_group=1, stream=2),
    "together-pair": dict(together=1, cta_group=2, stream=2),
    "together-narrow": dict(together=1, cta_group=1, width=32, stream=2),
    "together-wide": dict(together=1, cta_group=2, width=256, stream=2),
    "stream": dict(stream=1),
    "auto": dict(),
}
gradients = pytest.mark.parametrize("variant", GRADIENTS.values(), ids=GRADIENTS.keys())


def check_linear(M, N, K, *, activation=None, bias=None, residual=False, save=False, dtype=bf, seed=0, **options):
    x, w = randn(M, K, seed=seed), randn(N, K, seed=seed + 1, scale=max(K, 1) ** -0.5)
    b = None if bias is None else randn(N, seed=seed + 2).to(bias)
    r = randn(M, N, seed=seed + 3) if residual else None
    with ffn.options(**options):
        got = ffn.linear(*gpu(x, w, b), activation, gpu(r), save=save, out_dtype=dtype)
    y, z, ey, ez = ref.linear(x, w, b, activation, r)
    if save:
        assert ref.close(got[1], z, ez)
        got = got[0]
    assert got.dtype == dtype and ref.close(got, y, ey, dtype)


# ------------------------------------------------------------------ linear
@variants
@pytest.mark.parametrize("M,N,K", [(128, 128, 64), (1, 1, 1), (300, 257, 520), (37, 600, 1000), (513, 33, 72), (40, 1, 2000)])
def test_linear_variants(variant, M, N, K):
    check_linear(M, N, K, stream=2, **variant)
    check_linear(M, N, K, activation="silu", bias=bf, residual=True, save=True, stream=2, **variant)
    check_linear(M, N, K, activation="gelu", bias=torch.float32, residual=True, dtype=torch.float32, stream=2, **variant)


@pytest.mark.parametrize("width", [16, 32, 48, 64, 96, 112, 160, 208, 224, 256])
@pytest.mark.parametrize("cta_group,transposed", [(1, 1), (1, 2), (2, 1), (2, 2)])
def test_linear_widths(width, cta_group, transposed):
    if width % 32 and (cta_group == 2):
        pytest.skip("pairs take multiples of 32")
    cols = width if width % 32 else 600  # a width that is no multiple of 32 must hold all columns
    M, N = (300, cols) if transposed == 1 else (cols, 300)
    check_linear(M, N, 200, bias=bf, residual=True, stream=2, width=width, cta_group=cta_group, transposed=transposed)
    # both gradients, whose operands are contiguous along their rows
    x, w, dy = randn(M, 200, seed=1), randn(N, 200, seed=2, scale=0.1), randn(M, N, seed=3)
    with ffn.options(width=width if width % 32 == 0 else 0, cta_group=cta_group, transposed=transposed):
        dx, dw, _ = ffn.linear_backward(*gpu(dy, x, w))
    for got, a, b in ((dx, dy, w.T), (dw, dy.T, x.T)):
        want, mag = ref.product(a, b)
        assert ref.close(got, want, ref.sum_error(a.shape[1]) * mag)


@pytest.mark.parametrize("activation", ffn.ACTIVATIONS)
@pytest.mark.parametrize("dtype", [bf, torch.float32])
def test_activations_over_their_range(activation, dtype):
    # z itself, from far below to far above: 1 x 1 weights
    x = torch.cat([torch.linspace(-40, 40, 2000), torch.tensor([0.0, -0.0, 1e30, -1e30, 1e-30, 3e-39])]).to(bf)[:, None]
    w = torch.ones(1, 1).to(bf)
    for options in (dict(stream=2), dict(transposed=2, stream=2)):
        with ffn.options(**options):
            y = ffn.linear(*gpu(x, w), activation=activation, out_dtype=dtype)
        want = ref.act(activation, x.double())
        # subnormal results and their like are 0
        assert ref.close(y, want, ref.act_error(x.double(), want) + 1e-37, dtype)


def test_the_slope_over_its_range():
    z = torch.cat([torch.linspace(-40, 40, 4000), torch.tensor([0.0, 1e30, -1e30, 1e-30])]).to(bf)[None, :]
    dy, x, w = torch.ones_like(z), torch.ones(1, 8).to(bf), torch.zeros(z.shape[1], 8).to(bf)
    for activation in ffn.ACTIVATIONS:
        _, dw, db = ffn.linear_backward(*gpu(dy, x, w, z), activation=activation, bias=True, grad_dtype=torch.float32)
        want = ref.slope(activation, z.double())[0]
        assert ref.close(db, want, ref.ACT_ERROR * (want.abs() + 1), torch.float32)
        assert ref.close(dw[:, 0], want, ref.ACT_ERROR * (want.abs() + 1))  # dz, rounded to bf16


@variants
def test_linear_integers_are_exact(variant):
    M, N, K = 333, 520, 776
    x, w, b, r = ints(M, K, seed=1), ints(N, K, seed=2), ints(N, seed=3, top=9), ints(M, N, seed=4, top=9)
    z = x.double() @ w.double().T + b.double()
    with ffn.options(stream=2, **variant):
        y, zs = ffn.linear(*gpu(x, w, b), "relu", gpu(r), save=True)
        y32 = ffn.linear(*gpu(x, w, b), None, gpu(r), out_dtype=torch.float32)
    assert y.cpu().equal((z.clamp_min(0) + r.double()).to(bf)) and zs.cpu().equal(z.to(bf))
    assert y32.cpu().double().equal(z + r.double())


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("N,K", [(1, 8), (5, 64), (700, 72), (1000, 1000), (8192, 512), (38912, 64)])
def test_few_tokens(M, N, K):
    for options in (dict(stream=1), dict(stream=2), dict()):
        check_linear(M, N, K, activation="gelu_tanh", bias=bf, residual=True, save=True, **options)
        with ffn.options(**options):
            if options == dict(stream=1):
                ffn.linear(*gpu(randn(M, K), randn(N, K)))
                assert ffn.plan_info()["tiles"] == 0
    x, w, r = ints(M, K, seed=1), ints(N, K, seed=2), ints(M, N, seed=4, top=9)
    with ffn.options(stream=1):
        y = ffn.linear(*gpu(x, w), residual=gpu(r), out_dtype=torch.float32)
        h, (g, u) = ffn.gated(*gpu(x, w, w.flip(0)), activation="relu", save="bf16")
    z = x.double() @ w.double().T
    assert y.cpu().double().equal(z + r.double())
    assert g.cpu().equal(z.to(bf)) and u.cpu().equal(z.flip(1).to(bf))
    assert h.cpu().equal((z.clamp_min(0) * z.flip(1)).to(bf))


def strided(t, pitch, offset):
    """t on the GPU, rows `pitch` elements apart, `offset` elements into its storage."""
    base = torch.full((t.shape[0] * pitch + offset + 64,), 1024.0, dtype=t.dtype, device="cuda")
    view = base.as_strided(t.shape, (pitch, 1), offset)
    view.copy_(t)
    return view


@pytest.mark.parametrize("M,N,K", [(1, 200, 304), (20, 200, 304), (300, 201, 303)])
@pytest.mark.parametrize("add,offset", [(0, 0), (0, 1), (1, 0), (3, 5), (8, 8), (24, 0), (5, 64)])
def test_rows_at_any_pitch_and_offset(M, N, K, add, offset):
    x, w, r, dy = randn(M, K, seed=1), randn(N, K, seed=2, scale=0.1), randn(M, N, seed=3), randn(M, N, seed=4)
    y, z, ey, ez = ref.linear(x, w, None, "silu", r)
    xs, ws, rs = strided(x, K + add, offset), strided(w, K + add, offset), strided(r, N + add, offset)
    for dtype in (bf, torch.float32):
        base = torch.full((M * (N + add) + offset + 64,), 7.0, dtype=dtype, device="cuda")
        out = base.as_strided((M, N), (N + add, 1), offset)
        got = ffn.linear(xs, ws, activation="silu", residual=rs, out=out)
        assert got is out or got.data_ptr() == out.data_ptr()
        assert ref.close(out, y, ey, dtype)
        out.fill_(7.0)
        assert bool((base == 7.0).all())  # nothing beside the rows was written
    _, zs = ffn.linear(xs, ws, save=True)
    assert ref.close(zs, z, ez)
    zs = strided(z.to(bf), N + add, offset)
    dx, dw, db = ffn.linear_backward(strided(dy, N + add, offset), xs, ws, zs, "silu", bias=True)
    wx, ww, wb = ref.linear_backward(dy, x, w, z.to(bf), "silu")
    assert ref.close_rms(dx, wx, extra=2.0**-12) and ref.close_rms(dw, ww, extra=2.0**-12)
    assert ref.close(db, wb, 2.0**-15 * dy.double().abs().sum(0), torch.float32)


def test_a_result_may_replace_the_residual():
    x, w, r = randn(70, 96, seed=1), randn(136, 96, seed=2, scale=0.1), randn(70, 136, seed=3)
    y, _, ey, _ = ref.linear(x, w, residual=r)
    for options in (dict(), dict(transposed=2), dict(transposed=1), dict(stream=2)):
        for t in (r.cuda(), strided(r, 137, 3)):
            with ffn.options(**options):
                got = ffn.linear(*gpu(x, w), residual=t, out=t)
            assert got.data_ptr() == t.data_ptr() and ref.close(t, y, ey)
    one = randn(1, 136, seed=5).cuda()
    y, _, ey, _ = ref.linear(x[:1], w, residual=one.cpu())
    ffn.linear(*gpu(x[:1], w), residual=one, out=one)
    assert ref.close(one, y, ey)


def test_results_over_what_is_read_are_refused():
    base = torch.zeros(80, 400, dtype=bf, device="cuda")
    x, w = base[:, :96], randn(96, 96).cuda()
    with pytest.raises(ValueError, match="out lies over x"):
        ffn.linear(x, w, out=base[:, 40:136])
    with pytest.raises(ValueError, match="out lies over weight"):
        ffn.linear(x, base[:, 200:296], out=base[:, 250:330])
    with pytest.raises(ValueError, match="out lies over residual"):
        ffn.linear(x, w, residual=base[:, 200:296], out=base[:, 201:297])
    with pytest.raises(ValueError, match="out lies over residual"):
        ffn.linear(x, w, residual=base[:, 200:296], out=base[:, 200:392].view(torch.float32))
    ffn.linear(x, w, out=base[:, 96:192])  # rows beside each other
    with pytest.raises(ValueError, match="one device"):
        ffn.linear(x, w.cpu())


@pytest.mark.parametrize("cta_group", (1, 2))
@pytest.mark.parametrize("width", range(32, 257, 32))
def test_every_chunk_of_many_tiles_is_stored(width, cta_group):
    """Short sums, so that a tile's chunks follow each other at once, an odd number of them a warp or an even one."""
    x, w, want = problem(1400, 5896, 144, 51)
    shifted = torch.empty(1400, 5897, dtype=bf, device="cuda")[:, 1:]
    with ffn.options(cta_group=cta_group, transposed=1, width=width, stream=2):
        for out in (None, shifted):
            for _ in range(3):
                assert ffn.linear(x, w, out=out).cpu().equal(want)
        assert all(t.cpu().equal(want) for t in ffn.linear(x, w, save=True))


# ------------------------------------------------------------------ linear_backward
@gradients
@pytest.mark.parametrize("M,N,K", [(128, 128, 128), (1, 1, 1), (300, 257, 520), (16, 600, 1000), (700, 72, 33), (3, 520, 8)])
def test_linear_backward_variants(variant, M, N, K):
    x, w, dy, z = randn(M, K, seed=1), randn(N, K, seed=2, scale=0.1), randn(M, N, seed=3), randn(M, N, seed=4)
    for dtype in (bf, torch.float32):
        with ffn.options(**variant):
            dx, dw, none = ffn.linear_backward(*gpu(dy, x, w), grad_dtype=dtype)
            again = ffn.linear_backward(*gpu(dy, x, w), grad_dtype=dtype)
        assert none is None and dx.equal(again[0]) and dw.equal(again[1])
        want, mag = ref.product(dy, w.T)
        assert ref.close(dx, want, ref.sum_error(N) * mag)
        want, mag = ref.product(dy.T, x.T)
        assert ref.close(dw, want, ref.sum_error(M) * mag, dtype)
    with ffn.options(**variant):
        dx, dw, db = ffn.linear_backward(*gpu(dy, x, w, z), activation="gelu", bias=True)
    wx, ww, wb = ref.linear_backward(dy, x, w, z, "gelu")
    assert ref.close_rms(dx, wx, extra=2.0**-12) and ref.close_rms(dw, ww, extra=2.0**-12)
    # 1.13 a slope at most, a column's sum in fp32
    assert ref.close(db, wb, (ref.ACT_ERROR * 2.2 + M * 2.0**-24 * 1.13) * dy.double().abs().sum(0), torch.float32)


@gradients
def test_gradients_of_integers_are_exact(variant):
    M, N, K = 400, 264, 328
    x, w, dy, z = ints(M, K, seed=1), ints(N, K, seed=2), ints(M, N, seed=3), ints(M, N, seed=4)
    dz = dy.double() * (z.double() > 0)
    with ffn.options(**variant):
        dx, dw, db = ffn.linear_backward(*gpu(dy, x, w, z), activation="relu", bias=True, grad_dtype=torch.float32)
    assert dx.cpu().equal((dz @ w.double()).to(bf))
    assert dw.cpu().double().equal(dz.T @ x.double())
    assert db.cpu().double().equal(dz.sum(0))


@pytest.mark.parametrize("M,N", [(1, 1), (5, 7), (1000, 64), (37, 255), (513, 257), (8, 5000), (4096, 33), (6143, 5999)])
def test_bias_gradients(M, N):
    dy, z = ints(M, N, seed=1, top=4), ints(M, N, seed=2)
    x, w = ints(M, 8, seed=3), ints(N, 8, seed=4)
    _, _, db = ffn.linear_backward(*gpu(dy, x, w), bias=True)
    assert db.cpu().double().equal(dy.double().sum(0))
    dx, _, db = ffn.linear_backward(*gpu(dy, x, w, z), activation="relu", bias=True)
    dz = dy.double() * (z.double() > 0)
    assert db.cpu().double().equal(dz.sum(0)) and dx.cpu().equal((dz @ w.double()).to(bf))


@pytest.mark.parametrize("N,K", [(1, 8), (15, 1), (16, 520), (33, 584), (500, 4096), (1003, 7), (40, 20000), (6000, 72), (2040, 8200)])
@pytest.mark.parametrize("M", [1, 2, 8, 9, 16])
def test_gradients_of_few_tokens(M, N, K):
    x, w, dy = randn(M, K, seed=1), ints(N, K, seed=2), ints(M, N, seed=3)
    pitch = -(-K // 8) * 8 + 8
    for rows in (lambda t: t.cuda(), lambda t: strided(t, pitch, 8)):
        held = strided(dy, -(-N // 8) * 8 + 8, 8)
        with ffn.options(stream=1):
            dx, dw, _ = ffn.linear_backward(held, x.cuda(), rows(w))
            again = ffn.linear_backward(held, x.cuda(), rows(w))[0]
        assert dx.cpu().equal((dy.double() @ w.double()).to(bf)) and dx.equal(again)
        want, mag = ref.product(dy.T, x.T)
        assert ref.close(dw, want, ref.sum_error(M) * mag)
    dyr, wr = randn(M, N, seed=4), randn(N, K, seed=5)
    with ffn.options(stream=1):
        dx = ffn.linear_backward(strided(dyr, -(-N // 8) * 8, 8), x.cuda(), strided(wr, pitch, 0))[0]
    want, mag = ref.product(dyr, wr.T)
    assert ref.close(dx, want, ref.sum_error(N) * mag)


@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("save", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,C,F,N", [(1, 8, 8, 8), (3, 40, 1032, 24), (16, 520, 136, 1000), (9, 1000, 5000, 33)])
def test_gated_gradients_of_few_tokens(M, C, F, N, save, activation):
    x, wg, wu = randn(M, C, seed=1), randn(F, C, seed=2, scale=C**-0.5), randn(F, C, seed=3, scale=C**-0.5)
    wd, dy = randn(N, F, seed=4, scale=F**-0.5), randn(M, N, seed=5)
    _, saved = ffn.gated(*gpu(x, wg, wu), activation=activation, save=save)
    g, u = saved if save == "bf16" else (torch.from_numpy(fp8ref.values(saved[i].cpu(), saved[i + 1].cpu())) for i in (0, 2))
    rows = [strided(t, -(-t.shape[1] // 8) * 8, 0) for t in (dy, x)]
    weights = [strided(t, -(-t.shape[1] // 8) * 8, 8) for t in (wg, wu, wd)]
    with ffn.options(stream=1):
        got = ffn.gated_backward(*rows, saved, *weights, activation=activation)
        again = ffn.gated_backward(*rows, saved, *weights, activation=activation)
    want = ref.gated_backward(dy, x, g.cpu(), u.cpu(), wg, wu, wd, activation)
    for a, b, v in zip(got, again, want):
        # as in test_gated_backward_variants
        assert ref.close_rms(a, v, extra=2.0**-10) and a.equal(b)


# ------------------------------------------------------------------ gated
GATED = {k: v for k, v in VARIANTS.items()}


@variants
@pytest.mark.parametrize("M,C,F", [(128, 64, 128), (1, 1, 1), (300, 520, 257), (37, 1000, 600), (20, 2000, 130), (513, 72, 33)])
def test_gated_variants(variant, M, C, F):
    x, wg, wu = randn(M, C, seed=1), randn(F, C, seed=2, scale=C**-0.5), randn(F, C, seed=3, scale=C**-0.5)
    for activation in ("silu", "gelu_tanh"):
        h, g, u, eh, eg, eu = ref.gated(x, wg, wu, activation)
        with ffn.options(stream=2, **variant):
            got = ffn.gated(*gpu(x, wg, wu), activation=activation)
            hs, (gs, us) = ffn.gated(*gpu(x, wg, wu), activation=activation, save="bf16")
        assert ref.close(got, h, eh) and ref.close(hs, h, eh)  # perhaps tiled otherwise, summed in another order
        assert ref.close(gs, g, eg) and ref.close(us, u, eu)


@variants
def test_gated_integers_are_exact(variant):
    x, wg, wu = ints(200, 136, seed=1), ints(392, 136, seed=2), ints(392, 136, seed=3)
    g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
    with ffn.options(stream=2, **variant):
        h, (gs, us) = ffn.gated(*gpu(x, wg, wu), activation="relu", save="bf16")
    assert h.cpu().equal((g.clamp_min(0) * u).to(bf))
    assert gs.cpu().equal(g.to(bf)) and us.cpu().equal(u.to(bf))


@pytest.mark.parametrize("M,C,F", [(1, 8, 1), (1, 136, 500), (20, 136, 128), (200, 136, 392), (333, 72, 1025), (129, 0, 130)])
@pytest.mark.parametrize("cta_group", [0, 1, 2])
def test_checkpoints_in_8_bits(M, C, F, cta_group):
    # sums are integers, exact in fp32: so are the codes and scales
    x, wg, wu = ints(M, C, seed=1), ints(F, C, seed=2), ints(F, C, seed=3)
    with ffn.options(cta_group=cta_group):
        h, (gc, gs, uc, us) = ffn.gated(*gpu(x, wg, wu), save="e4m3", activation="relu")
    g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
    assert h.cpu().equal((g.clamp_min(0) * u).to(bf))
    for codes, scales, v in ((gc, gs, g), (uc, us, u)):
        want, e = fp8ref.quantize(v.numpy())
        bytes_, padding = fp8ref.scale_bytes(scales, F)
        assert (bytes_ == e).all() and (padding == 127).all()
        assert codes.cpu().double().equal(torch.from_numpy(want))
        # the format of fp8's quantisers, which give the same of the same values
        qc, qs = fp8.quantize(v.float().cuda())
        assert qc.view(torch.uint8).equal(codes.view(torch.uint8)) and qs.view(torch.uint8).equal(scales.view(torch.uint8))


@gradients
@pytest.mark.parametrize("save", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,C,F,N", [(128, 128, 128, 128), (1, 1, 1, 1), (300, 136, 257, 200), (20, 520, 600, 264), (70, 33, 1030, 7)])
def test_gated_backward_variants(variant, save, M, C, F, N):
    x, wg, wu = randn(M, C, seed=1), randn(F, C, seed=2, scale=C**-0.5), randn(F, C, seed=3, scale=C**-0.5)
    wd, dy = randn(N, F, seed=4, scale=F**-0.5), randn(M, N, seed=5)
    for activation in ("silu", "gelu"):
        if save == "bf16":
            saved = randn(M, F, seed=6), randn(M, F, seed=7)
            g, u = saved
        else:
            saved = ()
            for s in (6, 7):
                codes, e = fp8ref.quantize(torch.randn(M, F, generator=torch.Generator().manual_seed(s)).numpy())
                held = torch.zeros(M, -(-F // 128) * 128, dtype=torch.uint8)
                held[:, :F] = torch.from_numpy(codes).float().to(torch.float8_e4m3fn).view(torch.uint8)
                saved += held.view(torch.float8_e4m3fn)[:, :F], fp8ref.pack_scales(e)
            g, u = (torch.from_numpy(fp8ref.values(*saved[i:i + 2])) for i in (0, 2))
            held = [t.cuda() if i % 2 else torch.empty_strided(t.shape, (-(-F // 128) * 128, 1), dtype=t.dtype, device="cuda")
                    for i, t in enumerate(saved)]
            for a, b in zip(held, saved):
                a.view(torch.uint8).copy_(b.view(torch.uint8))
            saved = tuple(held)
        with ffn.options(**variant):
            got = ffn.gated_backward(*gpu(dy, x), tuple(t.cuda() for t in saved), *gpu(wg, wu, wd), activation=activation)
            f32 = ffn.gated_backward(*gpu(dy, x), tuple(t.cuda() for t in saved), *gpu(wg, wu, wd), activation=activation,
                                     grad_dtype=torch.float32)
        want = ref.gated_backward(dy, x, g, u, wg, wu, wd, activation)
        # terms that round to the other side: one in some thousand, by a step of 2^-7
        for a, b, w in zip(got, f32, want):
            assert ref.close_rms(a, w, extra=2.0**-10)
            assert b.dtype == (bf if w is want[0] else torch.float32)
            assert ref.close_rms(b, w, bf if w is want[0] else torch.float32, extra=2.0**-10)


@gradients
def test_gated_gradients_of_integers_are_exact(variant):
    M, C, F, N = 200, 136, 264, 72
    x, wg, wu, wd = ints(M, C, seed=1, top=1), ints(F, C, seed=2, top=1), ints(F, C, seed=3, top=1), ints(N, F, seed=4, top=1)
    dy, g, u = ints(M, N, seed=5, top=1), ints(M, F, seed=6), ints(M, F, seed=7)
    with ffn.options(**variant):
        got = ffn.gated_backward(*gpu(dy, x), (g.cuda(), u.cuda()), *gpu(wg, wu, wd), activation="relu",
                                 grad_dtype=torch.float32)
    want = ref.gated_backward(dy, x, g, u, wg, wu, wd, "relu")
    assert got[0].cpu().equal(want[0].to(bf))
    for a, b in zip(got[1:], want[1:]):
        assert a.cpu().double().equal(b)


@pytest.mark.parametrize("M,F", [(300, 201), (5, 201), (1, 40)])
@pytest.mark.parametrize("add,offset", [(0, 1), (1, 0), (8, 8), (16, 0)])
def test_checkpoints_at_any_pitch_and_offset(M, F, add, offset):
    C, N = 40, 24
    x, wg, wu, wd, dy = ints(M, C, seed=1, top=1), ints(F, C, seed=2), ints(F, C, seed=3), ints(N, F, seed=4, top=1), ints(M, N, seed=5)
    g, u = ints(M, F, seed=6), ints(M, F, seed=7)
    want = ref.gated_backward(dy, x, g, u, wg, wu, wd, "relu")
    got = ffn.gated_backward(strided(dy, N + add, offset), strided(x, C + add, offset),
                             (strided(g, F + add, offset), strided(u, F + add + 1, offset)),
                             strided(wg, C + add, offset), strided(wu, C + add, offset), strided(wd, F + add, offset),
                             activation="relu", grad_dtype=torch.float32)
    assert got[0].cpu().equal(want[0].to(bf))
    for a, b in zip(got[1:], want[1:]):
        assert a.cpu().double().equal(b)
    # codes at multiples of 16 bytes that are none of 32
    held = torch.zeros(M, -(-F // 16) * 16 + 16, dtype=torch.uint8, device="cuda")
    codes = held[:, 16:16 + F].view(torch.float8_e4m3fn)
    codes.view(torch.uint8).copy_(g.float().to(torch.float8_e4m3fn).view(torch.uint8))
    ones = torch.full((-(-F // 512), M, 4), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    got = ffn.gated_backward(*gpu(dy, x), (codes, ones, codes, ones), *gpu(wg, wu, wd), activation="relu")
    want = ref.gated_backward(dy, x, g, g, wg, wu, wd, "relu")
    for a, b in zip(got, want):
        assert a.cpu().equal(b.to(bf))


# ------------------------------------------------------------------ empty sums, values that are not finite
def test_sizes_of_zero():
    e = lambda *s: torch.zeros(*s, dtype=bf, device="cuda")  # noqa: E731
    b, r = randn(20, seed=1).cuda(), randn(5, 20, seed=2).cuda()
    assert ffn.linear(e(0, 8), e(20, 8)).shape == (0, 20) and ffn.linear(e(5, 8), e(0, 8)).shape == (5, 0)
    for options in (dict(), dict(transposed=2), dict(cta_group=2), dict(transposed=1, cta_group=2)):
        with ffn.options(**options):
            y, z = ffn.linear(e(5, 0), e(20, 0), b, "relu", r, save=True)
            assert z.equal(b.expand(5, 20))
            assert ref.close(y, b.double().cpu().clamp_min(0).expand(5, 20) + r.double().cpu(), 0)
            assert ffn.linear(e(300, 0), e(200, 0), out_dtype=torch.float32).equal(torch.zeros(300, 200, device="cuda"))
            h, saved = ffn.gated(e(300, 0), e(200, 0), e(200, 0), save="bf16")
            assert not h.any() and not saved[0].any() and not saved[1].any()
            dx, dw, db = ffn.linear_backward(e(0, 20), e(0, 8), e(20, 8), bias=True)
            assert dx.shape == (0, 8) and dw.equal(e(20, 8)) and db.equal(torch.zeros(20, device="cuda"))
            dx, dw, db = ffn.linear_backward(e(0, 20), e(0, 8), e(20, 8), e(0, 20), "silu", bias=True)
            assert dw.equal(e(20, 8)) and db.equal(torch.zeros(20, device="cuda"))
            dx, dw, db = ffn.linear_backward(e(5, 0), e(5, 8), e(0, 8), bias=True)
            assert dx.equal(e(5, 8)) and dw.shape == (0, 8) and db.shape == (0,)
            for M, C, F, N in ((0, 8, 16, 8), (5, 0, 16, 8), (5, 8, 0, 8), (5, 8, 16, 0)):
                h, saved = ffn.gated(e(M, C), e(F, C), e(F, C), save="e4m3")
                got = ffn.gated_backward(e(M, N), e(M, C), saved, e(F, C), e(F, C), e(N, F))
                assert [tuple(t.shape) for t in got] == [(M, C), (F, C), (F, C), (N, F)]
                assert not any(t.any() for t in got)


@pytest.mark.parametrize("options", [dict(stream=1), dict(stream=2), dict(transposed=1), dict(transposed=2)])
def test_values_that_are_not_finite_stay_in_their_rows(options):
    M, N, K = 20, 136, 136
    x, w = randn(M, K, seed=1), randn(N, K, seed=2)
    x[3, 5], x[7, 0], w[9, K - 1] = float("inf"), float("nan"), float("-inf")
    with ffn.options(**options):
        y = ffn.linear(*gpu(x, w)).cpu()
        h = ffn.gated(*gpu(x, w, w)).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3], bad[7], bad[:, 9] = True, True, True
    assert bool(torch.isfinite(y[~bad]).all()) and not bool(torch.isfinite(y[bad]).any())
    assert bool(torch.isfinite(h[~bad]).all()) and not bool(torch.isfinite(h[bad]).any())
    # infinities are no part of a block's scale
    _, (gc, gs, _, _) = ffn.gated(*gpu(x, w, w), save="e4m3")
    got = fp8ref.values(gc.cpu(), gs.cpu())
    row = [i for i in range(N) if i != 9]
    want, mag = ref.product(x[:1], w)
    held = ref.checkpoint(torch.where(torch.isfinite(want), want, torch.zeros_like(want)))
    assert bool(torch.isnan(torch.from_numpy(got[0, 9:10])).all())
    limit = 2.0**-4 * want.abs() + 2.0**-9 * want[0, row].abs().max()
    assert ((torch.from_numpy(got[0, row]) - held[0, row]).abs() <= limit[0, row]).all()


# ------------------------------------------------------------------ through the C ABI
def raw(M, N, K):
    return torch.full((M * N + K,), 5.0, dtype=bf, device="cuda")


def matrix(t):
    return ffn.Matrix(t.data_ptr(), t.stride(0))


def c_call(name, args, fill=None):
    lib, need = ffn.load(), ctypes.c_int64(-1)
    assert getattr(lib, f"ffn_{name}_workspace")(ctypes.byref(args), ctypes.byref(need)) == ffn.OK
    work = torch.empty(max(need.value, 256) + 256, dtype=torch.uint8, device="cuda")
    if fill is not None:
        work.fill_(fill)
    call = lambda p, n: getattr(lib, f"ffn_{name}")(  # noqa: E731
        ctypes.byref(args), p, n, torch.cuda.current_stream().cuda_stream)
    if need.value:
        assert call(None, need.value) == ffn.ERR_WORKSPACE
        assert call(work.data_ptr(), need.value - 1) == ffn.ERR_WORKSPACE
        assert call(work.data_ptr() + 16, need.value) == ffn.ERR_ALIGNMENT
    assert call(work.data_ptr(), need.value) == ffn.OK
    torch.cuda.synchronize()
    assert bool((work[need.value:] == (fill or 0)).all()) if fill is not None else True
    return need.value


@pytest.mark.parametrize("M,N,K", [(200, 264, 520), (1, 264, 520), (37, 201, 303)])
def test_only_the_results_rows_are_written(M, N, K):
    def held(R, C, dtype=bf):
        base = torch.full((R, C + 72), 5.0, dtype=dtype, device="cuda")
        return base, base[:, 8:8 + C]

    def untouched(base, C):
        return bool((base[:, :8] == 5.0).all()) and bool((base[:, 8 + C:] == 5.0).all())

    x, w, dy = ints(M, K, seed=1).cuda(), ints(N, K, seed=2).cuda(), ints(M, N, seed=3).cuda()
    (yb, y), (zb, z) = held(M, N), held(M, N)
    c_call("linear", ffn.LinearArgs(M=M, N=N, K=K, x=matrix(x), weight=matrix(w), y=matrix(y), z=matrix(z)), 255)
    want = x.double() @ w.double().T
    assert y.equal(want.to(bf)) and z.equal(y) and untouched(yb, N) and untouched(zb, N)
    (dxb, dx), (dwb, dw) = held(M, K), held(N, K, torch.float32)
    db = torch.full((N + 8,), 5.0, device="cuda")
    c_call("linear_backward", ffn.LinearBackwardArgs(M=M, N=N, K=K, dy=matrix(dy), x=matrix(x), weight=matrix(w),
                                                     dx=matrix(dx), dweight=matrix(dw), dweight_type=1,
                                                     dbias=db.data_ptr()), 1)
    assert dx.equal((dy.double() @ w.double()).to(bf)) and untouched(dxb, K)
    assert dw.double().equal(dy.double().T @ x.double()) and untouched(dwb, K)
    assert db[:N].double().equal(dy.double().sum(0)) and bool((db[N:] == 5.0).all())
    # one gradient at a time
    for part in ("dx", "dweight", "dbias"):
        a = ffn.LinearBackwardArgs(M=M, N=N, K=K, dy=matrix(dy), x=matrix(x), weight=matrix(w))
        dx.fill_(5), dw.fill_(5), db.fill_(5)
        setattr(a, part, {"dx": matrix(dx), "dweight": matrix(dw), "dbias": db.data_ptr()}[part])
        a.dweight_type = 1
        c_call("linear_backward", a)
        assert dx.equal((dy.double() @ w.double()).to(bf)) == (part == "dx")
        assert dw.double().equal(dy.double().T @ x.double()) == (part == "dweight")
        assert db[:N].double().equal(dy.double().sum(0)) == (part == "dbias")
    (hb, h), (gb, g), (ub, u) = held(M, N), held(M, N), held(M, N)
    c_call("gated", ffn.GatedArgs(M=M, F=N, C=K, x=matrix(x), w_gate=matrix(w), w_up=matrix(w), activation=1,
                                  h=matrix(h), g=matrix(g), u=matrix(u)), 255)
    assert g.equal(want.to(bf)) and u.equal(g) and h.equal((want.clamp_min(0) * want).to(bf))
    assert untouched(hb, N) and untouched(gb, N) and untouched(ub, N)
    pitch, kt = -(-N // 128) * 128 + 128, -(-N // 512)
    codes = torch.full((2, M, pitch), 3, dtype=torch.uint8, device="cuda")
    scales = torch.full((2, kt * M * 4 + 8), 3, dtype=torch.uint8, device="cuda")
    q = [ffn.Quantized(codes[i].data_ptr(), pitch, scales[i].data_ptr()) for i in (0, 1)]
    c_call("gated", ffn.GatedArgs(M=M, F=N, C=K, x=matrix(x), w_gate=matrix(w), w_up=matrix(w), activation=1,
                                  h=matrix(h), qg=q[0], qu=q[1]), 255)
    qc, qs = fp8.quantize(want.float())
    for i in (0, 1):
        assert codes[i][:, :N].equal(qc.view(torch.uint8)) and bool((codes[i][:, pitch - 128:] == 3).all())
        assert scales[i][:-8].equal(qs.view(torch.uint8).flatten()) and bool((scales[i][-8:] == 3).all())


@pytest.mark.parametrize("M", (1, 7, 13))
def test_streamed_gradients_write_their_rows_alone(M):
    N, K = 264, 520
    x, w, dy = ints(M, K, seed=1).cuda(), ints(N, K, seed=2).cuda(), ints(M, N, seed=3).cuda()
    want = (dy.double() @ w.double()).to(bf)
    for offset, pitch in ((8, K + 72), (7, K + 71)):
        base = torch.full((M, pitch), 5.0, dtype=bf, device="cuda")
        dx = base[:, offset:offset + K]
        with ffn.options(stream=1):
            c_call("linear_backward", ffn.LinearBackwardArgs(M=M, N=N, K=K, dy=matrix(dy), x=matrix(x), weight=matrix(w),
                                                             dx=ffn.Matrix(dx.data_ptr(), pitch)))
        assert ffn.plan_info()["tiles"] == 0
        assert dx.equal(want) and bool((base[:, :offset] == 5.0).all()) and bool((base[:, offset + K:] == 5.0).all())
    # what is not finite stays in its token and its column
    dy[M - 1, 40], w[100, 300] = float("inf"), float("nan")
    with ffn.options(stream=1):
        dx = ffn.linear_backward(dy, x, w)[0]
    clean = torch.ones(M, K, dtype=torch.bool)
    clean[M - 1], clean[:, 300] = False, False
    assert dx.cpu()[clean].equal(want.cpu()[clean]) and not dx[:, 300].isfinite().any()
    assert not dx[M - 1, w[40] != 0].isfinite().any()


def test_gated_backward_parts():
    M, C, F, N = 40, 72, 136, 24
    x, wg, wu, wd = ints(M, C, seed=1, top=1), ints(F, C, seed=2, top=1), ints(F, C, seed=3, top=1), ints(N, F, seed=4, top=1)
    dy, g, u = ints(M, N, seed=5, top=1), ints(M, F, seed=6), ints(M, F, seed=7)
    want = ref.gated_backward(dy, x, g, u, wg, wu, wd, "relu")
    ts = {k: v.cuda() for k, v in dict(x=x, w_gate=wg, w_up=wu, w_down=wd, dy=dy, g=g, u=u).items()}
    outs = dict(dx=(M, C), dw_gate=(F, C), dw_up=(F, C), dw_down=(N, F))
    for parts in (("dx",), ("dw_gate", "dw_up"), ("dw_down",), tuple(outs)):
        made = {k: torch.full(s, 5.0, dtype=bf, device="cuda") for k, s in outs.items()}
        a = ffn.GatedBackwardArgs(M=M, F=F, C=C, N=N, activation=1, **{k: matrix(v) for k, v in ts.items()},
                                  **{k: matrix(made[k]) for k in parts})
        c_call("gated_backward", a, 1)
        for k, w in zip(outs, want):
            assert made[k].cpu().equal(w.to(bf)) if k in parts else bool((made[k] == 5.0).all())


# ------------------------------------------------------------------ offsets past 32 bits
def test_offsets_past_32_bits():
    M, K, N = 70001, 32768, 24
    x = torch.zeros(M, K, dtype=bf, device="cuda")
    rows = [0, 1, 40000, 65535, 65536, M - 1]
    x[rows] = ints(len(rows), K, seed=1).cuda()
    w = ints(N, K, seed=2).cuda()
    want = x[rows].double() @ w.double().T
    for options in (dict(), dict(transposed=1), dict(transposed=2)):
        with ffn.options(**options):
            y = ffn.linear(x, w, out_dtype=torch.float32)
        assert y[rows].double().equal(want) and int(torch.count_nonzero(y)) == int(torch.count_nonzero(want))
    # x as the gradient of a wide result: read by the slope, as an operand, and the products of both
    v = ints(K, N, seed=3).cuda()
    z = torch.ones(1, 1, dtype=bf, device="cuda").expand(M, K).contiguous()
    dx, dw, db = ffn.linear_backward(x, y.to(bf), v, z, "relu", bias=True, grad_dtype=torch.float32)
    assert dx[rows].equal((x[rows].double() @ v.double()).to(bf))
    assert dw.double().equal(x[rows].double().T @ y.to(bf)[rows].double())
    assert db.double().equal(x[rows].double().sum(0))
    del z, dx
    # rows far apart
    far = torch.empty((1 << 32) + K, dtype=bf, device="cuda").as_strided((3, K), ((1 << 31) - 64, 1))
    far.copy_(x[rows[:3]])
    assert ffn.linear(far, w, out_dtype=torch.float32).double().equal(want[:3])


# ------------------------------------------------------------------ streams, graphs, launches that give up
def problem(M, N, K, seed):
    x, w = ints(M, K, seed=seed), ints(N, K, seed=seed + 1)
    return x.cuda(), w.cuda(), (x.double() @ w.double().T).to(bf)


SPLIT = dict(cta_group=1, transposed=2, width=32, split=2, stream=2)  # tiles meet through global memory


def test_graphs_replayed_at_once_on_two_streams():
    M, N, K = 20, 2560, 6000
    work = [problem(M, N, K, seed) for seed in (3, 14)]
    graphs, outs = [], []
    with ffn.options(**SPLIT):
        for x, w, _ in work:
            ffn.linear(x, w)
        assert ffn.plan_info()["split_tiles"] == 20 and ffn.plan_info()["cluster"] == 1
        torch.cuda.synchronize()
        for x, w, _ in work:
            graphs.append(torch.cuda.CUDAGraph())
            outs.append(torch.empty(M, N, dtype=bf, device="cuda"))
            with torch.cuda.graph(graphs[-1]):
                for _ in range(8):
                    ffn.linear(x, w, out=outs[-1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for o in outs:
            o.fill_(0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, (_, _, want) in zip(outs, work):
            assert o.cpu().equal(want)


def test_calls_at_once_on_streams_of_their_own():
    work = [problem(20, 2560, 6000, seed) for seed in (5, 16, 27)]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    outs = [[] for _ in work]
    with ffn.options(**SPLIT):
        for _ in range(6):
            for i, ((x, w, _), s) in enumerate(zip(work, streams)):
                outs[i].append(ffn.linear(x, w, stream=s if i else s.cuda_stream))
    torch.cuda.synchronize()
    for o, (_, _, want) in zip(outs, work):
        assert all(t.cpu().equal(want) for t in o)


def test_split_tiles_meet_beside_other_streams():
    """Launches of SM pairs and of single SMs, all split, on streams of two priorities: each finds its places
    piecemeal, and none may wait for a CTA that the others keep from starting."""
    low, high = torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-1)
    work = [(low, dict(SPLIT, cta_group=2, width=64), problem(300, 2560, 6000, 5)),
            (high, SPLIT, problem(20, 2560, 6000, 16)),
            (low, dict(SPLIT, width=64), problem(100, 2600, 4000, 27)),
            (high, dict(SPLIT, cta_group=2, width=64), problem(260, 2000, 4000, 38))]
    torch.cuda.synchronize()
    outs = [[] for _ in work]
    for _ in range(30):
        for o, (stream, options, (x, w, _)) in zip(outs, work):
            with ffn.options(**options):
                o.append(ffn.linear(x, w, stream=stream))
    assert ffn.device_status() == (ffn.OK, 0)
    for o, (_, _, (_, _, want)) in zip(outs, work):
        assert all(t.cpu().equal(want) for t in o)


def test_a_backward_pass_from_a_graph():
    M, C, F, N = 200, 136, 264, 136
    x, wg, wu, wd = (ints(*s, seed=i, top=1).cuda() for i, s in enumerate(((M, C), (F, C), (F, C), (N, F))))
    dy = ints(M, N, seed=9, top=1).cuda()
    run = lambda: (lambda h, s: ffn.gated_backward(dy, x, s, wg, wu, wd, "relu"))(*ffn.gated(x, wg, wu, "relu", save="e4m3"))  # noqa: E731
    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in (20, 30):
        for t, s in ((x, seed), (dy, seed + 1)):
            t.copy_(ints(*t.shape, seed=s, top=1))
        graph.replay()
        want = run()
        assert all(a.equal(b) for a, b in zip(got, want))


@variants
def test_a_launch_may_give_up_at_any_load(variant):
    # loads in the ring's first lap and later ones: stages that follow the missing load are not
    # filled again, and the next launch is right
    x, w, want = problem(200, 640, 6000, 1)
    if variant == {}:
        variant = dict(cta_group=2, width=256, transposed=1)
    for skip in (0, 1, 2, 3, 5, 8, 13, 20, 40):
        with ffn.options(watchdog_ns=4000000, fault_skip_load=skip, stream=2, **variant):
            ffn.linear(x, w)
            st, _ = ffn.device_status()
        assert st in (ffn.ERR_DEVICE_TIMEOUT, ffn.OK)  # OK: no CTA has that many loads
        assert st == ffn.ERR_DEVICE_TIMEOUT or skip > 1
        with ffn.options(stream=2, **variant):
            assert ffn.linear(x, w).cpu().equal(want)
        assert ffn.device_status() == (ffn.OK, 0)


def test_products_of_one_launch_may_give_up():
    x, w, _ = problem(300, 640, 2000, 1)
    dy = ints(300, 640, seed=3).cuda()
    for variant, skip in itertools.product((dict(cta_group=1, width=64), dict(cta_group=2, width=256), dict(cta_group=2, width=32)), (0, 1, 6, 17)):
        with ffn.options(together=1, **variant):
            want = ffn.linear_backward(dy, x, w, grad_dtype=torch.float32)
            assert ffn.plan_info()["products"] == 2
        with ffn.options(together=1, watchdog_ns=4000000, fault_skip_load=skip, **variant):
            ffn.linear_backward(dy, x, w)
            st, _ = ffn.device_status()
        assert st == ffn.ERR_DEVICE_TIMEOUT or (st == ffn.OK and skip > 6)
        with ffn.options(together=1, **variant):
            got = ffn.linear_backward(dy, x, w, grad_dtype=torch.float32)
        assert got[0].equal(want[0]) and got[1].equal(want[1])
        assert got[1].double().equal(dy.double().T @ x.double())
        assert ffn.device_status() == (ffn.OK, 0)


def test_a_gated_launch_may_give_up():
    x, w, _ = problem(200, 640, 6000, 1)
    for variant, skip in itertools.product((VARIANTS["one"], VARIANTS["pair"], VARIANTS["one-t"], VARIANTS["pair-t"]), (0, 7, 20)):
        want = ffn.gated(x, w, w, "relu")
        with ffn.options(watchdog_ns=4000000, fault_skip_load=skip, stream=2, **variant):
            ffn.gated(x, w, w, "relu")
            assert ffn.device_status()[0] == ffn.ERR_DEVICE_TIMEOUT
        with ffn.options(stream=2, **variant):
            assert ffn.gated(x, w, w, "relu").equal(want)
        assert ffn.device_status() == (ffn.OK, 0)


def test_every_run_gives_the_same_bits():
    x, w, dy = randn(300, 2000, seed=1).cuda(), randn(520, 2000, seed=2).cuda(), randn(300, 520, seed=3).cuda()
    first = (ffn.linear(x, w, activation="gelu"),) + ffn.linear_backward(dy, x, w, bias=True)
    for _ in range(5):
        again = (ffn.linear(x, w, activation="gelu"),) + ffn.linear_backward(dy, x, w, bias=True)
        assert all(a.equal(b) for a, b in zip(first, again))
