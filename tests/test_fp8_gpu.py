"""GPU parity of the 8-bit operators against 64-bit references on the CPU.

Where the format makes the result exact (integer codes with power-of-two scales
whose sums fit 24 bits; quantising values that are held exactly) it must be equal
bit for bit.  Elsewhere the tolerances follow from the arithmetic: u = 2^-24 is
half a unit of fp32, a sum of n terms is off by at most n 2u sum|terms|
(whatever its order, and also if additions truncate), bf16 rounds by 2^-9 and
e4m3 by 2^-4 of a normal value, or by half its least step.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_reference as ref
from warp_specialized_tma_gb300 import fp8

pytestmark = pytest.mark.gpu

U = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    fp8.load()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def held(codes: torch.Tensor, pitch=None) -> torch.Tensor:
    """codes on the GPU, rows at `pitch` bytes (default a multiple of 128), 0x7f (NaN) between them."""
    R, K = codes.shape
    pitch = -(-K // 128) * 128 if pitch is None else pitch
    buf = torch.full((R, pitch), 0x7F, dtype=torch.uint8, device="cuda")
    buf[:, :K] = codes.view(torch.uint8).cuda()
    return buf.view(torch.float8_e4m3fn)[:, :K]


def integer_operand(R, K, gen):
    """Codes that are integers in -4..4 and scales 2^-2..2^2: sums over K <= 2048 fit 24 bits."""
    c = torch.randint(-4, 5, (R, K), generator=gen).float().to(torch.float8_e4m3fn)
    e = torch.randint(125, 130, (R, -(-K // 128)), generator=gen).numpy()
    return c, ref.pack_scales(e)


def random_operand(R, K, gen, spread=3):
    """Any finite code, scales over 2 * spread powers of two."""
    b = torch.randint(0, 256, (R, K), generator=gen).to(torch.uint8)
    b[(b & 0x7F) == 0x7F] = 0  # NaN
    e = torch.randint(127 - spread, 128 + spread, (R, -(-K // 128)), generator=gen).numpy()
    return b.view(torch.float8_e4m3fn), ref.pack_scales(e)


def to_bf16(v: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(v).to(torch.bfloat16)


def run_gemm(a, sa, b, sb, out_dtype, pitch=None, **options):
    with fp8.Gemm(0, **options) as g:
        d = g.run(held(a, pitch), sa.cuda(), held(b, pitch), sb.cuda(), out_dtype=out_dtype)
        st, detail = g.device_status()
        assert st == fp8.OK, f"status {st} detail {detail:#x}"
        info = g.info()
    return d.cpu(), info


def exact_check(M, N, K, out_dtype, seed=0, pitch=None, **options):
    gen = torch.Generator().manual_seed(1000 * M + 10 * N + K + seed)
    a, sa = integer_operand(M, K, gen)
    b, sb = integer_operand(N, K, gen)
    d, info = run_gemm(a, sa, b, sb, out_dtype, pitch, **options)
    want = ref.values(a, sa) @ ref.values(b, sb).T
    if out_dtype == torch.float32:
        assert torch.equal(d.double(), torch.from_numpy(want))
    else:
        assert torch.equal(d, to_bf16(want))
    return info


SHAPES = [(1, 1, 1), (1, 128, 128), (3, 5, 17), (128, 32, 128), (128, 128, 512), (129, 33, 513), (256, 256, 256),
          (300, 500, 1000), (64, 1024, 2048), (1, 4096, 1024), (17, 999, 640), (1024, 16, 2048), (513, 257, 129)]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gemm_exact_integers(shape, out_dtype):
    exact_check(*shape, out_dtype)


@pytest.mark.parametrize("split", [0, 1, 2])
@pytest.mark.parametrize("transposed", [1, 2])
@pytest.mark.parametrize("cta_group,width", [(1, 32), (1, 64), (1, 128), (1, 160), (1, 224), (2, 32), (2, 96), (2, 128),
                                             (2, 192), (2, 224)])
def test_gemm_exact_every_tiling(cta_group, width, transposed, split):
    # 700 x 900: several tiles each way, the last ones partial, in every tiling
    info = exact_check(700, 900, 1500, torch.bfloat16, cta_group=cta_group, width=width, transposed=transposed,
                       split=split)
    assert (info["cta_group"], info["width"], info["transposed"]) == (cta_group, width, transposed - 1)
    exact_check(259, 130, 2048, torch.float32, cta_group=cta_group, width=width, transposed=transposed, split=split)


@pytest.mark.parametrize("tokens", [1, 15, 16, 17, 33, 64, 100])
def test_gemm_exact_few_tokens_both_ways(tokens):
    exact_check(tokens, 2000, 2048, torch.bfloat16)
    exact_check(2000, tokens, 2048, torch.float32)
    if tokens <= 16:  # the narrowest tile
        info = exact_check(tokens, 2000, 2048, torch.bfloat16, width=16, cta_group=1, transposed=2)
        assert info["width"] == 16


@pytest.mark.parametrize("tiles", [64, 48, 36, 30, 25, 21, 16, 5])
def test_gemm_exact_tiles_shared_by_clusters(tiles):
    # 152 // tiles CTAs to a tile, up to 8, as far as the device can place them
    info = exact_check(20, 128 * tiles - 3, 8192, torch.bfloat16, cta_group=1, transposed=2, width=32)
    assert 2 <= info["cluster"] <= 8 and info["split_tiles"] == tiles
    assert info["grid_ctas"] == tiles * info["cluster"]
    info = exact_check(128 * tiles - 1, 20, 8000, torch.float32, cta_group=1, transposed=1, width=32)
    assert 2 <= info["cluster"] <= 8


@pytest.mark.parametrize("over", [1, 3, 70, 140])
@pytest.mark.parametrize("cta_group,K", [(1, 8192), (2, 8192), (1, 12000)])
def test_gemm_exact_partial_wave_shared_by_all(cta_group, K, over):
    # a few tiles more than SMs (or SM pairs): the rest is split through global
    # memory, down to fewer k-blocks than there are clusters to take them
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sms // cta_group + over // cta_group
    info = exact_check(32, 128 * cta_group * tiles, K, torch.bfloat16, cta_group=cta_group, transposed=2, width=32,
                       split=2)
    assert info["tiles"] == tiles and info["split_tiles"] in (0, tiles - sms // cta_group)


@pytest.mark.parametrize("N", [127, 120, 124, 126])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_gemm_writes_only_its_matrix(N, out_dtype):
    # D inside a larger buffer: rows with and without the alignment TMA stores need
    gen = torch.Generator().manual_seed(N)
    M, K = 150, 300
    a, sa = integer_operand(M, K, gen)
    b, sb = integer_operand(N, K, gen)
    want = ref.values(a, sa) @ ref.values(b, sb).T
    for ld, first in ((N, 0), (128, 0), (136, 8), (131, 1)):
        for transposed in (1, 2):
            buf = torch.full((M + 2, ld + first), -7.0, dtype=out_dtype, device="cuda")
            out = buf[1:-1, first:first + N]
            with fp8.Gemm(0, transposed=transposed) as g:
                g.run(held(a), sa.cuda(), held(b), sb.cuda(), out=out)
                assert g.device_status()[0] == fp8.OK
            assert torch.equal(out.cpu(), torch.from_numpy(want).to(out_dtype))
            buf[1:-1, first:first + N] = -7.0
            assert bool((buf == -7.0).all())


def test_gemm_pitches():
    for pitch in (304, 320, 512):
        exact_check(200, 300, 300, torch.bfloat16, pitch=pitch)


@pytest.mark.parametrize("shape", [(200, 300, 5000), (1, 512, 8192), (40, 700, 4104), (600, 520, 640)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_gemm_any_codes(shape, out_dtype):
    M, N, K = shape
    gen = torch.Generator().manual_seed(M + N + K)
    a, sa = random_operand(M, K, gen)
    b, sb = random_operand(N, K, gen)
    d, _ = run_gemm(a, sa, b, sb, out_dtype)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    want = va @ vb.T
    tol = K * 2 * U * (np.abs(va) @ np.abs(vb).T)
    if out_dtype == torch.bfloat16:
        tol += 2.0**-8 * np.abs(want)
    assert (np.abs(d.double().numpy() - want) <= tol).all()


def test_gemm_scales_of_every_size():
    # products of scales from 2^-100 to 2^100, each row's own
    M, N, K = 130, 140, 1024
    gen = torch.Generator().manual_seed(5)
    a, _ = integer_operand(M, K, gen)
    b, _ = integer_operand(N, K, gen)
    ea = np.repeat(np.linspace(27, 127, M).astype(np.int64)[:, None], 8, 1)
    eb = np.repeat(np.linspace(127, 227, N).astype(np.int64)[:, None], 8, 1)
    sa, sb = ref.pack_scales(ea), ref.pack_scales(eb)
    d, _ = run_gemm(a, sa, b, sb, torch.float32)
    assert torch.equal(d.double(), torch.from_numpy(ref.values(a, sa) @ ref.values(b, sb).T))


def test_gemm_nan_reaches_its_row_and_column_only():
    gen = torch.Generator().manual_seed(6)
    a, sa = integer_operand(140, 300, gen)
    b, sb = integer_operand(150, 300, gen)
    a.view(torch.uint8)[7, 299] = 0x7F
    b.view(torch.uint8)[140, 0] = 0xFF
    d, _ = run_gemm(a, sa, b, sb, torch.float32)
    bad = torch.isnan(d)
    want = torch.zeros_like(bad)
    want[7, :] = True
    want[:, 140] = True
    assert torch.equal(bad, want)


def test_gemm_split_is_repeatable_and_survives_replanning():
    gen = torch.Generator().manual_seed(7)
    a, sa = random_operand(300, 6000, gen)
    b, sb = random_operand(700, 6000, gen)
    a2, sa2 = random_operand(16, 3000, gen)
    b2, sb2 = random_operand(900, 3000, gen)
    args = held(a), sa.cuda(), held(b), sb.cuda()
    args2 = held(a2), sa2.cuda(), held(b2), sb2.cuda()
    with fp8.Gemm(0) as g:
        first, first2 = g.run(*args), g.run(*args2)
        assert g.info()["split_tiles"] > 0
        for _ in range(30):
            d, d2 = g.run(*args), g.run(*args2)
            assert torch.equal(d, first) and torch.equal(d2, first2)
        assert g.device_status()[0] == fp8.OK


def test_gemm_in_a_graph():
    gen = torch.Generator().manual_seed(8)
    a, sa = integer_operand(8, 2000, gen)
    b, sb = integer_operand(1000, 2000, gen)
    args = held(a), sa.cuda(), held(b), sb.cuda()
    out = torch.empty(8, 1000, dtype=torch.float32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the handle of the capturing stream is made inside the capture
        fp8.gemm(*args, out=out)
        fp8.gemm(*args, out=out)
    want = torch.from_numpy(ref.values(a, sa) @ ref.values(b, sb).T)
    for _ in range(3):
        out.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu().double(), want)


def test_operators_on_another_stream():
    side = torch.cuda.Stream()
    x = torch.randn(300, 700, device="cuda").to(torch.bfloat16)
    w = torch.randn(64, 700, device="cuda").to(torch.bfloat16)
    wt = torch.ones(700, device="cuda")
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        q, s, h, rstd = fp8.rmsnorm(x, wt, stream=stream)
        qw, sw = fp8.quantize(w, tile=True, stream=stream)
        d = fp8.gemm(q, s, qw, sw, stream=stream)
        dx, dw = fp8.rmsnorm_backward(x, h, wt, rstd, stream=stream)
        side.synchronize()
        q2, s2, h2, rstd2 = fp8.rmsnorm(x, wt)
        qw2, sw2 = fp8.quantize(w, tile=True)
        d2 = fp8.gemm(q2, s2, qw2, sw2)
        dx2, dw2 = fp8.rmsnorm_backward(x, h2, wt, rstd2)
        torch.cuda.synchronize()
        for one, two in ((q.view(torch.uint8), q2.view(torch.uint8)), (d, d2), (dx, dx2), (dw, dw2)):
            assert torch.equal(one, two)


def test_gemm_watchdog_reports_and_recovers():
    gen = torch.Generator().manual_seed(9)
    a, sa = integer_operand(300, 1500, gen)
    b, sb = integer_operand(300, 1500, gen)
    args = held(a), sa.cuda(), held(b), sb.cuda()
    want = torch.from_numpy(ref.values(a, sa) @ ref.values(b, sb).T)
    for cta_group in (1, 2):
        with fp8.Gemm(0, cta_group=cta_group) as g:
            g.set_option("watchdog_ns", 3000000)
            g.set_option("fault_skip_load", 1)
            g.run(*args)
            st, detail = g.device_status()
            assert st == fp8.ERR_DEVICE_TIMEOUT and detail != 0
            g.set_option("fault_skip_load", -1)
            d = g.run(*args, out_dtype=torch.float32)
            assert g.device_status()[0] == fp8.OK
            assert torch.equal(d.cpu().double(), want)


def test_gemm_empty_sizes():
    def operand(R, K):
        q, s = fp8.empty_quantized(R, K, "cuda")
        return q, s
    assert fp8.gemm(*operand(0, 256), *operand(8, 256)).shape == (0, 8)
    assert fp8.gemm(*operand(8, 256), *operand(0, 256)).shape == (8, 0)
    out = torch.full((5, 9), 3.0, device="cuda")
    fp8.gemm(*operand(5, 0), *operand(9, 0), out=out)
    assert bool((out == 0).all())


# ---------------------------------------------------------------- quantiser
def spread_matrix(R, C, seed, dtype):
    """Magnitudes over forty powers of two, zero blocks, a block at 448 exactly and one just above."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=gen) * torch.exp2(torch.randint(-20, 20, (R, 1), generator=gen).float())
    x[::7, : min(C, 128)] = 0
    x[0, 0] = 448.0
    x[R // 2, C - 1] = 450.0
    return x.to(dtype)


def check_quantized(codes, scales, y, tile=False):
    want, e = ref.quantize(y, tile)
    got_e, pad = ref.scale_bytes(scales, y.shape[1])
    assert np.array_equal(got_e, e)
    assert (pad == 127).all()
    got = codes.cpu().float().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


QSHAPES = [(1, 1), (1, 128), (2, 129), (128, 128), (127, 500), (129, 512), (130, 513), (300, 1000), (1, 8192),
           (1000, 3), (257, 4104)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tile", [False, True], ids=["rows", "tiles"])
@pytest.mark.parametrize("shape", QSHAPES, ids=lambda s: "x".join(map(str, s)))
def test_quantize_exact(shape, tile, dtype):
    R, C = shape
    x = spread_matrix(R, C, R * C, dtype)
    if dtype == torch.float32:
        x = x * (1 + 2.0**-12)  # values that bf16 cannot hold
    y = x.double().numpy()
    d = x.cuda()
    q, s = fp8.quantize(d, tile=tile)
    qt, st = fp8.quantize_columns(d, tile=tile)
    check_quantized(q, s, y, tile)
    check_quantized(qt, st, y.T, tile)
    both = fp8.quantize_both(d, tile=tile)
    for one, two in zip(both, (q, s, qt, st)):
        assert torch.equal(one.view(torch.uint8), two.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_quantize_strided_input(dtype):
    big = spread_matrix(200, 700, 3, dtype).cuda()
    for view in (big[:, 1:600], big[3:, 8:], big[::2, :333], big[5:6, 7:]):
        q, s, qt, st = fp8.quantize_both(view)
        check_quantized(q, s, view.cpu().double().numpy())
        check_quantized(qt, st, view.cpu().double().numpy().T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_quantize_infinities_and_nan(dtype):
    x = spread_matrix(140, 300, 4, dtype)
    x[3, 5] = float("inf")
    x[139, 299] = float("-inf")
    x[70, 130] = float("nan")
    x[9, :128] = float("inf")  # a block with nothing finite
    x[10, :128] = torch.finfo(dtype).min  # the type's lowest value
    x[11, :128] = torch.finfo(dtype).tiny
    for tile in (False, True):
        q, s, qt, st = fp8.quantize_both(x.cuda(), tile=tile)
        check_quantized(q, s, x.double().numpy(), tile)
        check_quantized(qt, st, x.double().numpy().T, tile)


def check_near(codes, scales, y, rel):
    """Codes of values known to a relative `rel`: half a step of e4m3 and that error off at most."""
    got = ref.values(codes, scales)
    e, pad = ref.scale_bytes(scales, y.shape[1])
    assert (pad == 127).all()
    amax = ref.block_amax(y, False)
    assert (e >= ref.scale_exponents(amax * (1 - rel))).all() and (e <= ref.scale_exponents(amax * (1 + rel))).all()
    step = np.repeat(np.exp2(e - 127 - 10), 128, 1)[:, : y.shape[1]]
    assert (np.abs(got - y) <= np.abs(y) * ((1 + rel) * 2.0**-4 + rel) + step).all()


@pytest.mark.parametrize("cdtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 70), (130, 129), (500, 640)], ids=lambda s: "x".join(map(str, s)))
def test_quantize_factors(shape, cdtype):
    R, C = shape
    gen = torch.Generator().manual_seed(R)
    x = torch.randn(R, C, generator=gen).to(torch.bfloat16)
    f = torch.rand(R, generator=gen) + 0.1
    w = torch.randn(C, generator=gen).to(cdtype)
    y = x.double().numpy() * f.double().numpy()[:, None] * w.double().numpy()
    qt, st = fp8.quantize_columns(x.cuda(), row_factor=f.cuda(), column_factor=w.cuda())
    check_near(qt, st, y.T, 4 * U)
    q, s = fp8.quantize(x.cuda(), row_factor=f.cuda())
    check_near(q, s, x.double().numpy() * f.double().numpy()[:, None], 4 * U)


def test_quantize_empty():
    q, s = fp8.quantize(torch.empty(0, 300, device="cuda"))
    assert q.shape == (0, 300) and s.shape == (1, 0, 4)


# ---------------------------------------------------------------- norm
NSHAPES = [(1, 1), (1, 128), (3, 7), (5, 256), (2, 1000), (7, 1024), (400, 64), (333, 1032), (2, 4104), (400, 2048),
           (310, 5999), (1, 8192), (320, 8192), (3, 16392), (1, 32768)]


def norm_inputs(R, C, seed, wdtype, residual):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(R, C, generator=gen) * 3).to(torch.bfloat16)
    res = torch.randn(R, C, generator=gen).to(torch.bfloat16) if residual else None
    w = (1 + 0.3 * torch.randn(C, generator=gen)).to(wdtype)
    return x, res, w


def norm_rel(C):
    # the mean square is off by (C + 4) 2u / 2 at most, then five roundings
    return (C + 4) * U + 6 * U


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", NSHAPES, ids=lambda s: "x".join(map(str, s)))
def test_rmsnorm(shape, wdtype, residual):
    R, C = shape
    x, res, w = norm_inputs(R, C, R + C, wdtype, residual)
    q, s, h, rstd = fp8.rmsnorm(x.cuda(), w.cuda(), residual=None if res is None else res.cuda(), eps=1e-5)
    kept = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(h.cpu(), kept)
    y, want = ref.rmsnorm(kept.double().numpy(), w.double().numpy(), 1e-5)
    rel = norm_rel(C)
    assert (np.abs(rstd.cpu().double().numpy() - want) <= rel * want).all()
    check_near(q, s, y, rel)


def test_rmsnorm_in_place_and_strided():
    x, res, w = norm_inputs(20, 700, 1, torch.bfloat16, True)
    want = fp8.rmsnorm(x.cuda(), w.cuda(), residual=res.cuda())
    for which in (0, 1):
        a, b = x.cuda(), res.cuda()
        got = fp8.rmsnorm(a, w.cuda(), residual=b, out_h=(a, b)[which])
        assert got[2].data_ptr() == (a, b)[which].data_ptr()
        for one, two in zip(got, want):
            assert torch.equal(one.contiguous().view(torch.uint8), two.contiguous().view(torch.uint8))
    big, bigr = torch.zeros(40, 709, dtype=torch.bfloat16, device="cuda"), torch.zeros(20, 720, dtype=torch.bfloat16, device="cuda")
    big[::2, 5:705] = x.cuda()
    bigr[:, 8:708] = res.cuda()
    got = fp8.rmsnorm(big[::2, 5:705], w.cuda(), residual=bigr[:, 8:708], out_h=bigr[:, 8:708])
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
    assert torch.equal(got[0].contiguous().view(torch.uint8), want[0].contiguous().view(torch.uint8))
    assert bool((bigr[:, :8] == 0).all()) and bool((bigr[:, 708:] == 0).all())


def test_rmsnorm_zero_and_nonfinite_rows():
    x, _, _ = norm_inputs(6, 512, 2, torch.float32, False)
    x[1] = 0
    x[2, 9] = float("inf")
    x[3, 9] = float("nan")
    q, s, _, rstd = fp8.rmsnorm(x.cuda(), torch.ones(512, device="cuda"), eps=0.0)
    v = q.float().cpu()
    assert bool(torch.isnan(v[1]).all())  # 0 * inf: a zero row without eps has no norm
    assert bool(torch.isnan(v[2, 9])) and bool((v[2, :9] == 0).all()) and bool((v[2, 10:] == 0).all())
    assert bool(torch.isnan(v[3]).all())
    q0, s0, _, _ = fp8.rmsnorm(x.cuda(), torch.ones(512, device="cuda"), eps=1e-6)
    assert bool((q0[1].float() == 0).all()) and bool((s0.view(torch.uint8)[:, 1] == 0).all())
    for r in (0, 4, 5):  # their neighbours are untouched by them
        y, _ = ref.rmsnorm(x[r:r + 1].double().numpy(), np.ones(512), 0.0)
        check_near(q[r:r + 1], s[:, r:r + 1], y, norm_rel(512))


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", NSHAPES, ids=lambda s: "x".join(map(str, s)))
def test_rmsnorm_backward(shape, wdtype, residual):
    R, C = shape
    h, _, w = norm_inputs(R, C, R * C + 1, wdtype, False)
    gen = torch.Generator().manual_seed(R * C + 2)
    dy = (torch.randn(R, C, generator=gen) * 0.01).to(torch.bfloat16)
    dres = (torch.randn(R, C, generator=gen) * 0.01).to(torch.bfloat16) if residual else None
    rstd = (1.0 / (h.double().square().mean(1) + 1e-6).sqrt()).float()
    dx, dw = fp8.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), None if dres is None else dres.cuda())
    hn, wn, dyn, rn = (t.double().numpy() for t in (h, w, dy, rstd))
    want, want_w = ref.rmsnorm_backward(dyn, hn, wn, rn, None if dres is None else dres.double().numpy())
    n, g = hn * rn[:, None], dyn * wn
    size = rn[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    tol = 2.0**-8 * np.abs(want) + (C + 16) * 2 * U * size
    assert (np.abs(dx.cpu().double().numpy() - want) <= tol).all()
    tol_w = (R + 16) * 2 * U * np.abs(dyn * n).sum(0)
    assert (np.abs(dw.cpu().double().numpy() - want_w) <= tol_w).all()
    again = fp8.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), None if dres is None else dres.cuda())
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


# several rows to each group of threads, in every layout of the gradient's rows: aligned and
# not, a warp's, part of a CTA's and a CTA's, up to four vectors of 8 columns a thread
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("shape", [(6000, 75), (3000, 901), (2500, 1808), (1000, 4001), (700, 4500), (500, 6634),
                                   (470, 9001), (470, 12288), (500, 16383)], ids=lambda s: "x".join(map(str, s)))
def test_rmsnorm_backward_many_rows(shape, residual):
    test_rmsnorm_backward(shape, torch.float32, residual)


def test_rmsnorm_backward_against_differences():
    R, C, eps = 3, 96, 1e-6
    h, _, w = norm_inputs(R, C, 11, torch.float32, False)
    gen = torch.Generator().manual_seed(12)
    dy = torch.randn(R, C, generator=gen).to(torch.bfloat16)
    hn, wn, dyn = (t.double().numpy() for t in (h, w, dy))
    rstd = torch.from_numpy(ref.rmsnorm(hn, wn, eps)[1]).float()
    dx, dw = (t.cpu().double().numpy() for t in fp8.rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda()))

    def loss(hv, wv):
        return (dyn * ref.rmsnorm(hv, wv, eps)[0]).sum()

    rng = np.random.RandomState(0)
    for _ in range(20):
        v, t = rng.randn(R, C), 1e-5
        slope = (loss(hn + t * v, wn) - loss(hn - t * v, wn)) / (2 * t)
        # bf16 dx: 2^-9 of each term, and the differences' own error below that
        assert abs(slope - (dx * v).sum()) <= 2.0**-8 * np.abs(dx * v).sum()
        u = rng.randn(C)
        slope = (loss(hn, wn + t * u) - loss(hn, wn - t * u)) / (2 * t)
        assert abs(slope - (dw * u).sum()) <= 1e-5 * np.abs(dw * u).sum()


def test_rmsnorm_empty():
    w = torch.ones(300, device="cuda")
    x = torch.empty(0, 300, dtype=torch.bfloat16, device="cuda")
    q, s, h, rstd = fp8.rmsnorm(x, w)
    assert q.shape == (0, 300) and rstd.shape == (0,)
    dx, dw = fp8.rmsnorm_backward(x, x, w, rstd)
    assert dx.shape == (0, 300) and bool((dw == 0).all())


# ---------------------------------------------------------------- refusals
def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    q, s = fp8.quantize(x)
    with pytest.raises(ValueError, match="contract"):
        fp8.gemm(q, s, *fp8.quantize(x[:, :128]))
    with pytest.raises(ValueError, match="a_scales"):
        fp8.gemm(q, s[:, :2], q, s)
    with pytest.raises(TypeError, match="float8"):
        fp8.gemm(x, s, q, s)
    with pytest.raises(ValueError, match="out must be"):
        fp8.gemm(q, s, q, s, out=torch.empty(4, 5, device="cuda"))
    with pytest.raises(TypeError, match="bf16 or fp32"):
        fp8.gemm(q, s, q, s, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA device"):
        fp8.quantize(x.cpu())
    with pytest.raises(TypeError, match="bf16 or fp32"):
        fp8.quantize(x.half())
    with pytest.raises(ValueError, match="contiguous rows"):
        fp8.quantize(x.t())
    with pytest.raises(ValueError, match="row_factor"):
        fp8.quantize(x, row_factor=w)
    with pytest.raises(ValueError, match="weight"):
        fp8.rmsnorm(x, w[:100])
    with pytest.raises(ValueError, match="out_h"):
        fp8.rmsnorm(x, w, out_h=x)
    with pytest.raises(TypeError, match="bf16"):
        fp8.rmsnorm(x.float(), w)
    wide = torch.zeros(1, fp8.NORM_MAX_COLUMNS + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fp8.Fp8Error, match="unsupported"):
        fp8.rmsnorm(wide, torch.ones(wide.shape[1], device="cuda"))
    # a pitch that TMA cannot step over
    odd = torch.zeros(4, 264, dtype=torch.uint8, device="cuda")[:, :256]
    with pytest.raises(fp8.Fp8Error, match="alignment"):
        fp8.gemm(odd.view(torch.float8_e4m3fn), s, q, s)
    shifted = torch.zeros(4 * 256 + 8, dtype=torch.uint8, device="cuda")[8:].view(4, 256)
    with pytest.raises(fp8.Fp8Error, match="alignment"):
        fp8.gemm(shifted.view(torch.float8_e4m3fn), s, q, s)
    with fp8.Gemm(0) as g:
        with pytest.raises(fp8.Fp8Error, match="invalid"):
            g.set_option("width", 40)
        with pytest.raises(fp8.Fp8Error, match="not planned"):
            g.info()
        g.set_option("width", 48)  # not a multiple of 32: only as the sole tile
        with pytest.raises(fp8.Fp8Error, match="unsupported"):
            g.plan(500, 500, 256)
