"""Long sums whose results stay in fp32, or go to 8 bits: added up in segments, as exact as short ones, in
every kernel variant; and the launches of these kernels that give up."""
from __future__ import annotations

import itertools

import numpy as np
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
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(bf)


def ints(*shape, seed=0, top=2):
    return torch.randint(-top, top + 1, shape, generator=torch.Generator().manual_seed(seed)).to(bf).cuda()


VARIANTS = {
    "one": dict(cta_group=1, transposed=1, split=0, stream=2),
    "pair": dict(cta_group=2, transposed=1, split=0, stream=2),
    "one-t": dict(cta_group=1, transposed=2, split=0, stream=2),
    "pair-t": dict(cta_group=2, transposed=2, split=0, stream=2),
    "ranges": dict(cta_group=1, transposed=1, split=2, stream=2),
    "pair-ranges-t": dict(cta_group=2, transposed=2, split=2, stream=2),
    "clusters": dict(cta_group=1, transposed=1, split=1, stream=2),
    "clusters-t": dict(cta_group=1, transposed=2, split=1, stream=2),
    "auto": dict(),
}
variants = pytest.mark.parametrize("variant", VARIANTS.values(), ids=VARIANTS.keys())

# An accumulator takes a segment of products, 512 for an fp32 result and 1024 for codes, 16 at a time: n = 32 or 64
# additions, the j-th of which loses at most 2^-23 of the sum so far.  With independent terms of one size s that sum
# is sqrt(16 j) s, root of mean squares, so a segment is off by at most 2^-23 s 4 (sqrt(1) + ... + sqrt(n)), and by
# that over sqrt(16 n) of its own size (21.9 units of 2^-23, or 43.1); and, the segments' errors being of products of
# their own, so is their sum, whatever its length.  The segments and pieces are then added in fp32, each addition off by
# half a unit at most.
def rms_bound(K: int, segment: int = 512) -> float:
    n = segment // 16
    return 2.0**-23 * 4 * sum(j**0.5 for j in range(1, n + 1)) / segment**0.5 + 2.0**-24 * (K / segment + 32) ** 0.5


def off(got, want) -> float:
    return float((got.double() - want).norm() / want.norm())


# ------------------------------------------------------------------ fp32 results
@variants
@pytest.mark.parametrize("K", [4096, 16384, 32768])
def test_linear_is_as_exact_as_for_short_sums(variant, K):
    x, w = randn(256, K, seed=1), randn(384, K, seed=2)
    with ffn.options(**variant):
        y = ffn.linear(x, w, out_dtype=torch.float32)
    assert off(y, x.double() @ w.double().T) <= rms_bound(K)


@pytest.mark.parametrize("M", [1, 8, 16, 32])
@pytest.mark.parametrize("N,K", [(8192, 16384), (384, 65536)])
def test_few_tokens_are_as_exact(M, N, K):
    x, w = randn(M, K, seed=1), randn(N, K, seed=2)
    want = x.double() @ w.double().T
    for options in (dict(stream=1), dict(stream=2), dict()):
        with ffn.options(**options):
            assert off(ffn.linear(x, w, out_dtype=torch.float32), want) <= rms_bound(K)


@pytest.mark.parametrize("options", [dict(together=1), dict(together=2), dict(together=2, cta_group=1, split=0), dict()],
                         ids=["together", "apart", "whole", "auto"])
@pytest.mark.parametrize("M", [4096, 16384])
def test_weight_gradients_are_as_exact(options, M):
    x, w, dy = randn(M, 256, seed=1), randn(384, 256, seed=2), randn(M, 384, seed=3)
    with ffn.options(**options):
        dx, dw, _ = ffn.linear_backward(dy, x, w, grad_dtype=torch.float32)
    assert off(dw, dy.double().T @ x.double()) <= rms_bound(M)
    want, mag = ref.product(dy, w.T)
    assert ref.close(dx, want.cpu(), ref.sum_error(384) * mag.cpu())
    wd, g, u = randn(256, 384, seed=4), randn(M, 384, seed=5), randn(M, 384, seed=6)
    with ffn.options(**options):
        got = ffn.gated_backward(x, x, (g, u), w, w, wd, activation=None, grad_dtype=torch.float32)
    # without an activation du = dh g and h = g u, rounded; the last product's operands are known
    assert off(got[3], x.double().T @ (g.double() * u.double()).to(bf).double()) <= rms_bound(M)


@variants
@pytest.mark.parametrize("M,N,K", [(300, 257, 513), (129, 200, 1000), (37, 600, 4100), (1, 33, 9000), (513, 385, 2048)])
def test_long_integer_sums_are_exact(variant, M, N, K):
    x, w, b, r = ints(M, K, seed=1), ints(N, K, seed=2), ints(N, seed=3, top=9), ints(M, N, seed=4, top=9)
    z = x.double() @ w.double().T + b.double()
    with ffn.options(**variant):
        plain = ffn.linear(x, w, out_dtype=torch.float32)
        y, zs = ffn.linear(x, w, b, "relu", r, save=True, out_dtype=torch.float32)
        base = torch.full((M, N + 5), 7.0, device="cuda")
        ffn.linear(x, w, b.float(), None, r, out=base[:, 3:3 + N])
    assert plain.double().equal(z - b.double())
    assert y.double().equal(z.clamp_min(0) + r.double()) and zs.equal(z.to(bf))
    assert base[:, 3:3 + N].double().equal(z + r.double())
    assert bool((base[:, :3] == 7).all()) and bool((base[:, 3 + N:] == 7).all())


@pytest.mark.parametrize("width", [32, 64, 96, 160, 192, 224, 256])
@pytest.mark.parametrize("cta_group,transposed", [(1, 1), (1, 2), (2, 1), (2, 2)])
def test_widths_of_long_sums(width, cta_group, transposed):
    x, w = ints(700, 1600, seed=1), ints(650, 1600, seed=2)
    want = x.double() @ w.double().T
    with ffn.options(width=width, cta_group=cta_group, transposed=transposed, stream=2):
        y = ffn.linear(x, w, out_dtype=torch.float32)
        # wider ones hold no sums in registers, but for an SM pair's: the widest that does stands for them
        assert ffn.plan_info()["width"] == (width if (cta_group, transposed) == (2, 1) else min(width, 192))
        assert y.double().equal(want)
        assert ffn.linear(x, w).equal(want.to(bf)) and ffn.plan_info()["width"] == width


@pytest.mark.parametrize("M", [1, 7, 16, 25, 32])
@pytest.mark.parametrize("N,K", [(5, 12000), (1000, 8200), (8192, 4104), (38912, 1096)])
def test_few_tokens_long_integer_sums_are_exact(M, N, K):
    x, w, r = ints(M, K, seed=1), ints(N, K, seed=2), ints(M, N, seed=4, top=9)
    with ffn.options(stream=1):
        y = ffn.linear(x, w, residual=r, out_dtype=torch.float32)
        assert ffn.plan_info()["tiles"] == 0
    assert y.double().equal(x.double() @ w.double().T + r.double())


@pytest.mark.parametrize("options", [dict(together=1), dict(together=1, cta_group=1), dict(together=1, cta_group=2, width=256),
                                     dict(together=2), dict(together=2, split=2), dict(together=2, transposed=2), dict()],
                         ids=lambda o: "-".join(f"{k}{v}" for k, v in o.items()) or "auto")
@pytest.mark.parametrize("M", [513, 2000, 5003])
def test_gradients_of_many_tokens_are_exact(options, M):
    N, K = 264, 328
    x, w, dy = ints(M, K, seed=1), ints(N, K, seed=2), ints(M, N, seed=3)
    with ffn.options(**options):
        dx, dw, db = ffn.linear_backward(dy, x, w, bias=True, grad_dtype=torch.float32)
    assert dx.equal((dy.double() @ w.double()).to(bf)) and db.double().equal(dy.double().sum(0))
    assert dw.double().equal(dy.double().T @ x.double())
    C, F = 136, 264
    x, wg, wu, wd = ints(M, C, seed=1, top=1), ints(F, C, seed=2, top=1), ints(F, C, seed=3, top=1), ints(72, F, seed=4, top=1)
    dy, g, u = ints(M, 72, seed=5, top=1), ints(M, F, seed=6), ints(M, F, seed=7)
    with ffn.options(**options):
        got = ffn.gated_backward(dy, x, (g, u), wg, wu, wd, activation="relu", grad_dtype=torch.float32)
    want = ref.gated_backward(*(t.cpu() for t in (dy, x, g, u, wg, wu, wd)), "relu")
    assert got[0].cpu().equal(want[0].to(bf))
    for a, b in zip(got[1:], want[1:]):
        assert a.cpu().double().equal(b)


# ------------------------------------------------------------------ 8 bits
@pytest.mark.parametrize("M,C,F", [(1, 600, 1), (20, 2056, 128), (64, 5000, 300), (65, 1024, 257), (300, 513, 1025),
                                   (200, 4096, 392), (4100, 520, 650)])
@pytest.mark.parametrize("cta_group", [0, 1, 2])
def test_checkpoints_of_long_integer_sums_are_exact(M, C, F, cta_group):
    x, wg, wu = ints(M, C, seed=1, top=1), ints(F, C, seed=2, top=1), ints(F, C, seed=3, top=1)
    with ffn.options(cta_group=cta_group):
        h, (gc, gs, uc, us) = ffn.gated(x, wg, wu, save="e4m3", activation="relu")
    g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
    # a product of two sums of fp32's whole numbers: rounded to fp32, then to bf16
    assert h.equal((g.clamp_min(0).float() * u.float()).to(bf))
    for codes, scales, v in ((gc, gs, g), (uc, us, u)):
        qc, qs = fp8.quantize(v.float())
        assert qc.view(torch.uint8).equal(codes.view(torch.uint8)) and qs.view(torch.uint8).equal(scales.view(torch.uint8))
    want, e = fp8ref.quantize(g[:70].cpu().numpy())
    got, padding = fp8ref.scale_bytes(gs[:, :70].contiguous(), F)
    assert (got == e).all() and (padding == 127).all() and gc[:70].cpu().double().equal(torch.from_numpy(want))


@pytest.mark.parametrize("cta_group", [0, 1, 2])
@pytest.mark.parametrize("C", [2048, 16384])
def test_codes_are_those_of_the_exact_sums(C, cta_group):
    """A code rounds to the other side where a tie lies between the sum and the exact one: for a share of
    |error| / step of the values, step being the distance of two codes there."""
    M, F = 256, 512
    x, wg, wu = randn(M, C, seed=1), randn(F, C, seed=2), randn(F, C, seed=3)
    with ffn.options(cta_group=cta_group):
        _, saved = ffn.gated(x, wg, wu, save="e4m3")
    other = limit = 0.0
    for i, w in ((0, wg), (2, wu)):
        v = (x.double() @ w.double().T).cpu()
        codes, e = fp8ref.quantize(v.numpy())
        scale = np.repeat(np.exp2(e - 127), 128, 1)[:, :F]
        got = fp8ref.values(saved[i].cpu(), saved[i + 1].cpu())
        other += (got != codes * scale).sum()
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v.numpy() / scale), 2.0**-6))) - 3) * scale
        limit += (rms_bound(C, 1024) * float(v.square().mean().sqrt()) / step).sum()
    assert other <= limit + 4 * limit**0.5


def test_values_that_are_not_finite_stay_in_their_rows():
    M, F, C = 70, 300, 2056
    x, w = randn(M, C, seed=1), randn(F, C, seed=2)
    x[3, 5], x[7, 2000], w[9, C - 1] = float("inf"), float("nan"), float("-inf")
    bad = torch.zeros(M, F, dtype=torch.bool, device="cuda")
    bad[3], bad[7], bad[:, 9] = True, True, True
    y = ffn.linear(x, w, out_dtype=torch.float32)
    h, (gc, gs, _, _) = ffn.gated(x, w, w, save="e4m3")
    for t in (y, h, torch.from_numpy(fp8ref.values(gc.cpu(), gs.cpu())).cuda()):
        assert bool(torch.isfinite(t[~bad]).all()) and not bool(torch.isfinite(t[bad]).any())


# ------------------------------------------------------------------ launches that give up
@variants
def test_a_launch_may_give_up_at_any_load(variant):
    x, w = ints(200, 6000, seed=1), ints(640, 6000, seed=2)
    want = x.double() @ w.double().T
    variant = dict(variant, stream=2)
    for skip in (0, 1, 2, 3, 7, 8, 9, 15, 16, 17, 33):
        with ffn.options(watchdog_ns=4000000, fault_skip_load=skip, **variant):
            ffn.linear(x, w, out_dtype=torch.float32)
            st, _ = ffn.device_status()
        assert st in (ffn.ERR_DEVICE_TIMEOUT, ffn.OK)  # OK: no CTA has that many loads
        assert st == ffn.ERR_DEVICE_TIMEOUT or skip > 1
        with ffn.options(**variant):
            assert ffn.linear(x, w, out_dtype=torch.float32).double().equal(want)
        assert ffn.device_status() == (ffn.OK, 0)


def test_a_launch_to_8_bits_may_give_up():
    x, w = ints(200, 6000, seed=1), ints(640, 6000, seed=2)
    for cta_group, skip in itertools.product((1, 2), (0, 1, 7, 8, 9, 16, 20, 40, 93)):
        with ffn.options(cta_group=cta_group):
            want = ffn.gated(x, w, w, "relu", save="e4m3")
        with ffn.options(cta_group=cta_group, watchdog_ns=4000000, fault_skip_load=skip):
            ffn.gated(x, w, w, "relu", save="e4m3")
            assert ffn.device_status()[0] == ffn.ERR_DEVICE_TIMEOUT
        with ffn.options(cta_group=cta_group):
            got = ffn.gated(x, w, w, "relu", save="e4m3")
        assert got[0].equal(want[0])
        assert all(a.view(torch.uint8).equal(b.view(torch.uint8)) for a, b in zip(got[1], want[1]))
        assert ffn.device_status() == (ffn.OK, 0)


def test_products_of_one_launch_may_give_up():
    x, w, dy = ints(2000, 640, seed=1), ints(300, 640, seed=2), ints(2000, 300, seed=3)
    for cta_group, skip in itertools.product((1, 2), (0, 1, 8, 9, 17)):
        with ffn.options(together=1, cta_group=cta_group, watchdog_ns=4000000, fault_skip_load=skip):
            ffn.linear_backward(dy, x, w, grad_dtype=torch.float32)
            assert ffn.plan_info()["products"] == 2
            assert ffn.device_status()[0] == ffn.ERR_DEVICE_TIMEOUT
        with ffn.options(together=1, cta_group=cta_group):
            dx, dw, _ = ffn.linear_backward(dy, x, w, grad_dtype=torch.float32)
        assert dx.equal((dy.double() @ w.double()).to(bf)) and dw.double().equal(dy.double().T @ x.double())
        assert ffn.device_status() == (ffn.OK, 0)


# ------------------------------------------------------------------ calls at once
def test_calls_at_once_on_streams_of_their_own():
    x, w = ints(20, 6000, seed=1), ints(2560, 6000, seed=2)
    tall = ints(300, 6000, seed=3)
    want = [(t.double() @ w.double().T).float() for t in (x, tall)]
    split = dict(cta_group=1, transposed=2, width=32, split=2, stream=2)  # tiles meet through global memory
    with ffn.options(cta_group=1):
        codes = ffn.gated(tall, w, w, "relu", save="e4m3")
    streams = [torch.cuda.Stream(priority=-1), torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], [], []]
    for _ in range(20):
        with ffn.options(**split):
            got[0].append(ffn.linear(x, w, out_dtype=torch.float32, stream=streams[0]))
        with ffn.options(cta_group=2, transposed=1, width=64, split=2):
            got[1].append(ffn.linear(tall, w, out_dtype=torch.float32, stream=streams[1]))
        got[2].append(ffn.gated(tall, w, w, "relu", save="e4m3", stream=streams[2]))
    assert ffn.device_status() == (ffn.OK, 0)
    for a, e in zip(got, want):
        assert all(t.equal(e) for t in a)
    for h, saved in got[2]:
        assert h.equal(codes[0])
        assert all(a.view(torch.uint8).equal(b.view(torch.uint8)) for a, b in zip(saved, codes[1]))


def test_graphs_replayed_at_once_share_no_workspace():
    work = [(ints(20, 6000, seed=s), ints(2560, 6000, seed=s + 1)) for s in (1, 5)]
    graphs, outs = [], []
    with ffn.options(cta_group=1, transposed=2, width=32, split=2, stream=2):
        for x, w in work:
            graphs.append(torch.cuda.CUDAGraph())
            outs.append(torch.empty(20, 2560, device="cuda"))
            torch.cuda.synchronize()
            with torch.cuda.graph(graphs[-1]):
                for _ in range(8):
                    ffn.linear(x, w, out=outs[-1])
        assert ffn.plan_info()["split_tiles"] > 0
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for o in outs:
            o.fill_(0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, (x, w) in zip(outs, work):
            assert o.double().equal(x.double() @ w.double().T)
