"""Which kernel the gradients of few tokens run on: where they are to be streamed, they are, and their results are
the references'; where rows do not allow it, they run on the other one."""
from __future__ import annotations

import ctypes

import pytest
import torch

import ffn_reference as ref
from warp_specialized_tma_gb300 import ffn

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)
    yield
    assert ffn.device_status() == (ffn.OK, 0)


def ints(*shape, seed=0, top=2):
    return torch.randint(-top, top + 1, shape, generator=torch.Generator().manual_seed(seed)).to(bf)


def rows(t, pitch, offset=0):
    """t on the GPU, rows `pitch` elements apart."""
    view = torch.zeros(t.shape[0] * pitch + offset, dtype=bf, device="cuda").as_strided(t.shape, (pitch, 1), offset)
    view.copy_(t)
    return view


def matrix(t):
    return ffn.Matrix(t.data_ptr(), t.stride(0))


def call(name, args):
    lib, need = ffn.load(), ctypes.c_int64()
    assert getattr(lib, f"ffn_{name}_workspace")(ctypes.byref(args), ctypes.byref(need)) == ffn.OK
    work = torch.empty(max(need.value, 1), dtype=torch.uint8, device="cuda")
    assert getattr(lib, f"ffn_{name}")(ctypes.byref(args), work.data_ptr(), need.value,
                                       torch.cuda.current_stream().cuda_stream) == ffn.OK
    torch.cuda.synchronize()
    return ffn.plan_info()["tiles"]  # of the last product: none where the weights are streamed


def eights(n):
    return -(-n // 8) * 8


@pytest.mark.parametrize("M", [1, 2, 8, 9, 16, 17])
@pytest.mark.parametrize("N,K", [(1, 8), (15, 1), (33, 584), (500, 4096), (1003, 7), (40, 20000), (2040, 8200)])
def test_input_gradients(M, N, K):
    w, dy = ints(N, K, seed=2), ints(M, N, seed=3)
    want = (dy.double() @ w.double()).to(bf)
    for pitch, streamed in ((eights(K) + 8, M <= 16), (eights(K) + 9, M <= 16 and N == 1)):
        held, weight = rows(dy, eights(N)), rows(w, pitch)
        dx = torch.zeros(M, K, dtype=bf, device="cuda")
        a = ffn.LinearBackwardArgs(M=M, N=N, K=K, dy=matrix(held), weight=matrix(weight), dx=matrix(dx))
        with ffn.options(stream=1):
            assert (call("linear_backward", a) == 0) == streamed
        assert dx.cpu().equal(want)
        with ffn.options(stream=2):
            assert call("linear_backward", a) > 0
        assert dx.cpu().equal(want)


@pytest.mark.parametrize("save", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,C,F,N", [(1, 8, 8, 8), (3, 40, 1032, 24), (16, 520, 136, 1000), (9, 1000, 5000, 33), (17, 40, 136, 24)])
def test_gated_gradients(M, C, F, N, save):
    x, wg, wu, wd = ints(M, C, seed=1, top=1), ints(F, C, seed=2, top=1), ints(F, C, seed=3, top=1), ints(N, F, seed=4, top=1)
    dy, g, u = ints(M, N, seed=5, top=1), ints(M, F, seed=6), ints(M, F, seed=7)
    want = ref.gated_backward(dy, x, g, u, wg, wu, wd, "relu")[0].to(bf)
    ts = {k: rows(t, eights(t.shape[1])) for k, t in dict(dy=dy, x=x, w_gate=wg, w_up=wu, w_down=wd).items()}
    saved, keep = {}, []
    for k, t in (("g", g), ("u", u)):
        if save == "bf16":
            keep.append(t.cuda())
            saved[k] = matrix(keep[-1])
        else:
            pitch = -(-F // 16) * 16
            codes = torch.zeros(M, pitch, dtype=torch.uint8, device="cuda")
            codes[:, :F] = t.float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            ones = torch.full((-(-F // 512), M, 4), 127, dtype=torch.uint8, device="cuda")
            keep += codes, ones
            saved["q" + k] = ffn.Quantized(codes.data_ptr(), pitch, ones.data_ptr())
    dx = torch.zeros(M, C, dtype=bf, device="cuda")
    fields = dict(M=M, F=F, C=C, N=N, activation=1, **{k: matrix(t) for k, t in ts.items()}, **saved)
    for stream in (1, 2):
        with ffn.options(stream=stream):
            # nothing asked for: dg, du and h alone; then dx of them
            for more in ({}, dict(dx=matrix(dx))):
                tiles = call("gated_backward", ffn.GatedBackwardArgs(**fields, **more))
                assert (tiles == 0) == (stream == 1 and M <= 16)
        assert dx.cpu().equal(want)
        dx.zero_()
