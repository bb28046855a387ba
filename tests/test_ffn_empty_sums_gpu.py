"""Empty sums of more tiles than SMs, through the C ABI: results start out filled with a value that no
result has, so that what a launch leaves unwritten cannot pass for zero."""
from __future__ import annotations

import ctypes

import pytest
import torch

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


def sentinel(*shape, dtype=bf):
    return torch.full(shape, 7.0, dtype=dtype, device="cuda")


def matrix(t):
    return ffn.Matrix(t.data_ptr(), max(t.stride(0), 1))


def call(name, **fields):
    lib, need, args = ffn.load(), ctypes.c_int64(), getattr(ffn, "".join(w.title() for w in name.split("_")) + "Args")(**fields)
    assert getattr(lib, f"ffn_{name}_workspace")(ctypes.byref(args), ctypes.byref(need)) == ffn.OK
    work = torch.full((max(need.value, 1),), 255, dtype=torch.uint8, device="cuda")
    assert getattr(lib, f"ffn_{name}")(ctypes.byref(args), work.data_ptr(), need.value,
                                       torch.cuda.current_stream().cuda_stream) == ffn.OK
    torch.cuda.synchronize()


OPTIONS = [dict(), dict(transposed=1), dict(transposed=2), dict(transposed=2, cta_group=2), dict(split=2), dict(split=0)]


@pytest.mark.parametrize("options", OPTIONS, ids=lambda o: "-".join(f"{k}{v}" for k, v in o.items()) or "auto")
@pytest.mark.parametrize("M,N", [(281, 12248), (1675, 1886), (300, 8192), (8192, 300), (4096, 520)])
def test_results_are_written(M, N, options):
    x, w = sentinel(M, 0), sentinel(N, 0)
    with ffn.options(**options):
        for act in (0, 2):
            h, g, u = sentinel(M, N), sentinel(M, N), sentinel(M, N)
            call("gated", M=M, F=N, C=0, x=matrix(x), w_gate=matrix(w), w_up=matrix(w), activation=act, h=matrix(h),
                 g=matrix(g), u=matrix(u))
            assert not h.any() and not g.any() and not u.any()
        h = sentinel(M, N)
        pitch = -(-N // 128) * 128
        codes, scales = sentinel(2, M, pitch).to(torch.uint8), sentinel(2, -(-N // 512), M, 4).to(torch.uint8)
        q = [ffn.Quantized(codes[i].data_ptr(), pitch, scales[i].data_ptr()) for i in (0, 1)]
        call("gated", M=M, F=N, C=0, x=matrix(x), w_gate=matrix(w), w_up=matrix(w), activation=2, h=matrix(h), qg=q[0],
             qu=q[1])
        assert not h.any() and not codes[:, :, :N].any() and not bool((scales == 7).any())
        bias = torch.arange(N, device="cuda", dtype=torch.float32) % 100
        r = torch.ones(M, N, dtype=bf, device="cuda")
        y, z = sentinel(M, N, dtype=torch.float32), sentinel(M, N)
        call("linear", M=M, N=N, K=0, x=matrix(x), weight=matrix(w), bias=bias.data_ptr(), bias_type=1, residual=matrix(r),
             y=matrix(y), y_type=1, z=matrix(z))
        assert y.equal((bias + 1).expand(M, N)) and z.equal(bias.to(bf).expand(M, N))


@pytest.mark.parametrize("options", [dict(), dict(together=1), dict(together=2), dict(transposed=2)],
                         ids=["auto", "together", "apart", "transposed"])
def test_gradients_of_empty_sums_are_written(options):
    M, C, F = 4100, 2600, 4096
    x, w, wd = sentinel(M, C), sentinel(F, C), sentinel(C, F)
    no_rows, none = ffn.Matrix(x.data_ptr(), F), ffn.Matrix(None, 0)
    with ffn.options(**options):
        # no tokens: the weights' gradients are zero
        for dtype, kind in ((bf, 0), (torch.float32, 1)):
            dw, db = sentinel(F, C, dtype=dtype), sentinel(F, dtype=torch.float32)
            call("linear_backward", M=0, N=F, K=C, dy=no_rows, x=no_rows, weight=matrix(w), dx=none, dweight=matrix(dw),
                 dweight_type=kind, dbias=db.data_ptr())
            assert not dw.any() and not db.any()
            outs = [sentinel(F, C, dtype=dtype), sentinel(F, C, dtype=dtype), sentinel(C, F, dtype=dtype)]
            call("gated_backward", M=0, F=F, C=C, N=C, dy=no_rows, x=no_rows, g=no_rows, u=no_rows, w_gate=matrix(w),
                 w_up=matrix(w), w_down=matrix(wd), activation=2, dweight_type=kind, dx=none, dw_gate=matrix(outs[0]),
                 dw_up=matrix(outs[1]), dw_down=matrix(outs[2]))
            assert not any(t.any() for t in outs)
        # no columns of the result: dx is zero
        dx = sentinel(M, C)
        call("linear_backward", M=M, N=0, K=C, dy=none, x=matrix(x), weight=none, dx=matrix(dx), dweight=none)
        assert not dx.any()
        # dh is an empty sum, so dg and du are zero, and what is made of them
        few, many = 300, 8192
        wide, g = sentinel(many, C), torch.ones(few, many, dtype=bf, device="cuda")
        dx, dwg, dwu = sentinel(few, C), sentinel(many, C), sentinel(many, C)
        call("gated_backward", M=few, F=many, C=C, N=0, dy=none, x=matrix(x), g=matrix(g), u=matrix(g), w_gate=matrix(wide),
             w_up=matrix(wide), w_down=none, activation=2, dx=matrix(dx), dw_gate=matrix(dwg), dw_up=matrix(dwu),
             dw_down=none)
        assert not dx.any() and not dwg.any() and not dwu.any()
