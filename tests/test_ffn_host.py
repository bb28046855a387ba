"""Host-only checks of the feed-forward operators: the library builds, loads without a GPU and
exports what include/ffn_ops.h declares; argument checks and status strings behave as documented;
the kernels' work split; the 64-bit references of the GPU tests against differences.  No kernel
runs here."""
from __future__ import annotations

import ctypes
import os
import re
import subprocess

import pytest
import torch

import ffn_reference as ref
import fp8_reference as fp8ref
from warp_specialized_tma_gb300 import build as libbuild
from warp_specialized_tma_gb300 import feedforward, ffn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ffn_ops.h")
bf = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return ffn.load()


def test_the_abi_is_what_is_exported_and_bound(lib):
    names = set(re.findall(r"FFN_API\s+[\w\s\*]+?\b(ffn_\w+)\s*\(", open(HEADER).read()))
    assert names == set(ffn._SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", ffn.LIB_PATH], capture_output=True, text=True)
    if out.returncode != 0:
        pytest.skip("nm unavailable")
    syms = {line.split()[-1] for line in out.stdout.splitlines() if line.strip()}
    assert {s for s in syms if not s.startswith("_")} == names


def test_strings(lib):
    assert lib.ffn_strerror(0) == b"ok"
    for st in range(-7, 0):
        assert lib.ffn_strerror(st) not in (b"", b"unknown status")
    assert lib.ffn_strerror(-99) == b"unknown status"
    assert "sm_103a" in ffn.version()


def test_mirrors_of_the_header():
    text = open(HEADER).read()
    kinds = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "ffn_matrix": ffn.Matrix,
             "ffn_quantized": ffn.Quantized, "const void *": ctypes.c_void_p, "float *": ctypes.c_void_p,
             "void *": ctypes.c_void_p}
    for struct, mirror in (("ffn_plan_info_t", ffn.PlanInfo), ("ffn_matrix", ffn.Matrix), ("ffn_quantized", ffn.Quantized),
                           ("ffn_linear_args", ffn.LinearArgs), ("ffn_linear_backward_args", ffn.LinearBackwardArgs),
                           ("ffn_gated_args", ffn.GatedArgs), ("ffn_gated_backward_args", ffn.GatedBackwardArgs)):
        body = re.search(r"typedef struct \w+ \{([^}]*)\} %s;" % struct, text).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = []
        for line in body.split(";"):
            m = re.match(r"\s*(const void \*|void \*|float \*|\w+)\s*(.+)", line.strip(), re.S)
            if m:
                fields += [(name.strip(), kinds[m.group(1)]) for name in m.group(2).split(",")]
        assert [(n, c) for n, c in mirror._fields_] == fields, struct
    body = re.search(r"typedef enum ffn_option \{(.*?)\} ffn_option;", text, re.S).group(1)
    assert {n.lower(): int(v) for n, v in re.findall(r"FFN_OPT_(\w+)\s*=\s*(\d+)", body)} == ffn.OPTIONS
    body = re.search(r"typedef enum ffn_activation \{(.*?)\} ffn_activation;", text, re.S).group(1)
    want = {n.lower(): int(v) for n, v in re.findall(r"FFN_ACT_(\w+)\s*=\s*(\d+)", body)}
    assert want == {"none" if k is None else k: v for k, v in ffn.ACTIVATIONS.items()}


def linear_args(**over):
    a = ffn.LinearArgs(M=4, N=16, K=8, x=ffn.Matrix(0x10000, 8), weight=ffn.Matrix(0x20000, 8), y=ffn.Matrix(0x30000, 16))
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(M=-1), ffn.ERR_INVALID_ARG),
    (dict(K=1 << 31), ffn.ERR_INVALID_ARG),
    (dict(activation=5), ffn.ERR_INVALID_ARG),
    (dict(activation=-1), ffn.ERR_INVALID_ARG),
    (dict(y_type=2), ffn.ERR_INVALID_ARG),
    (dict(bias=0x40000, bias_type=3), ffn.ERR_INVALID_ARG),
    (dict(bias=0x40001), ffn.ERR_ALIGNMENT),
    (dict(bias=0x40002, bias_type=1), ffn.ERR_ALIGNMENT),
    (dict(x=ffn.Matrix(None, 8)), ffn.ERR_INVALID_ARG),
    (dict(x=ffn.Matrix(0x10001, 8)), ffn.ERR_INVALID_ARG),
    (dict(x=ffn.Matrix(0x10000, 7)), ffn.ERR_INVALID_ARG),        # pitch below the width
    (dict(weight=ffn.Matrix(0x20000, 7)), ffn.ERR_INVALID_ARG),
    (dict(y=ffn.Matrix(None, 16)), ffn.ERR_INVALID_ARG),
    (dict(y=ffn.Matrix(0x30000, 15)), ffn.ERR_INVALID_ARG),
    (dict(y=ffn.Matrix(0x30002, 16), y_type=1), ffn.ERR_INVALID_ARG),
    (dict(residual=ffn.Matrix(0x40000, 15)), ffn.ERR_INVALID_ARG),
    (dict(y=ffn.Matrix(0x10000, 16)), ffn.ERR_INVALID_ARG),       # over x
    (dict(y=ffn.Matrix(0x20010, 16)), ffn.ERR_INVALID_ARG),       # over the weight
    (dict(residual=ffn.Matrix(0x30002, 16)), ffn.ERR_INVALID_ARG),  # over part of the residual
    (dict(z=ffn.Matrix(0x30010, 16)), ffn.ERR_INVALID_ARG),       # results over each other
    (dict(bias=0x30010), ffn.ERR_INVALID_ARG),
    (dict(M=1 << 20, x=ffn.Matrix(0x10000, 1 << 36)), ffn.ERR_INVALID_ARG),  # sizes that overflow
])
def test_linear_refuses(lib, over, want):
    n = ctypes.c_int64(-1)
    assert lib.ffn_linear_workspace(ctypes.byref(linear_args(**over)), ctypes.byref(n)) == want
    assert lib.ffn_linear(ctypes.byref(linear_args(**over)), None, 0, None) == want


def test_valid_calls_reach_the_device(lib):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    n = ctypes.c_int64(-1)
    for over in ({}, dict(residual=ffn.Matrix(0x30000, 16)), dict(bias=0x40000), dict(K=0),
                 dict(x=ffn.Matrix(0x10000, 32), y=ffn.Matrix(0x10010, 32), N=16)):  # rows beside each other
        assert lib.ffn_linear_workspace(ctypes.byref(linear_args(**over)), ctypes.byref(n)) == ffn.ERR_CUDA, over
    with pytest.raises(ffn.FfnError):
        ffn.device_status()


def test_null_arguments(lib):
    n = ctypes.c_int64()
    for name in ("linear", "linear_backward", "gated", "gated_backward"):
        assert getattr(lib, f"ffn_{name}_workspace")(None, ctypes.byref(n)) == ffn.ERR_INVALID_ARG
        assert getattr(lib, f"ffn_{name}")(None, None, 0, None) == ffn.ERR_INVALID_ARG
    assert lib.ffn_linear_workspace(ctypes.byref(linear_args()), None) == ffn.ERR_INVALID_ARG


def backward_args(**over):
    m = ffn.Matrix
    a = ffn.LinearBackwardArgs(M=4, N=16, K=8, dy=m(0x10000, 16), x=m(0x20000, 8), weight=m(0x30000, 8),
                               z=m(0x40000, 16), activation=2, dx=m(0x50000, 8), dweight=m(0x60000, 8), dbias=0x70000)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over", [
    dict(z=ffn.Matrix(None, 0)), dict(dweight_type=9), dict(dy=ffn.Matrix(0x10000, 15)), dict(dx=ffn.Matrix(0x10000, 8)),
    dict(dweight=ffn.Matrix(0x50000, 8)), dict(dbias=0x70002), dict(dbias=0x10000), dict(x=ffn.Matrix(None, 8)),
    dict(dweight=ffn.Matrix(0x60002, 8), dweight_type=1),
])
def test_linear_backward_refuses(lib, over):
    n = ctypes.c_int64(-1)
    assert lib.ffn_linear_backward_workspace(ctypes.byref(backward_args(**over)), ctypes.byref(n)) == ffn.ERR_INVALID_ARG


def gated_args(**over):
    m = ffn.Matrix
    a = ffn.GatedArgs(M=4, F=160, C=8, x=m(0x10000, 8), w_gate=m(0x20000, 8), w_up=m(0x30000, 8), activation=2,
                      h=m(0x40000, 160))
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(g=ffn.Matrix(0x50000, 160)), ffn.ERR_INVALID_ARG),  # one of the two
    (dict(g=ffn.Matrix(0x50000, 160), u=ffn.Matrix(0x50000, 160)), ffn.ERR_INVALID_ARG),  # the same
    (dict(qg=ffn.Quantized(0x50000, 256, 0x70000)), ffn.ERR_INVALID_ARG),
    (dict(qg=ffn.Quantized(0x50000, 160, 0x70000), qu=ffn.Quantized(0x60000, 256, 0x78000)), ffn.ERR_ALIGNMENT),
    (dict(qg=ffn.Quantized(0x50008, 256, 0x70000), qu=ffn.Quantized(0x60000, 256, 0x78000)), ffn.ERR_ALIGNMENT),
    (dict(qg=ffn.Quantized(0x50000, 256, None), qu=ffn.Quantized(0x60000, 256, 0x78000)), ffn.ERR_INVALID_ARG),
    (dict(qg=ffn.Quantized(0x50000, 256, 0x70000), qu=ffn.Quantized(0x60000, 256, 0x70008)), ffn.ERR_INVALID_ARG),
    (dict(h=ffn.Matrix(0x20000, 160)), ffn.ERR_INVALID_ARG),
    (dict(w_up=ffn.Matrix(None, 8)), ffn.ERR_INVALID_ARG),
])
def test_gated_refuses(lib, over, want):
    n = ctypes.c_int64(-1)
    assert lib.ffn_gated_workspace(ctypes.byref(gated_args(**over)), ctypes.byref(n)) == want


def gated_backward_args(**over):
    m = ffn.Matrix
    a = ffn.GatedBackwardArgs(M=4, F=160, C=8, N=8, dy=m(0x10000, 8), x=m(0x20000, 8), g=m(0x30000, 160),
                              u=m(0x40000, 160), w_gate=m(0x50000, 8), w_up=m(0x60000, 8), w_down=m(0x70000, 160),
                              activation=2, dx=m(0x80000, 8), dw_gate=m(0x90000, 8), dw_up=m(0xa0000, 8),
                              dw_down=m(0xb0000, 160))
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(qg=ffn.Quantized(0xc0000, 256, 0xd0000), qu=ffn.Quantized(0xe0000, 256, 0xf0000)), ffn.ERR_INVALID_ARG),  # both
    (dict(g=ffn.Matrix(None, 160)), ffn.ERR_INVALID_ARG),
    (dict(g=ffn.Matrix(None, 0), u=ffn.Matrix(None, 0), qg=ffn.Quantized(0xc0000, 168, 0xd0000),
          qu=ffn.Quantized(0xe0000, 256, 0xf0000)), ffn.ERR_ALIGNMENT),
    (dict(dw_up=ffn.Matrix(None, 8)), ffn.ERR_INVALID_ARG),
    (dict(dx=ffn.Matrix(0x10000, 8)), ffn.ERR_INVALID_ARG),
    (dict(dw_down=ffn.Matrix(0x30000, 160)), ffn.ERR_INVALID_ARG),
    (dict(activation=7), ffn.ERR_INVALID_ARG),
    (dict(M=1 << 30, F=1 << 30, g=ffn.Matrix(0x30000, 1 << 30), u=ffn.Matrix(0x30000, 1 << 30)), ffn.ERR_INVALID_ARG),
    (dict(M=1 << 30, F=1 << 30, g=ffn.Matrix(None, 0), u=ffn.Matrix(None, 0),
          qg=ffn.Quantized(0xc0000, 1 << 30, 0xd0000), qu=ffn.Quantized(0xe0000, 1 << 30, 0xf0000)), ffn.ERR_INVALID_ARG),
])
def test_gated_backward_refuses(lib, over, want):
    n = ctypes.c_int64(-1)
    assert lib.ffn_gated_backward_workspace(ctypes.byref(gated_backward_args(**over)), ctypes.byref(n)) == want


def test_options(lib):
    for name, key in ffn.OPTIONS.items():
        v = ctypes.c_int64(-9)
        assert lib.ffn_get_option(key, ctypes.byref(v)) == ffn.OK
        for bad in (-2, 1 << 40):
            assert lib.ffn_set_option(key, bad) == ffn.ERR_INVALID_ARG, name
    assert lib.ffn_set_option(99, 0) == ffn.ERR_INVALID_ARG
    assert lib.ffn_set_option(ffn.OPTIONS["watchdog_ns"], 99999) == ffn.ERR_INVALID_ARG
    assert lib.ffn_set_option(ffn.OPTIONS["width"], 24) == ffn.ERR_INVALID_ARG
    v = ctypes.c_int64()
    with pytest.raises(RuntimeError, match="inside"):
        with ffn.options(cta_group=2, width=64):
            assert lib.ffn_get_option(1, ctypes.byref(v)) == ffn.OK and v.value == 2
            raise RuntimeError("inside")
    assert lib.ffn_get_option(1, ctypes.byref(v)) == ffn.OK and v.value == 0
    with pytest.raises(ffn.FfnError):
        with ffn.options(cta_group=1, width=24):
            pass
    assert lib.ffn_get_option(1, ctypes.byref(v)) == ffn.OK and v.value == 0


def cpu(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call,what", [
    (lambda: ffn.linear(cpu(4, 8), cpu(16, 8)), "CUDA device"),
    (lambda: ffn.linear(cpu(4, 8), cpu(16, 9)), "weight must be 16 x 8"),
    (lambda: ffn.linear(cpu(4, 8, dtype=torch.float16), cpu(16, 8)), "x must be bf16"),
    (lambda: ffn.linear(cpu(8), cpu(16, 8)), "matrices"),
    (lambda: ffn.linear(cpu(8, 4).t(), cpu(16, 8)), "contiguous rows"),
    (lambda: ffn.linear(cpu(1, 8).expand(4, 8), cpu(16, 8)), "overlap"),
    (lambda: ffn.linear(cpu(4, 8), cpu(16, 8), bias=cpu(15)), "vector of 16"),
    (lambda: ffn.linear(cpu(4, 8), cpu(16, 8), bias=cpu(16, dtype=torch.int32)), "bf16 or fp32"),
    (lambda: ffn.linear(cpu(4, 8), cpu(16, 8), activation="tanh"), "activation must be one of"),
    (lambda: ffn.linear(cpu(4, 8), cpu(16, 8), activation=[]), "activation must be one of"),
    (lambda: ffn.linear(cpu(4, 8), cpu(16, 8), residual=cpu(4, 8)), "residual must be 4 x 16"),
    (lambda: ffn.linear(cpu(4, 8), cpu(16, 8).requires_grad_()), "requires a gradient"),
    (lambda: ffn.linear(None, cpu(16, 8)), "x must be a tensor"),
    (lambda: ffn.linear_backward(cpu(4, 16), cpu(4, 8), cpu(16, 8), activation="silu"), "needs z"),
    (lambda: ffn.linear_backward(cpu(4, 15), cpu(4, 8), cpu(16, 8)), "dy must be 4 x 16"),
    (lambda: ffn.linear_backward(cpu(4, 16), cpu(4, 8), cpu(16, 8), grad_dtype=torch.float16), "grad_dtype"),
    (lambda: ffn.gated(cpu(4, 8), cpu(16, 8), cpu(15, 8)), "w_up must be 16 x 8"),
    (lambda: ffn.gated(cpu(4, 8), cpu(16, 8), cpu(16, 8), save="fp8"), "save must be one of"),
    (lambda: feedforward.GatedFeedForward(cpu(16, 8), cpu(16, 8), cpu(8, 15)), "N x F"),
    (lambda: feedforward.FeedForward(cpu(16, 8), cpu(8, 15)), "N x F"),
])
def test_python_refuses(lib, call, what):
    with pytest.raises((ValueError, TypeError), match=what):
        call()


def test_status_needs_a_cuda_device(lib):
    with pytest.raises(ValueError, match="device"):
        ffn.device_status(-1)
    with pytest.raises(ValueError, match="device"):
        ffn.device_status("cpu")


def test_work_split_and_tile_order(tmp_path):
    """Host functions of the kernel's header: tests/ffn_split_check.cu."""
    exe = tmp_path / "ffn_split_check"
    build = subprocess.run(
        [libbuild.nvcc(), "-std=c++17", "-O2", *libbuild.ARCH, "-I", libbuild.INCLUDE, "-I", libbuild.CSRC,
         os.path.join(ROOT, "tests", "ffn_split_check.cu"), "-o", str(exe)], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.endswith("splits\n"), run.stdout + run.stderr


def test_the_library_lies_beside_the_one_of_its_binding(monkeypatch, tmp_path):
    monkeypatch.setattr(libbuild, "FP8_LIB", str(tmp_path / "libfp8_ops.so"))
    assert libbuild.ffn_lib() == str(tmp_path / "libffn_ops.so")


# ------------------------------------------------------------------ the references
@pytest.mark.parametrize("name", [n for n in ffn.ACTIVATIONS if n])
def test_slopes_are_the_activations_differences(name):
    z = torch.linspace(-6, 6, 400, dtype=torch.float64) + 0.0101
    h = 1e-5
    num = (ref.act(name, z + h) - ref.act(name, z - h)) / (2 * h)
    assert (num - ref.slope(name, z)).abs().max() < 1e-8


@pytest.mark.parametrize("activation", ["silu", "gelu", "gelu_tanh"])
def test_gradients_are_the_loss_differences(activation):
    gen = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, wg, wu, wd, r = rand(3, 5), rand(7, 5), rand(7, 5), rand(4, 7), rand(3, 4)
    loss = lambda: float(((ref.act(activation, x @ wg.T) * (x @ wu.T)) @ wd.T * r).sum())  # noqa: E731
    monkey = ref.bf16
    ref.bf16 = lambda v: v  # the formula itself
    try:
        grads = ref.gated_backward(r, x, x @ wg.T, x @ wu.T, wg, wu, wd, activation)
    finally:
        ref.bf16 = monkey
    for t, g in zip((x, wg, wu, wd), grads):
        for i in range(0, t.numel(), 3):
            flat, h = t.view(-1), 1e-6
            at = flat[i].item()
            flat[i] = at + h
            up = loss()
            flat[i] = at - h
            down = loss()
            flat[i] = at
            assert abs((up - down) / (2 * h) - g.reshape(-1)[i].item()) < 1e-6


def test_checkpoints_are_fp8s_format():
    v = torch.randn(5, 300, dtype=torch.float64, generator=torch.Generator().manual_seed(1)) * 3
    held = ref.checkpoint(v)
    codes, e = fp8ref.quantize(v.numpy())
    assert torch.equal(held, torch.from_numpy(fp8ref.values(torch.from_numpy(codes).float().to(torch.float8_e4m3fn),
                                                            fp8ref.pack_scales(e))))
    assert ((held - v).abs() <= 2.0**-4 * v.abs() + 2.0**-10 * v.abs().max()).all()
