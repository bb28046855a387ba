"""Host-only checks of the 8-bit operators' C ABI: the library builds, loads
without a GPU and exports what include/fp8_ops.h declares; argument checks and
status strings behave as documented.  No kernel runs here.  The 64-bit
references of the GPU tests are checked against torch's own e4m3 and against
differences."""
from __future__ import annotations

import os
import re
import subprocess

import numpy as np
import pytest
import torch

import fp8_reference as ref
from warp_specialized_tma_gb300 import build as libbuild
from warp_specialized_tma_gb300 import fp8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8_ops.h")


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return fp8.load()


def declared_entry_points():
    return re.findall(r"FP8_API\s+[\w\s\*]+?\b(fp8_\w+)\s*\(", open(HEADER).read())


def test_the_abi_is_what_is_exported_and_bound(lib):
    names = set(declared_entry_points())
    assert names == set(fp8._SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", fp8.LIB_PATH], capture_output=True, text=True)
    if out.returncode != 0:
        pytest.skip("nm unavailable")
    syms = {line.split()[-1] for line in out.stdout.splitlines() if line.strip()}
    assert {s for s in syms if not s.startswith("_")} == names


def test_strings(lib):
    assert lib.fp8_strerror(0) == b"ok"
    for st in range(-7, 0):
        assert lib.fp8_strerror(st) not in (b"", b"unknown status")
    assert lib.fp8_strerror(-99) == b"unknown status"
    assert "sm_103a" in fp8.version()


def test_mirrors_of_the_header():
    text = open(HEADER).read()
    body = re.search(r"typedef struct fp8_gemm_plan_info_s \{(.*?)\} fp8_gemm_plan_info_t;", text, re.S).group(1)
    fields = re.findall(r"^\s*(int32_t|int64_t)\s+(\w+);", body, re.M)
    assert [n for n, _ in fp8.PlanInfo._fields_] == [n for _, n in fields]
    for (name, ct), (c, _) in zip(fp8.PlanInfo._fields_, fields):
        assert np.dtype(ct).itemsize == (8 if c == "int64_t" else 4), name
    body = re.search(r"typedef enum fp8_gemm_option \{(.*?)\} fp8_gemm_option;", text, re.S).group(1)
    assert {n.lower(): int(v) for n, v in re.findall(r"FP8_GEMM_OPT_(\w+)\s*=\s*(\d+)", body)} == fp8.OPTIONS
    assert int(re.search(r"FP8_NORM_MAX_COLUMNS (\d+)", text).group(1)) == fp8.NORM_MAX_COLUMNS


@pytest.mark.parametrize("args,want", [
    ((256, 256, 256, 256, 256, 256, 0), fp8.OK),
    ((6143, 5999, 4104, 4224, 4112, 5999, 1), fp8.OK),
    ((0, 4, 8, 16, 16, 4, 0), fp8.OK),
    ((4, 4, 0, 0, 0, 4, 0), fp8.OK),
    ((-1, 4, 8, 16, 16, 4, 0), fp8.ERR_INVALID_ARG),
    ((4, 4, 32, 16, 32, 4, 0), fp8.ERR_INVALID_ARG),   # lda < K
    ((4, 4, 32, 32, 16, 4, 0), fp8.ERR_INVALID_ARG),   # ldb < K
    ((4, 8, 32, 32, 32, 7, 0), fp8.ERR_INVALID_ARG),   # ldd < N
    ((4, 4, 16, 16, 16, 4, 2), fp8.ERR_INVALID_ARG),   # no such type
    ((4, 4, 20, 24, 32, 4, 0), fp8.ERR_ALIGNMENT),
    ((4, 4, 20, 32, 24, 4, 0), fp8.ERR_ALIGNMENT),
    ((1 << 31, 4, 16, 16, 16, 4, 0), fp8.ERR_INVALID_ARG),
])
def test_check_problem(lib, args, want):
    assert lib.fp8_gemm_check_problem(*args) == want


def test_null_and_misaligned_arguments_are_refused(lib):
    assert lib.fp8_gemm_plan(None, 8, 8, 16, 16, 16, 8, 0) == fp8.ERR_INVALID_ARG
    assert lib.fp8_gemm_run(None, 16, 16, 16, 16, 16, None) == fp8.ERR_INVALID_ARG
    assert lib.fp8_gemm_create(0, None) == fp8.ERR_INVALID_ARG
    assert lib.fp8_gemm_destroy(None) == fp8.OK
    q = lambda **k: lib.fp8_quantize(*({"x": 256, "xt": 0, "ldx": 128, "R": 4, "C": 128, "tile": 0, "rf": None,  # noqa: E731
                                        "cf": None, "ct": 0, "q": 256, "ldq": 128, "s": 256, "qt": None, "ldqt": 0,
                                        "st": None, "stream": None} | k).values())
    assert q(x=None) == fp8.ERR_INVALID_ARG
    assert q(s=None) == fp8.ERR_INVALID_ARG
    assert q(q=None, s=None) == fp8.ERR_INVALID_ARG
    assert q(qt=256, st=256, ldqt=0) == fp8.ERR_INVALID_ARG
    assert q(xt=7) == fp8.ERR_INVALID_ARG
    assert q(ldx=100) == fp8.ERR_INVALID_ARG
    assert q(ldq=136) == fp8.ERR_ALIGNMENT
    assert q(q=264) == fp8.ERR_ALIGNMENT
    assert q(x=257) == fp8.ERR_ALIGNMENT
    assert q(R=0) == fp8.OK
    n = lambda **k: lib.fp8_rmsnorm(*({"x": 256, "ldx": 128, "r": None, "ldr": 0, "w": 256, "wt": 0, "R": 4, "C": 128,  # noqa: E731
                                       "eps": 1e-6, "h": None, "ldh": 0, "q": 256, "ldq": 128, "s": 256, "rstd": 256,
                                       "stream": None} | k).values())
    assert n(C=0) == fp8.ERR_INVALID_ARG
    assert n(C=fp8.NORM_MAX_COLUMNS + 1, ldx=1 << 20, ldq=1 << 20) == fp8.ERR_UNSUPPORTED
    assert n(r=256, ldr=128) == fp8.ERR_INVALID_ARG  # no pitch, then no place, for h
    assert n(r=256, ldr=128, ldh=128) == fp8.ERR_INVALID_ARG
    assert n(eps=-1.0) == fp8.ERR_INVALID_ARG
    assert n(eps=float("nan")) == fp8.ERR_INVALID_ARG
    assert n(w=None) == fp8.ERR_INVALID_ARG
    assert n(rstd=258) == fp8.ERR_ALIGNMENT
    assert n(R=0) == fp8.OK
    assert lib.fp8_rmsnorm_backward_workspace(4, 128, None) == fp8.ERR_INVALID_ARG


def test_create_without_a_usable_gpu_fails_cleanly(lib):
    import ctypes
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    h = ctypes.c_void_p()
    assert lib.fp8_gemm_create(0, ctypes.byref(h)) in (fp8.ERR_CUDA, fp8.ERR_UNSUPPORTED)
    assert not h.value
    with pytest.raises(ValueError, match="CUDA device"):
        fp8.quantize(torch.zeros(2, 3))


def test_reference_rounding_is_that_of_e4m3():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    v = np.unique(v[~torch.isnan(v)].numpy())
    mid = (v[1:] + v[:-1]) / 2  # ties, and points beside them
    x = np.concatenate([v, mid, mid + 1e-7, mid - 1e-7, np.random.RandomState(0).uniform(-448, 448, 5000)])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ref.e4m3_round(x.astype(np.float64)), want)


def test_reference_scales_are_the_least():
    amax = np.exp2(np.random.RandomState(1).uniform(-60, 60, 2000))
    amax = np.concatenate([amax, 448.0 * np.exp2(np.arange(-20, 20)), 448.0 * np.exp2(np.arange(-20, 20)) * (1 + 2.0**-40)])
    e = ref.scale_exponents(amax) - 127
    assert (amax <= 448 * np.exp2(e)).all() and (amax > 448 * np.exp2(e - 1)).all()
    assert ref.scale_exponents(np.array([0.0, 2.0**-149]))[0] == 0


def test_reference_gradient_is_that_of_the_norm():
    rng = np.random.RandomState(2)
    h, w, dy, eps = rng.randn(3, 40), rng.randn(40), rng.randn(3, 40), 1e-6
    _, rstd = ref.rmsnorm(h, w, eps)
    dx, dw = ref.rmsnorm_backward(dy, h, w, rstd)
    v, u, t = rng.randn(3, 40), rng.randn(40), 1e-6
    loss = lambda a, b: (dy * ref.rmsnorm(a, b, eps)[0]).sum()  # noqa: E731
    assert (loss(h + t * v, w) - loss(h - t * v, w)) / (2 * t) == pytest.approx((dx * v).sum(), rel=1e-6)
    assert (loss(h, w + t * u) - loss(h, w - t * u)) / (2 * t) == pytest.approx((dw * u).sum(), rel=1e-6)


def test_work_split(tmp_path):
    """The product's work split (host functions of its kernel's header): tests/fp8_split_check.cu."""
    nvcc = libbuild.nvcc()
    exe = tmp_path / "fp8_split_check"
    build = subprocess.run(
        [nvcc, "-std=c++17", "-O2", *libbuild.ARCH, "-I", libbuild.INCLUDE, "-I", libbuild.CSRC,
         os.path.join(ROOT, "tests", "fp8_split_check.cu"), "-o", str(exe)], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.endswith("splits\n"), run.stdout + run.stderr


def test_a_launch_takes_its_workspace_from_the_caller(lib):
    import ctypes
    need = ctypes.c_int64(-1)
    assert lib.fp8_gemm_workspace(None, ctypes.byref(need)) == fp8.ERR_INVALID_ARG
    assert lib.fp8_gemm_run_in(None, 16, 16, 16, 16, 16, 256, 1 << 20, None) == fp8.ERR_INVALID_ARG


def test_the_module_level_product_has_a_status(lib):
    with pytest.raises(ValueError, match="device"):
        fp8.device_status(-1)
    with pytest.raises(ValueError, match="device"):
        fp8.device_status("cpu")
    if not torch.cuda.is_available():
        with pytest.raises(fp8.Fp8Error):
            fp8.device_status(0)


def test_tile_order(tmp_path):
    """The product's tile order for any band height and number of tiles: tests/fp8_tiles_check.cu."""
    exe = tmp_path / "fp8_tiles_check"
    build = subprocess.run(
        [libbuild.nvcc(), "-std=c++17", "-O2", *libbuild.ARCH, "-I", libbuild.INCLUDE, "-I", libbuild.CSRC,
         os.path.join(ROOT, "tests", "fp8_tiles_check.cu"), "-o", str(exe)], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.endswith("orders\n"), run.stdout + run.stderr


def test_tensors_that_require_a_gradient_are_refused(lib):
    # on the CPU: with or without, the tensors are on the wrong device, which is found later
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    w, rstd = torch.ones(128), torch.ones(2)
    q, s = torch.zeros(2, 128, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(1, 2, 4, dtype=torch.uint8)
    out = torch.zeros(2, 2)
    calls = {
        "x": lambda t: fp8.quantize(t(x)),
        "row_factor": lambda t: fp8.quantize_columns(x, row_factor=t(rstd)),
        "column_factor": lambda t: fp8.quantize_both(x, column_factor=t(w)),
        "weight": lambda t: fp8.rmsnorm(x, t(w)),
        "residual": lambda t: fp8.rmsnorm(x, w, residual=t(x)),
        "out_h": lambda t: fp8.rmsnorm(x, w, residual=x, out_h=t(x)),
        "dy": lambda t: fp8.rmsnorm_backward(t(x), x, w, rstd),
        "h": lambda t: fp8.rmsnorm_backward(x, t(x), w, rstd),
        "rstd": lambda t: fp8.rmsnorm_backward(x, x, w, t(rstd)),
        "dresidual": lambda t: fp8.rmsnorm_backward(x, x, w, rstd, dresidual=t(x)),
        "out": lambda t: fp8._ops().gemm(0, q, s, q, s, t(out), torch.float32),
    }
    for name, call in calls.items():
        with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
            call(lambda t: t.clone().requires_grad_())
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
            call(lambda t: t.clone().requires_grad_())
        with pytest.raises(ValueError, match="CUDA device"):
            call(lambda t: t)


def test_rows_written_over_part_of_rows_read(lib, tmp_path):
    """csrc/fp8_overlap.h against a count of every byte, and that the calls refuse what it finds."""
    exe = tmp_path / "fp8_overlap_check"
    build = subprocess.run([libbuild.cxx(), "-std=c++17", "-O2", "-I", libbuild.CSRC,
                            os.path.join(ROOT, "tests", "fp8_overlap_check.cpp"), "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.endswith("clash\n"), run.stdout + run.stderr
    far = 1 << 20
    norm = lambda x, r, h: lib.fp8_rmsnorm(x, 128, r, 128, 256, 0, 4, 128, 1e-6, h, 128, 256, 128, 256, None, None)  # noqa: E731
    back = lambda dy, h, dr, dx: lib.fp8_rmsnorm_backward(dy, 128, h, 128, 256, 0, 256, dr, 128, dx, 128, 256, 4, 128,  # noqa: E731
                                                          256, 1 << 40, None)
    assert norm(far, 2 * far, far + 2) == fp8.ERR_INVALID_ARG
    assert norm(far, 2 * far, far + 256) == fp8.ERR_INVALID_ARG  # a row further
    assert norm(far, 2 * far, 2 * far - 768) == fp8.ERR_INVALID_ARG  # its last row over residual's first
    if torch.cuda.is_available():
        return  # the workspace's size is asked of the device first; from here a GPU is expected
    for dx in (far + 2, 2 * far - 768, 3 * far + 254):
        assert back(far, 2 * far, 3 * far, dx) in (fp8.ERR_INVALID_ARG, fp8.ERR_CUDA, fp8.ERR_UNSUPPORTED)
