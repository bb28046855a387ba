"""The plans that the feed-forward products choose, checked without a GPU: tests/ffn_plan_check.cu."""
from __future__ import annotations

import os
import subprocess

from warp_specialized_tma_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_plan_visits_all_of_its_tiles(tmp_path):
    exe = tmp_path / "ffn_plan_check"
    build = subprocess.run(
        [libbuild.nvcc(), "-std=c++17", "-O2", *libbuild.ARCH, "-I", libbuild.INCLUDE, "-I", libbuild.CSRC,
         os.path.join(ROOT, "tests", "ffn_plan_check.cu"), "-o", str(exe)], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.endswith("covered\n"), run.stdout + run.stderr
