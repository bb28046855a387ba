"""What the build needs: the libraries nvcc alone, the Python binding torch besides.  No compiler
runs here: commands are recorded, and their output files made empty."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from warp_specialized_tma_gb300 import build as libbuild


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """Builds go to tmp_path; returns the list of files that commands were asked to make."""
    made, broken = [], set()

    def run(cmd, **kwargs):
        if "-o" not in cmd:
            return subprocess.CompletedProcess(cmd, 0, "release 13.0\n", "")
        out = os.path.basename(cmd[cmd.index("-o") + 1]).split(".tmp")[0]
        if out in broken:
            return subprocess.CompletedProcess(cmd, 1, "", "broken")
        made.append(out)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(libbuild.subprocess, "run", run)
    monkeypatch.setattr(libbuild, "BUILD_DIR", str(tmp_path))
    for name in ("LIB", "FP8_LIB", "FP8_BIND"):
        monkeypatch.setattr(libbuild, name, str(tmp_path / os.path.basename(getattr(libbuild, name))))
    return made, broken


LIBRARIES = {"libgemm_bf16.so", "libfp8_ops.so"}


def test_the_libraries_build_without_torch(fake, monkeypatch):
    made, _ = fake
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    assert not libbuild.up_to_date()
    assert libbuild.build() == libbuild.LIB
    assert LIBRARIES <= set(made) and "_fp8_bind.so" not in made
    assert libbuild.up_to_date()
    made.clear()
    libbuild.build()
    assert made == []


def test_the_binding_follows_where_torch_is(fake, monkeypatch):
    made, _ = fake
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        libbuild.build()
    made.clear()
    assert not libbuild.up_to_date()
    libbuild.build()
    assert set(made) == {"fp8_bind.o", "_fp8_bind.so"}  # the libraries stand
    assert libbuild.up_to_date()
    made.clear()
    libbuild.build(force=True)
    assert LIBRARIES | {"_fp8_bind.so"} <= set(made)


def test_a_binding_that_fails_leaves_the_libraries(fake):
    made, broken = fake
    broken.add("fp8_bind.o")
    with pytest.raises(RuntimeError, match="fp8_bind"):
        libbuild.build()
    assert LIBRARIES <= set(made) and libbuild.libraries_up_to_date() and not libbuild.up_to_date()
    broken.clear()
    made.clear()
    libbuild.build()
    assert set(made) == {"fp8_bind.o", "_fp8_bind.so"}
