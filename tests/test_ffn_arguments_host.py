"""Arguments of the feed-forward operators that do not go together are refused.  No kernel runs here: a call
that is not refused goes on to ask for a CUDA device."""
from __future__ import annotations

import pytest
import torch

from warp_specialized_tma_gb300 import build as libbuild
from warp_specialized_tma_gb300 import ffn

bf, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()


def cpu(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("out,out_dtype,what", [
    (bf, f32, "out is not of out_dtype"),
    (f32, bf, "out is not of out_dtype"),
    (bf, torch.float16, "out_dtype must be bf16 or fp32"),
    (None, torch.float16, "out_dtype must be bf16 or fp32"),
    (None, "bf16", "out_dtype must be a torch.dtype"),
    # these go together
    (bf, bf, "CUDA device"),
    (f32, f32, "CUDA device"),
    (f32, None, "CUDA device"),
    (bf, None, "CUDA device"),
    (None, f32, "CUDA device"),
    (None, None, "CUDA device"),
])
def test_the_results_type(out, out_dtype, what):
    with pytest.raises((ValueError, TypeError), match=what):
        ffn.linear(cpu(4, 8), cpu(16, 8), out=None if out is None else cpu(4, 16, dtype=out), out_dtype=out_dtype)
