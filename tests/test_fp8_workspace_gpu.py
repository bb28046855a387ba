"""The workspace of the product's split tiles and the status of its launches, where launches
follow one that gave up, overlap, or belong to graphs.  Operands are integers whose products'
sums are exact, so every result must equal the 64-bit one bit for bit."""
from __future__ import annotations

import pytest
import torch

import fp8_reference as ref
from warp_specialized_tma_gb300 import fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from warp_specialized_tma_gb300 import build as libbuild
    libbuild.build()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def operand(R, K, gen):
    """(codes, scales) on the GPU and the 64-bit values: integers in -4..4, scales 2^-2..2^2."""
    codes = torch.randint(-4, 5, (R, K), generator=gen).float().to(torch.float8_e4m3fn)
    scales = ref.pack_scales(torch.randint(125, 130, (R, -(-K // 128)), generator=gen).numpy())
    held = torch.zeros(R, -(-K // 128) * 128, dtype=torch.uint8, device="cuda")
    held[:, :K] = codes.view(torch.uint8).cuda()
    return held.view(torch.float8_e4m3fn)[:, :K], scales.cuda(), ref.values(codes, scales)


def problem(M, N, K, seed):
    """Arguments of a product and its exact result in bf16."""
    gen = torch.Generator().manual_seed(seed)
    a, sa, va = operand(M, K, gen)
    b, sb, vb = operand(N, K, gen)
    return (a, sa, b, sb), torch.from_numpy(va @ vb.T).to(torch.bfloat16)


# 20 tiles of 94 k-blocks in 152 ranges, of 12 or 13 units: through global memory
SPLIT = {"cta_group": 1, "transposed": 2, "width": 32, "split": 2}


def test_a_launch_that_gave_up_leaves_nothing_to_the_next():
    args, want = problem(20, 2560, 12000, 1)
    with fp8.Gemm(0, **SPLIT) as g:
        assert g.run(*args).cpu().equal(want)
        assert g.info()["split_tiles"] == 20 and g.info()["cluster"] == 1
        assert g.device_status()[0] == fp8.OK
        # Load 12 is the last of the longer ranges: they give up, among them tiles' owners
        # whose pieces come from shorter ranges and are left unread.
        for skip in (12, 5, 12):
            g.set_option("watchdog_ns", 3000000)
            g.set_option("fault_skip_load", skip)
            g.run(*args)
            g.set_option("fault_skip_load", -1)
            g.set_option("watchdog_ns", 2000000000)
            args, want = problem(20, 2560, 12000, skip)
            assert g.run(*args).cpu().equal(want)
        assert g.device_status()[0] == fp8.ERR_DEVICE_TIMEOUT
        assert g.run(*args).cpu().equal(want)
        assert g.device_status()[0] == fp8.OK
