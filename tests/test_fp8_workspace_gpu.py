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


# one SM and pairs, whole tiles, tiles split through global memory and among clusters (rank 0
# adding the pieces, and every rank its part), an fp32 D in segments
@pytest.mark.parametrize("options,dtype", [
    (SPLIT, torch.bfloat16),
    ({"cta_group": 1, "transposed": 2, "width": 32, "split": 0}, torch.bfloat16),
    ({"cta_group": 2, "transposed": 1, "width": 224, "split": 0}, torch.bfloat16),
    ({"cta_group": 2, "transposed": 2, "width": 64, "split": 2}, torch.bfloat16),
    ({"cta_group": 1, "transposed": 1, "width": 224, "split": 1}, torch.bfloat16),
    ({"cta_group": 1, "transposed": 2, "width": 32, "split": 1}, torch.bfloat16),
    ({"cta_group": 2, "transposed": 1, "width": 96, "split": 2}, torch.float32),
], ids=["ranges", "whole", "pairs", "pair-ranges", "clusters", "spread", "segments"])
def test_a_launch_may_give_up_at_any_load(options, dtype):
    # loads in the ring's first lap and later ones: stages that follow the missing load
    # are not filled again, and the next launch is right
    args, want = problem(200, 2560, 12000, 10)
    with fp8.Gemm(0, **options) as g:
        for skip in (0, 1, 2, 7, 8, 9, 13, 20, 40):
            g.set_option("watchdog_ns", 4000000)
            g.set_option("fault_skip_load", skip)
            g.run(*args, out_dtype=dtype)
            st, _ = g.device_status()
            assert st in (fp8.ERR_DEVICE_TIMEOUT, fp8.OK)  # OK: no CTA has that many loads
            assert st == fp8.ERR_DEVICE_TIMEOUT or skip > 1
            g.set_option("fault_skip_load", -1)
            g.set_option("watchdog_ns", 2000000000)
            d = g.run(*args, out_dtype=dtype)
            assert d.cpu().to(torch.bfloat16).equal(want)
            assert g.device_status() == (fp8.OK, 0)


def test_a_workspace_may_hold_anything():
    args, want = problem(20, 2560, 12000, 2)
    out = torch.empty(20, 2560, dtype=torch.bfloat16, device="cuda")
    lib = fp8.load()
    with fp8.Gemm(0, **SPLIT) as g:
        g.plan(20, 2560, 12000)
        need = fp8._L()
        assert lib.fp8_gemm_workspace(g.h, need) == fp8.OK and need.value > 0
        work = torch.empty(need.value // 4, dtype=torch.int32, device="cuda")
        ptrs = [t.data_ptr() for t in args] + [out.data_ptr()]
        stream = torch.cuda.current_stream().cuda_stream
        run = lambda w, n: lib.fp8_gemm_run_in(g.h, *ptrs, w, n, stream)  # noqa: E731
        for value in (1, 0, -1, 1):  # 1: every flag set
            work.fill_(value)
            out.fill_(0)
            assert run(work.data_ptr(), need.value) == fp8.OK
            assert out.cpu().equal(want)
        assert run(None, need.value) == fp8.ERR_INVALID_ARG
        assert run(work.data_ptr(), need.value - 1) == fp8.ERR_INVALID_ARG
        assert run(work.data_ptr() + 4, need.value) == fp8.ERR_ALIGNMENT
        # a workspace of the handle's own
        out.fill_(0)
        assert lib.fp8_gemm_run(g.h, *ptrs, stream) == fp8.OK
        assert out.cpu().equal(want)
        assert g.device_status()[0] == fp8.OK


# a product whose default plan splits tiles through global memory
M, N, K = 588, 2033, 24654


def splits_through_global_memory():
    with fp8.Gemm(0) as g:
        info = g.plan(M, N, K)
    return info["split_tiles"] > 0 and info["cluster"] == 1


def test_graphs_replayed_at_once_on_two_streams():
    assert splits_through_global_memory()
    work = [problem(M, N, K, seed) for seed in (3, 4)]
    graphs, outs = [], []
    for args, _ in work:  # both captured on torch's one stream for captures
        graphs.append(torch.cuda.CUDAGraph())
        outs.append(torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
        with torch.cuda.graph(graphs[-1]):
            for _ in range(3):
                fp8.gemm(*args, out=outs[-1])
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for out in outs:
            out.fill_(-1)
        torch.cuda.synchronize()
        for _ in range(4):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for out, (_, want) in zip(outs, work):
            assert out.cpu().equal(want)


def test_calls_at_once_on_two_streams_beside_a_graph():
    work = [problem(M, N, K, seed) for seed in (5, 6, 7)]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph, held = torch.cuda.CUDAGraph(), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        fp8.gemm(*work[0][0], out=held)
    with fp8.Gemm(0) as g:  # one handle on two streams: the calls' workspaces are their own
        for _ in range(20):
            held.fill_(-1)
            torch.cuda.synchronize()
            graph.replay()  # on the current stream
            one = g.run(*work[1][0], stream=side)
            two = g.run(*work[2][0], stream=other)
            torch.cuda.synchronize()
            for got, (_, want) in zip((held, one, two), work):
                assert got.cpu().equal(want)
        assert g.device_status()[0] == fp8.OK


def test_no_workspace_is_kept_for_a_stream():
    assert splits_through_global_memory()
    args, want = problem(M, N, K, 8)
    fp8.gemm(*args)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    for _ in range(20):
        got = fp8.gemm(*args, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        assert got.cpu().equal(want)
    del got
    torch.cuda.empty_cache()
    # 20 MB each, if they were
    assert torch.cuda.mem_get_info()[0] > free - 100 * 2**20


def test_status_of_a_graph_replayed_on_another_stream():
    args, want = problem(20, 2560, 12000, 9)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with fp8.Gemm(0, watchdog_ns=20000000, fault_skip_load=1, **SPLIT) as g:
        g.run(*args)
        assert g.device_status()[0] == fp8.ERR_DEVICE_TIMEOUT
        with torch.cuda.graph(graph):
            g.run(*args)
        for _ in range(3):
            with torch.cuda.stream(side):
                graph.replay()
            st, detail = g.device_status()  # waits for the replay
            assert st == fp8.ERR_DEVICE_TIMEOUT and detail != 0
            assert g.device_status() == (fp8.OK, 0)


def test_status_of_the_module_level_product():
    args, want = problem(20, 2560, 12000, 11)
    assert fp8.gemm(*args).cpu().equal(want)
    assert fp8.device_status() == (fp8.OK, 0)
    lib, kept = fp8.load(), fp8._P(fp8._ops().kept_handle(0))
    option = lambda name, value: lib.fp8_gemm_set_option(kept, fp8.OPTIONS[name], value)  # noqa: E731
    assert option("watchdog_ns", 4000000) == fp8.OK and option("fault_skip_load", 1) == fp8.OK
    try:
        fp8.gemm(*args, stream=torch.cuda.Stream())
        st, detail = fp8.device_status("cuda:0")
        assert st == fp8.ERR_DEVICE_TIMEOUT and detail != 0
    finally:
        assert option("watchdog_ns", 2000000000) == fp8.OK and option("fault_skip_load", -1) == fp8.OK
    assert fp8.gemm(*args).cpu().equal(want)
    assert fp8.device_status(torch.device("cuda", 0)) == (fp8.OK, 0)


def test_the_default_stream_by_its_raw_handle():
    side = torch.cuda.Stream()
    for raw in (torch.cuda.default_stream().cuda_stream, 1):
        with torch.cuda.stream(side):  # not the current stream
            with fp8._on(raw, torch.device("cuda", 0)):
                assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with fp8._on(side.cuda_stream, torch.device("cuda", 0)):
        assert torch.cuda.current_stream().cuda_stream == side.cuda_stream
    # ordered behind the default stream's work
    x = torch.zeros(8192, 8192, device="cuda")
    for value in (1.0, 2.0, 3.0):
        x.fill_(value)
        q, s = fp8.quantize(x, stream=0)
        torch.cuda.synchronize()
        assert bool((q.float() * torch.exp2(s.view(torch.uint8)[0, :, :1].float() - 127) == value).all())


def test_the_watchdogs_limit_is_no_shorter_than_loads_take():
    with fp8.Gemm(0) as g:
        for limit in (0, 1000, 99999, 60000000001):
            with pytest.raises(fp8.Fp8Error, match="invalid"):
                g.set_option("watchdog_ns", limit)
        g.set_option("watchdog_ns", 100000)
        assert g.get_option("watchdog_ns") == 100000
