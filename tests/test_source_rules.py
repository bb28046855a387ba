"""Rules on the kernel sources that need no GPU.

The kernels read only this GPU's own memory: no TMA copy (cp.async.bulk...)
uses cluster multicast.  The one `multicast::cluster` in the sources is
tcgen05.commit's arrive on both CTAs' barriers of an SM pair, which moves no
data.
"""
from __future__ import annotations

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "warp_specialized_tma_gb300", "csrc")


def _sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(CSRC, name)) as fh:
                yield name, fh.read()


def test_no_tma_multicast_copy():
    for name, text in _sources():
        for m in re.finditer(r"cp\.(?:reduce\.)?async\.bulk[^\"]*", text):
            assert "multicast" not in m.group(0), f"{name}: {m.group(0)}"


def test_multicast_only_in_the_pair_commit():
    hits = [(name, line.strip()) for name, text in _sources() for line in text.splitlines() if "multicast" in line
            and not line.strip().startswith("//")]
    assert hits, "the SM-pair commit is expected to multicast its arrive"
    for name, line in hits:
        assert "tcgen05.commit" in line, f"{name}: {line}"


def test_lanes_are_synchronised_after_lane_0_acquires_for_them():
    """In the 8-bit product one lane waits for a partial that all lanes then load: a shuffle of the
    outcome orders no memory, so a __syncwarp stands between the wait and the loads."""
    text = dict(_sources())["fp8_gemm.cuh"]
    collect = re.search(r"auto collect = \[&\]\(\) \{(.*?)\n {12}\};", text, re.S).group(1)
    waits = re.findall(r"(?:warp_wait_flag\(|ctl\.wait<true>\(ready_bar)(.*?)(?=warp_wait_flag\(|ctl\.wait<true>|\Z)",
                       collect, re.S)
    assert len(waits) == 2
    for after in waits:
        assert "__syncwarp();" in after


def test_the_gradients_ring_is_not_refilled_after_a_wait_that_ran_out():
    """A slot whose copies have not landed must not be given another arrival, and the waits
    that follow one that ran out must be short: there may be a million rows."""
    text = dict(_sources())["fp8_norm.cu"]
    assert re.search(r"if \(t == 0 && before >= 0 && ok\)\s*fill\(before", text)
    assert len(re.findall(r"\bfill\(", text)) == 2  # that, and the first lap's
    assert "ok ? 200u : 1u" in text
