"""Data that lanes of one wave hand each other through LDS without a workgroup
barrier: the source has to keep the compiler to that order, which shows as a
wave barrier between the accesses in the gfx950 code.  (CPU only: hipcc
cross-compiles to assembly, nothing runs.)"""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from copy_reduce_snac_amd.build import CSRC, DEVICE_FLAGS, HIPCC, SOURCE_FLAGS

pytestmark = pytest.mark.skipif(shutil.which(HIPCC) is None, reason="hipcc not available")

EVENTS = {"ds_write_b16": "w", "ds_write": "W", "ds_add": "A", "ds_read_u16": "r", "ds_read": "R", "; wave barrier": "|",
          "s_barrier": "#"}


@pytest.fixture(scope="module")
def lds_events(tmp_path_factory):
    """source, kernel -> the LDS accesses and barriers of each of its instances, in the order of the text."""
    d = tmp_path_factory.mktemp("lane_order")
    done = {}

    def events(source: str, kernel: str) -> dict[str, str]:
        if source not in done:
            out = d / (source + ".s")
            flags = [f for f in DEVICE_FLAGS if f != "-fPIC"] + SOURCE_FLAGS.get(source, [])
            subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(CSRC, source), "-o", str(out)],
                           check=True, capture_output=True)
            done[source] = out.read_text()
        found = {}
        for m in re.finditer(r"^(_ZN\S*" + kernel + r"\S*):.*?^\.Lfunc_end", done[source], re.S | re.M):
            seen = re.findall(r"^\s+(" + "|".join(EVENTS) + ")", m[0], re.M)
            found[m[1]] = "".join(EVENTS[e] for e in seen)
        assert found, f"no {kernel} in {source}"
        return found

    return events


def test_route_backward(lds_events):
    """Every lane's zeros, then the chosen experts' terms in other lanes' slots, then every lane's own."""
    found = lds_events("route.hip", "route_backward_kernel")
    assert len(found) == 21
    for name, seen in found.items():
        assert re.fullmatch(r"W+\|A+\|R+", seen), (name, seen)


@pytest.mark.parametrize("kernel,instances", [("sort_place_kernel", 7), ("sort_alone_kernel", 2)])
def test_sort(lds_events, kernel, instances):
    """A wave's 16-bit counters: their zeros, and each step's new counts, before the next step reads them.  (A step
    reads a count and may write it; where the waves' counts are summed eight are read, then eight written.)"""
    found = lds_events("sort.hip", kernel)
    assert len(found) == instances
    for name, seen in found.items():
        assert seen.startswith("W|"), (name, seen)
        assert seen.count("rw|") >= 4 and "rwr" not in seen, (name, seen)
