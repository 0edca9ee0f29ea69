"""Properties of the operators' gfx950 code: what tests/test_codegen.py holds
for the collectives' (no packed fp32 arithmetic, no writes through the scalar
data cache), global and not flat accesses, nothing spilled, and no kernel
whose registers live in memory."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from test_codegen import CSRC, PACKED, SCALAR_WRITES, hipcc

pytestmark = pytest.mark.skipif(hipcc is None, reason="hipcc not available")

SOURCES = ["route.hip", "sort.hip", "dispatch.hip", "embedding.hip", "grads.hip"]


@pytest.fixture(scope="module")
def asm(tmp_path_factory) -> dict[str, str]:
    from copy_reduce_snac_amd.build import DEVICE_FLAGS, SOURCE_FLAGS

    d = tmp_path_factory.mktemp("ops_asm")
    flags = [f for f in DEVICE_FLAGS if f not in ("-fPIC",)]
    procs = {}
    for name in SOURCES:
        out = d / (name + ".s")
        cmd = [hipcc, *flags, *SOURCE_FLAGS.get(name, []), "--cuda-device-only", "-S", os.path.join(CSRC, name), "-o", str(out)]
        procs[name] = (out, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE))
    res = {}
    for name, (out, p) in procs.items():
        _, err = p.communicate()
        assert p.returncode == 0, f"{name}: {err.decode()[-2000:]}"
        res[name] = out.read_text()
    return res


@pytest.mark.parametrize("src", SOURCES)
def test_code(asm, src):
    text = asm[src]
    for op in PACKED:
        assert op not in text, f"{op} emitted"
    assert not SCALAR_WRITES.findall(text)
    assert not re.search(r"^\s*flat_(load|store)", text, re.M), "flat accesses"
    assert not re.search(r"\.vgpr_spill_count:\s*[1-9]", text), "spilled vector registers"
    assert not re.search(r"\.private_segment_fixed_size:\s*[1-9]", text), "scratch memory"
