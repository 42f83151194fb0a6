"""The 4-bit product's lanes hand values to other lanes of their wave through LDS. In the built units a wave
barrier (no instruction, an order for the compiler) or a block's barrier stands between such writes and the
reads after them, and between reads and the writes that come over what they read."""
import os
import re

import pytest

from structured_sparse_gemm_nm_amd import build

UNITS = ("nm_w4_f16", "nm_w4_bf16", "nm_w4_i8", "nm_w4_i8_bf16")


def unordered(lines):
    """Pairs of LDS accesses without a barrier between, in the order of the text. Writes that a block's barrier
    follows may stand after reads: they go to the part that all waves read afterwards."""
    steps = []
    for line in lines:
        t = line.strip()
        if t.startswith("; wave barrier"):
            steps.append("wave")
        elif t.startswith("s_barrier"):
            steps.append("block")
        elif re.match(r"ds_(read|write)", t):
            steps.append(t.split()[0][3:7])
    bad = []
    for i, (a, b) in enumerate(zip(steps, steps[1:])):
        if a == "writ" and b == "read":
            bad.append(i)
        if a == "read" and b == "writ" and next((s for s in steps[i + 1:] if s != "writ"), None) != "block":
            bad.append(i)
    return bad


@pytest.mark.parametrize("steps,count", [
    ("", 0), ("w w b r r b w b r", 0), ("w w s r", 0), ("w r", 1), ("b w b r w b r", 1), ("b w b r r w w s r", 0), ("b w b r w r s", 2),
])
def test_the_reading_of_the_assembly(steps, count):
    text = {"w": "\tds_write_b64 v1, v[2:3]", "r": "\tds_read_b128 v[0:3], v4 offset:16", "b": "\t; wave barrier", "s": "\ts_barrier"}
    assert len(unordered([text[s] for s in steps.split()])) == count


@pytest.mark.parametrize("unit", UNITS)
def test_the_built_units_order_their_lds(unit):
    asm = os.path.join(build.BUILD, "%s-hip-amdgcn-amd-amdhsa-%s.s" % (unit, build.ARCH))
    if not os.path.exists(asm):
        pytest.skip("library not built here")
    kernels, name = {}, None
    for line in open(asm):
        m = re.match(r"(_ZN2nm9w4_kernel\w+):", line)
        if m:
            name = m.group(1)
            kernels[name] = []
        elif name:
            kernels[name].append(line)
            if line.strip().startswith(".Lfunc_end"):
                name = None
    assert kernels
    for name, lines in kernels.items():
        assert any("ds_write" in line for line in lines)
        assert not unordered(lines), name
