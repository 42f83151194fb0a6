"""Shared memory that the adapters' and the log probabilities' kernels read in vectors of 16 bytes says so itself: read from
the device code's IR, where a variable has the alignment that the source gives it."""
import os
import re
import subprocess

import pytest

from structured_sparse_gemm_nm_amd import build


@pytest.mark.parametrize("unit,name,least", [("nm_lora", "E2ts", 64), ("nm_logprobs", "E3lds", 16)])
def test_vectors_of_16_bytes(unit, name, least, tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc here")
    ir = str(tmp_path / "unit.ll")
    cmd = [build.HIPCC] + build.CFLAGS + ["--cuda-device-only", "-S", "-emit-llvm", os.path.join(build.CSRC, unit + ".hip"), "-o", ir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"^@\S*%s = [^=]*addrspace\(3\) global .*, align (\d+)$" % name, open(ir).read(), re.M)
    assert len(found) >= least and {int(a) % 16 for a in found} == {0}
