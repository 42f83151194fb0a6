"""8-bit rows of 8 to 15 columns may start at any byte (rows under 16 bytes have no alignment rule), so the row
operators' 8-byte stores must not promise the compiler more than that. Read from the device code's IR."""
import os
import re
import subprocess

import pytest

from structured_sparse_gemm_nm_amd import build


def test_stores_of_eight_codes_promise_no_alignment(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc here")
    ir = str(tmp_path / "rowops.ll")
    cmd = [build.HIPCC] + build.CFLAGS + ["--cuda-device-only", "-S", "-emit-llvm", os.path.join(build.CSRC, "nm_rowops.hip"), "-o", ir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    stores = re.findall(r"store (\S+ x \S+|\S+) \S+, ptr addrspace\(1\) [^,]*, align (\d+)", open(ir).read())
    eight = [int(a) for t, a in stores if t in ("<2 x i32>", "i64", "<8 x i8>")]
    assert len(eight) >= 16 and set(eight) == {1}
