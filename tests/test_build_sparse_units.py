"""The build checks the operands of sparse matrix instructions in every unit that holds some: the others, read from
the device code of their objects, hold none."""
import os
import subprocess

import pytest

from structured_sparse_gemm_nm_amd import build

LLVM = os.path.dirname(build.CLANG)
BUNDLER, OBJCOPY, OBJDUMP = (os.path.join(LLVM, t) for t in ("clang-offload-bundler", "llvm-objcopy", "llvm-objdump"))


def test_calibration_loops_are_checked():
    text = open(os.path.join(build.CSRC, "nm_calib.hip")).read()
    assert "__builtin_amdgcn_smfmac" in text and "nm_calib.hip" in build.SPARSE_SOURCES


@pytest.mark.parametrize("src", [s for s in build.SOURCES + ["nm_calib.hip"] if s not in build.SPARSE_SOURCES])
def test_no_other_unit_holds_sparse_instructions(src, tmp_path):
    obj = os.path.join(build.BUILD, os.path.splitext(src)[0] + ".o")
    if not os.path.exists(obj) or not all(os.path.exists(t) for t in (BUNDLER, OBJCOPY, OBJDUMP)):
        pytest.skip("library not built here")
    bundle, code = str(tmp_path / "bundle"), str(tmp_path / "device.o")
    run = lambda *cmd: subprocess.run(cmd, capture_output=True, text=True, check=True).stdout  # noqa: E731
    run(OBJCOPY, "--dump-section=.hip_fatbin=" + bundle, obj, str(tmp_path / "copy.o"))
    run(BUNDLER, "--unbundle", "--type=o", "--targets=hipv4-amdgcn-amd-amdhsa--" + build.ARCH, "--input=" + bundle, "--output=" + code)
    text = run(OBJDUMP, "-d", code)
    if "__global__" in open(os.path.join(build.CSRC, src)).read():
        assert "s_endpgm" in text
    assert "v_smfmac" not in text
