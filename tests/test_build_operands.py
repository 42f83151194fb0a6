"""The build's check that no sparse matrix instruction writes over the registers it
reads as A or B, on hand-written assembly and on the built units."""
import os

import pytest

from structured_sparse_gemm_nm_amd import build

OK = """\
kernel:
\tv_smfmac_i32_16x16x128_i8 v[28:31], v[20:23], v[4:11], v68
\tv_smfmac_f32_32x32x32_f16 a[0:15], v[20:23], v[0:7], v68 cbsz:1 ; a and v are different registers
\tv_mfma_f32_16x16x32_f16 v[32:35], v[32:35], v[36:39], 0
\ts_endpgm
"""


def check(tmp_path, text):
    p = tmp_path / "k.s"
    p.write_text(text)
    return build.check_sparse_operands(str(p))


def test_sound_code_passes(tmp_path):
    assert check(tmp_path, OK) == []


@pytest.mark.parametrize("line", [
    "v_smfmac_i32_16x16x128_i8 v[28:31], v[20:23], v[24:31], v68",
    "v_smfmac_i32_16x16x128_i8 v[24:27], v[20:23], v[17:24], v69",
    "v_smfmac_f32_16x16x64_f16 v[20:23], v[20:23], v[0:7], v69",
    "v_smfmac_f32_16x16x64_f16 v[20:23], v[17:20], v[0:7], v69",
])
def test_overwritten_operands_are_reported(tmp_path, line):
    assert check(tmp_path, OK.replace("\ts_endpgm", "\t" + line + "\n\ts_endpgm")) == [line]


def test_the_built_units_pass():
    for src in build.SPARSE_SOURCES:
        asm = os.path.join(build.BUILD, "%s-hip-amdgcn-amd-amdhsa-%s.s" % (os.path.splitext(src)[0], build.ARCH))
        if not os.path.exists(asm):
            pytest.skip("library not built here")
        assert any("v_smfmac" in line for line in open(asm)) and build.check_sparse_operands(asm) == []
