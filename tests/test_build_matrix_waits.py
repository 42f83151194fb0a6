"""The build's check that no instruction uses a matrix instruction's result before its wait states have passed, on
hand-written assembly and on the built unit."""
import os

import pytest

from structured_sparse_gemm_nm_amd import build

MFMA = "v_mfma_f32_16x16x32_f16 v[0:3], v[4:7], v[8:11], v[0:3]"


@pytest.mark.parametrize("lines,count", [
    ([MFMA, "s_nop 7", "ds_write_b128 v57, v[0:3]"], 0),
    ([MFMA, "s_nop 6", "ds_write_b128 v57, v[0:3]"], 1),
    ([MFMA, "s_andn2_b64 vcc, exec, s[42:43]", "ds_write_b128 v57, v[0:3]"], 1),
    ([MFMA, MFMA, "s_nop 7", "v_add_f32_e32 v12, v0, v1"], 0),
    ([MFMA, MFMA, "v_add_f32_e32 v12, v0, v1"], 1),
    ([MFMA] + ["v_add_f32_e32 v12, v13, v14"] * 8 + ["v_mul_f32_e32 v12, v3, v3"], 0),
    ([MFMA] + ["v_add_f32_e32 v12, v13, v14"] * 7 + ["v_mul_f32_e32 v12, v3, v3"], 1),
    ([MFMA, "v_mov_b32_e32 v2, 0"], 1),                                  # written over before it arrives
    ([MFMA, "s_cbranch_scc1 .L2", "s_nop 7", "s_branch .L3", ".L2:", "ds_write_b128 v57, v[0:3]", ".L3:"], 1),
    ([".L1:", "global_store_dword v[20:21], v1, off", MFMA, "s_cbranch_scc1 .L1", "s_nop 7"], 1),
    ([MFMA, "s_endpgm", "ds_write_b128 v57, v[0:3]"], 0),
    (["v_mfma_f32_16x16x32_f16 a[0:3], v[4:7], v[8:11], a[0:3]", "v_accvgpr_read_b32 v0, a1"], 1),
    ([MFMA, "v_mfma_f32_16x16x32_f16 v[12:15], v[4:7], v[8:11], v[12:15]", "s_nop 7", "v_add_f32_e32 v12, v0, v1"], 0),
])
def test_the_reading_of_the_assembly(lines, count, tmp_path):
    asm = tmp_path / "unit.s"
    asm.write_text("kernel:\n" + "\n".join(lines) + "\n")
    assert len(build.check_matrix_waits(str(asm))) == count


@pytest.mark.parametrize("source", build.MATRIX_SOURCES)
def test_the_built_units(source):
    asm = os.path.join(build.BUILD, "%s-hip-amdgcn-amd-amdhsa-%s.s" % (source[:-4], build.ARCH))
    if not os.path.exists(asm):
        pytest.skip("library not built here")
    assert any("v_mfma" in line for line in open(asm))
    assert not build.check_matrix_waits(asm)
