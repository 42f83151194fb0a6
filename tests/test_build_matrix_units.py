"""The build's check of the matrix instructions' wait states over all units that hold such instructions, and what it
counts between two of them."""
import os
import re

import pytest

from structured_sparse_gemm_nm_amd import build

SMALL = "v_mfma_f32_16x16x32_f16 v[0:3], v[4:7], v[8:11], v[0:3]"
LARGE = "v_mfma_f32_32x32x16_f16 v[0:15], v[16:19], v[20:23], v[0:15]"
SPARSE = "v_smfmac_i32_16x16x128_i8 v[0:3], v[4:7], v[8:15], v16"


@pytest.mark.parametrize("lines,count", [
    ([SPARSE, "s_nop 7", "v_cvt_f32_i32_e32 v20, v0"], 0),
    ([SPARSE, "s_nop 6", "v_cvt_f32_i32_e32 v20, v0"], 1),
    # the early return that a loop's last sums go through
    ([SPARSE, "s_cbranch_scc1 .L1", "s_nop 7", ".L1:", "v_mov_b32_e32 v20, 0", "v_mov_b32_e32 v21, 0", "v_cvt_f32_i32_e32 v20, v0"], 1),
    # twice the passes for 32x32
    ([LARGE, "s_nop 11", "v_add_f32_e32 v30, v0, v1"], 0),
    ([LARGE, "s_nop 10", "v_add_f32_e32 v30, v0, v1"], 1),
    # a sum that goes on, in the same registers or in others
    ([SMALL, SMALL, "s_nop 7", "v_add_f32_e32 v30, v0, v1"], 0),
    ([SMALL, "v_mfma_f32_16x16x32_f16 v[40:43], v[4:7], v[8:11], v[0:3]", "s_nop 7", "v_add_f32_e32 v30, v40, v0"], 0),
    ([SMALL, "v_mfma_f32_16x16x32_f16 v[40:43], v[4:7], v[8:11], v[2:5]", "s_nop 7"], 1),
    # a result as another's A, B or index
    ([SMALL, "v_mfma_f32_16x16x32_f16 v[40:43], v[0:3], v[8:11], v[40:43]"], 1),
    ([SMALL, "v_mfma_f32_16x16x32_f16 v[40:43], v[8:11], v[0:3], v[40:43]"], 1),
    ([SMALL, "s_nop 7", "v_mfma_f32_16x16x32_f16 v[40:43], v[8:11], v[0:3], v[40:43]"], 0),
    ([SMALL, "v_smfmac_i32_16x16x128_i8 v[40:43], v[4:7], v[8:15], v3"], 1),
    ([SPARSE, "v_smfmac_i32_16x16x128_i8 v[40:43], v[0:3], v[8:15], v16"], 1),
])
def test_the_reading_of_two_instructions(lines, count, tmp_path):
    asm = tmp_path / "unit.s"
    asm.write_text("kernel:\n" + "\n".join(lines) + "\n")
    assert len(build.check_matrix_waits(str(asm))) == count


def _text(name):
    return open(os.path.join(build.CSRC, name)).read()


def test_every_unit_with_matrix_instructions_is_read():
    """By the sources: a unit that holds the instructions' builtins, or includes a header that does."""
    def holds(name):
        return re.search(r"__builtin_amdgcn_s?mf\w+", _text(name)) or any(
            holds(h) for h in re.findall(r'#include "(nm_\w+\.h)"', _text(name)))

    units = {u for u in build.SOURCES + ["nm_calib.hip"] if holds(u)}
    without = {u for u in build.SOURCES if u == "nm_gemm.hip" or u.startswith("nm_skinny")}      # the vector kernels
    assert units - without == set(build.MATRIX_SOURCES)


@pytest.mark.parametrize("unit", [s[:-4] for s in build.SOURCES if s.startswith("nm_w4_")])
def test_the_four_bit_products_wait(unit):
    asm = os.path.join(build.BUILD, "%s-hip-amdgcn-amd-amdhsa-%s.s" % (unit, build.ARCH))
    if not os.path.exists(asm):
        pytest.skip("library not built here")
    assert any("v_smfmac" in line for line in open(asm))
    assert not build.check_matrix_waits(asm)
