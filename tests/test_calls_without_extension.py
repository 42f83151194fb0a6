"""The library without its call extension (another torch or Python than it was built for, or no host compiler):
everything loads and the layer operators' calls go through the checks in Python."""
import os
import subprocess
import sys

import pytest

from structured_sparse_gemm_nm_amd import build

SCRIPT = """
import sys, warnings
sys.modules["structured_sparse_gemm_nm_amd._nmcall"] = None          # its import fails
import torch
import structured_sparse_gemm_nm_amd as nm
with warnings.catch_warnings():
    warnings.simplefilter("error")
    assert nm.lib() is not None and nm.nm_version() > 0
    nm.nm_plan_init(64, 16, 64)                                      # does not use it, and does not warn
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    norm, gate, product = nm.nm_rows_plan_init(8, 64), nm.nm_rows_plan_init(8, 64, op="swiglu"), nm.nm_w4_plan_init(64, 4, 256)
assert len(w) == 3 and all("_nmcall" in str(x.message) and x.filename == __file__ for x in w), [(x.filename, str(x.message)) for x in w]
x = torch.zeros((8, 64), dtype=torch.float16)
for call in (lambda: nm.nm_rmsnorm(norm, x, x[0], x.clone()), lambda: nm.nm_swiglu(gate, torch.cat((x, x), 1), x),
             lambda: nm.nm_w4_matvec(product, product.empty_packed(device="cpu"), torch.zeros((4, 256)).half(), torch.zeros((4, 64)).half())):
    try:
        call()
    except ValueError as e:
        assert "GPU" in str(e)
    else:
        raise AssertionError("a host tensor was taken")
for call in (lambda: nm.nm_rmsnorm(norm, 0x10000, 0x10000, None, stream=0), lambda: nm.nm_swiglu(gate, 0x10000, None, stream=0),
             lambda: nm.nm_w4_matvec(product, 0x10000, 0x10000, None, stream=0)):
    try:
        call()
    except nm.NmError as e:
        assert e.status == nm.NM_ERR_INVALID_ARG
    else:
        raise AssertionError("a missing output was taken")
norm.destroy(), gate.destroy(), product.destroy()
print("without the extension: ok")
"""


def test_the_library_loads_without_the_extension(tmp_path):
    script = tmp_path / "without.py"
    script.write_text(SCRIPT)
    r = subprocess.run([sys.executable, str(script)], capture_output=True, text=True, cwd=build.HERE + "/..",
                       env=dict(os.environ, PYTHONPATH=build.HERE + "/.."))
    assert r.returncode == 0 and "without the extension: ok" in r.stdout, r.stdout + r.stderr


def test_the_library_is_built_before_the_extension_is_missed(monkeypatch, tmp_path):
    """A failing host compiler is reported after the library is in its place."""
    done = []

    def fails():
        raise RuntimeError("no host compiler")

    class Linked:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        done.append("library")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Linked()

    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objs"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libnmsparse.so"))
    monkeypatch.setattr(build, "_m0_check", lambda: None)
    monkeypatch.setattr(build, "_compile", lambda src: src + ".o")
    monkeypatch.setattr(build, "_link", lambda *a: done.append("calibration"))
    monkeypatch.setattr(build, "_build_call", fails)
    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="no host compiler"):
        build.build(verbose=False)
    assert done == ["calibration", "library"] and (tmp_path / "libnmsparse.so").exists()


def test_an_older_extension_does_not_outlive_a_failed_build(monkeypatch, tmp_path):
    old = tmp_path / "_nmcall.so"
    old.write_text("older")
    monkeypatch.setattr(build, "CALL_LIB", str(old))

    class Failed:
        returncode, stdout, stderr = 1, "", "no headers"

    monkeypatch.setattr(build.subprocess, "run", lambda *a, **kw: Failed())
    with pytest.raises(RuntimeError, match="no headers"):
        build._build_call()
    assert not old.exists()
