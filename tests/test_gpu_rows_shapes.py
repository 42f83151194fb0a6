"""The row operators at the widths where the threads and pieces of a row change, with
row strides that no vector store fits, more rows than one grid dimension takes, and
magnitudes whose reciprocal is past fp32; tolerances as in tests/test_gpu_layer_ops.py."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from tests.test_gpu_layer_ops import CODE, row_check, row_inputs, row_run

pytestmark = pytest.mark.gpu

KINDS = [("16", None), ("16", "i8"), ("i32", None), ("i32", "i8")]


# 8 columns a thread: 64 threads up to 512, 1024 up to 8192, two pieces up to 16384, four up to 32768 (16 bits)
@pytest.mark.parametrize("cols", [505, 520, 1032, 3993, 8184, 8193, 8200, 12345, 16376, 16392, 20001, 32768, 32769, 33000])
@pytest.mark.parametrize("op", ["rmsnorm", "swiglu"])
def test_widths_where_the_split_changes(op, cols):
    for i, (x, y) in enumerate(KINDS):
        s = row_inputs(op, 2, cols, "f16" if i % 2 else "bf16", x, residual=i < 2, seed=cols + i)
        row_check(op, s, 2, cols, "f16" if i % 2 else "bf16", y, pad=16 * (i % 2))


@pytest.mark.parametrize("cols,ldy", [(9, 9), (15, 15), (8, 11), (7, 7), (1, 1), (13, 17)])
@pytest.mark.parametrize("op", ["rmsnorm", "swiglu"])
def test_short_rows_start_anywhere(op, cols, ldy):
    """Rows under 16 bytes need no alignment: 8-bit rows of 8 to 15 columns at odd strides."""
    rows = 37
    s = row_inputs(op, rows, cols, "f16", "16", True, 3)
    width = s["x"].shape[1]
    ldx = (width + 7) // 8 * 8
    x = torch.zeros((rows, ldx), dtype=torch.float16, device="cuda")[:, :width]
    x.copy_(s["x"])
    ld = (cols + 7) // 8 * 8
    plan = nm.nm_rows_plan_init(rows, cols, op=op, y_dtype="i8", ldx=ldx, ldy=ldy, ldr=ld, ldh=ld)
    raw = torch.full((rows * ldy + 64,), 93, dtype=torch.int8, device="cuda")
    y, scale = raw[:rows * ldy].view(rows, ldy)[:, :cols], torch.empty(rows, device="cuda")
    if op == "rmsnorm":
        res = torch.zeros((rows, ld), dtype=torch.float16, device="cuda")[:, :cols]
        res.copy_(s["residual"])
        nm.nm_rmsnorm(plan, x, s["gamma"].cuda(), y, y_scale=scale, residual=res)
    else:
        nm.nm_swiglu(plan, x, y, y_scale=scale)
    torch.cuda.synchronize()
    assert (raw[rows * ldy:] == 93).all() and (raw[:rows * ldy].view(rows, ldy)[:, cols:] == 93).all()
    want, ws, _ = row_run(op, s, rows, cols, "f16", "i8", 0, 1e-6, False)
    assert torch.equal(y, want) and torch.equal(scale, ws)


@pytest.mark.parametrize("op", ["rmsnorm", "swiglu"])
def test_more_rows_than_a_grid_dimension(op):
    rows, cols = (1 << 20) + 77, 8
    s = row_inputs(op, rows, cols, "bf16", "16", False, 4)
    row_check(op, s, rows, cols, "bf16", "i8")


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -64, 2.0 ** -100, 2.0 ** -122])
@pytest.mark.parametrize("cols", [40, 4096, 40000])
def test_codes_of_tiny_rows(size, cols):
    """127 / largest is past fp32 for the last: the codes are those of the row times a power of two."""
    s = row_inputs("rmsnorm", 3, cols, "bf16", "16", False, 5)
    s["x"] = s["x"].clamp(-4, 4)
    s["gamma"] = torch.ones_like(s["gamma"])
    # eps carries the mean in both, so the factor is the same and only the sizes differ
    big, bs, _ = row_run("rmsnorm", s, 3, cols, "bf16", "i8", 0, 2.0 ** 40, False)
    s["x"] = s["x"] * size
    assert (s["x"] != 0).any(1).all()
    got, gs, _ = row_run("rmsnorm", s, 3, cols, "bf16", "i8", 0, 2.0 ** 40, False)
    v = s["x"].double()
    top = v.abs().amax(1, keepdim=True)
    assert ((got.double().cpu() - v / top * 127).abs() <= CODE).all()
    if size >= 2.0 ** -100:                       # no subnormals: the same codes
        assert torch.equal(got, big)


def test_codes_of_tiny_activations():
    gate = torch.full((1, 64), 2.0 ** -66).bfloat16()
    up = (torch.arange(64) - 63).double() * 2.0 ** -60      # no ties: k 127 / 63 is never half a whole number
    s = dict(x=torch.cat((gate, up[None].bfloat16()), 1), row_scale=None, col_scale=None)
    got, scale, _ = row_run("swiglu", s, 1, 64, "bf16", "i8", 0, 0.0, False)
    assert torch.equal(got[0].double().cpu(), torch.round(up / 63 / 2.0 ** -60 * 127))
    assert float(scale[0]) == pytest.approx(2.0 ** -67 * 63 * 2.0 ** -60 / 127, rel=2.0 ** -15)


