"""The norm of rows of many millions of columns.

Tolerance of the scale: the sum of squares takes 8 additions in a piece, 2 roundings where pieces join in 64 bits
and 10 over the block; half of that after the square root, under 10 for the rest: 2^-19 = 32 steps."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from tests.test_gpu_layer_ops import TORCH, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1 << 24, (1 << 24) + 3])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_norm_of_many_millions_of_columns(cols, dtype):
    """A constant row: a plain fp32 sum of 2^14 such squares a thread is off by 2^-13 and more."""
    values = torch.tensor([0.7, 1.06, 3.3]).to(TORCH[dtype])
    rows, ld = 3, (cols + 15) // 16 * 16
    x = torch.empty((rows, ld), dtype=TORCH[dtype], device="cuda")
    x[:] = values.cuda()[:, None]
    plan = nm.nm_rows_plan_init(rows, cols, dtype=dtype, y_dtype="i8", ldx=ld, ldy=ld, ldr=ld, ldh=ld, eps=1e-6)
    y, scale = torch.zeros((rows, ld), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    gamma = torch.ones(cols, dtype=TORCH[dtype], device="cuda")
    nm.nm_rmsnorm(plan, x[:, :cols], gamma, y[:, :cols], y_scale=scale)
    v = values.double()
    want = v / (v * v + float(torch.tensor(1e-6))).sqrt() / 127
    close(scale, want, want * 2.0 ** -19, "y_scale")
    assert (y[:, :cols] == 127).all() and (y[:, cols:] == 0).all()
