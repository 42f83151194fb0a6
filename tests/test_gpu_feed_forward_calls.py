"""The feed-forward block's calls: a refused call leaves later calls as they were."""
import pytest
import torch

from structured_sparse_gemm_nm_amd.feed_forward import Rows
from tests.test_gpu_feed_forward import block, inputs

pytestmark = pytest.mark.gpu


def accumulators(n, hidden):
    g = torch.Generator(device="cuda").manual_seed(9)
    return Rows(torch.randint(-90000, 90000, (n, hidden), generator=g, device="cuda", dtype=torch.int32),
                0.02 + 0.02 * torch.rand(n, generator=g, device="cuda"),
                2e-4 + 3e-4 * torch.rand(hidden, generator=g, device="cuda"))


@pytest.mark.parametrize("few", [True, False])
def test_a_refused_call_leaves_later_calls_as_they_were(few):
    ff, _, _ = block(64, 96, torch.float16)
    other, _, _ = block(64, 96, torch.float16)
    x, r = inputs(5, 64, torch.float16)
    acc = accumulators(5, 64)
    for bad in (Rows(acc.values), Rows(acc.values, acc.row_scale), Rows(acc.values, None, acc.col_scale),
                Rows(x, acc.row_scale, acc.col_scale), Rows(x, None, acc.col_scale), x.bfloat16(), x.float(), x[:, :32], x[0]):
        with pytest.raises(ValueError):
            ff(bad, r, few=few)
    for good in (x, acc):
        (y, h), (want, hw) = ff(good, r, few=few), other(good, r, few=few)
        assert torch.equal(y.values, want.values) and torch.equal(h, hw)
