"""The gradient of rows whose token is past the vocabulary: NaN as its log probability is, but 0 where no gradient comes in."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("cols", [9, 4096])
def test_a_token_past_the_vocabulary(dtype, cols):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros((6, (cols + 7) // 8 * 8), dtype=dtype, device="cuda")[:, :cols]
    x.copy_(torch.randn((6, cols), generator=g, device="cuda"))
    tokens = torch.tensor([0, cols, cols + 5, cols, 1 << 40, cols - 1], device="cuda")
    plan = nm.nm_logprobs_plan_init(6, cols, dtype="f16" if dtype is torch.float16 else "f32", ldx=x.stride(0))
    lp, H, stats = torch.empty(6, device="cuda"), torch.empty(6, device="cuda"), torch.empty((6, 2), device="cuda")
    dx = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device="cuda")
    nm.nm_logprobs(plan, x, tokens, lp, entropy=H, stats=stats, workspace=plan.empty_workspace())
    assert lp[1:5].isnan().all() and lp[[0, 5]].isfinite().all()
    gl, gh = torch.tensor([1.0, 1.0, 0.0, -0.0, 0.0, 2.0], device="cuda"), torch.tensor([0.0, 0.0, 0.0, 0.0, 0.5, 0.0], device="cuda")
    nm.nm_logprobs_backward(plan, x, tokens, stats, dx, g_logprob=gl)
    assert dx[1].isnan().all() and (dx[2:5] == 0).all() and dx[[0, 5]].isfinite().all()
    nm.nm_logprobs_backward(plan, x, tokens, stats, dx, g_logprob=gl, g_entropy=gh, entropy=H)
    assert dx[1].isnan().all() and (dx[2:4] == 0).all() and dx[[0, 4, 5]].isfinite().all() and (dx[4] != 0).any()
