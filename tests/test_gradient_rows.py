"""Where the gradients of strided rows are put: in rows of their own width. A view of every n-th row of a larger tensor
(the last token of each sequence) does not ask for memory of that tensor's size."""
from types import SimpleNamespace

import pytest
import torch

from structured_sparse_gemm_nm_amd import logprobs

FAR = 1 << 20       # elements between the rows of the view; nothing lies there


def view(rows, cols, dtype):
    return torch.empty((rows - 1) * FAR + cols, dtype=dtype).as_strided((rows, cols), (FAR, 1))


def compact(dx, rows, cols):
    step = 16 // dx.element_size()
    width = (cols + step - 1) // step * step
    return dx.shape == (rows, cols) and dx.stride() == (width, 1) and dx.untyped_storage().nbytes() <= rows * width * dx.element_size()


@pytest.mark.parametrize("cols", [1000, 1003])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_logits(cols, dtype, monkeypatch):
    x, seen = view(3, cols, dtype), []
    plan = logprobs._plan(x, 0, 1.0)
    monkeypatch.setattr(logprobs, "nm_logprobs_backward", lambda plan, x, tokens, stats, dx, **kw: seen.append(dx))
    ctx = SimpleNamespace(saved_tensors=(x, None, None, None), plan=plan)
    dx = logprobs._TokenLogprobs.backward(ctx, torch.ones(3), None)[0]
    assert seen[0] is dx and compact(dx, 3, cols) and plan.problem.ldg == dx.stride(0) and plan.problem.ldx == FAR
