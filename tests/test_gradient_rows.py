"""Where the gradients of strided rows are put: in rows of their own width. A view of every n-th row of a larger tensor
(the last token of each sequence) does not ask for memory of that tensor's size."""
from types import SimpleNamespace

import pytest
import torch

from structured_sparse_gemm_nm_amd import heads, logprobs

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


def test_heads(monkeypatch):
    x, gamma, seen = view(3, 4 * 24, torch.float16), torch.ones(24, dtype=torch.float16), []
    plan = heads._plan(x, (2, 1, 1), 24, None, gamma, "halves", 1e-6)
    monkeypatch.setattr(heads, "nm_head_norm_rope_backward", lambda plan, x, q, k, at, table, dy, dx, **kw: seen.append(dx))
    ctx = SimpleNamespace(saved_tensors=(x, gamma, gamma, None, None), plan=plan, needs_input_grad=(True,) + (False,) * 7)
    dx = heads._NormRotate.backward(ctx, torch.zeros((3, 96), dtype=torch.float16))[0]
    assert seen[0] is dx and compact(dx, 3, 96) and plan.problem.ldg == 96 and plan.problem.ldx == FAR


def test_the_stride_of_the_heads_gradient():
    """0 is x's own; others keep the rules of the rows."""
    import structured_sparse_gemm_nm_amd as nm
    from tests.test_layer_ops import refused

    def plan(**kw):
        return nm.nm_heads_plan_init(**dict(dict(rows=8, heads_q=4, heads_k=2, heads_v=2, head_dim=64, rotary_dim=0), **kw))

    for kw, ld in ((dict(), 512), (dict(ldx=1024), 1024), (dict(ldx=1024, ldg=0), 1024), (dict(ldx=1024, ldg=520), 520)):
        assert plan(**kw)._back_specs[6][2] == ld
    plan(x_dtype="i32", ldx=516)                      # accumulators have no gradient
    refused(lambda: plan(ldg=511), nm.NM_ERR_SHAPE)
    refused(lambda: plan(ldg=-512), nm.NM_ERR_SHAPE)
    refused(lambda: plan(ldg=516), nm.NM_ERR_ALIGN)
    refused(lambda: plan(ldg=(1 << 46) + 8), nm.NM_ERR_SHAPE)
