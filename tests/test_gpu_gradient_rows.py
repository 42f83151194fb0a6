"""Gradients of rows that lie far apart in something larger: the same bits as those of rows of their own, in memory of
the rows' own size."""
import pytest
import torch

from structured_sparse_gemm_nm_amd.heads import norm_rotate, rotation_table
from structured_sparse_gemm_nm_amd.logprobs import token_logprobs

pytestmark = pytest.mark.gpu


def last(batch, steps, cols, dtype, seed):
    """(the last step's rows as a view of all, the same rows alone), both leaves of a graph."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    whole = torch.randn((batch, steps, cols), generator=g, device="cuda").to(dtype)
    alone = whole[:, -1].clone().requires_grad_()
    return whole[:, -1].detach().requires_grad_(), alone


def grown(step):
    """What a call's backward pass leaves allocated, in bytes."""
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    step()
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated() - before


@pytest.mark.parametrize("cols", [1000, 1024])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_last_logits(dtype, cols):
    view, alone = last(5, 600, cols, dtype, 1)
    at = torch.arange(5, device="cuda") * 7
    losses = []
    for x in (view, alone):
        out = token_logprobs(x, at, entropy=True)
        losses.append((out.logprob + 0.5 * out.entropy).sum())
    assert grown(losses[0].backward) < 1 << 20        # the whole is 6 MB and more
    losses[1].backward()
    assert torch.equal(view.grad, alone.grad) and view.grad.abs().sum() > 0


@pytest.mark.parametrize("rows", [1, 5])
def test_last_heads(rows):
    view, alone = last(rows, 6000, 8 * 64, torch.bfloat16, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    gains = [torch.randn(64, generator=g, device="cuda").bfloat16().requires_grad_() for _ in range(2)]
    at, table = torch.arange(rows, device="cuda") - 1, rotation_table(9, 64)
    dy = torch.randn((rows, 512), generator=g, device="cuda").bfloat16()
    y = norm_rotate(view, *gains, at, table, (4, 2, 2))
    assert grown(lambda: y.backward(dy)) < 1 << 20    # the whole is 6 MB and more
    got = [view.grad] + [t.grad.clone() for t in gains]
    for t in gains:
        t.grad = None
    norm_rotate(alone, *gains, at, table, (4, 2, 2)).backward(dy)
    assert all(torch.equal(a, b) for a, b in zip(got, [alone.grad] + [t.grad for t in gains])) and (got[0][0] == 0).all()
