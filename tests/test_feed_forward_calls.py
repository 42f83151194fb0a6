"""Host side of the feed-forward block: what a call refuses before a plan is made, and which plan a call is given."""
import pytest
import torch

from structured_sparse_gemm_nm_amd.feed_forward import MOST_PLANS, CompressedFeedForward, Rows, _Plans


def block(dtype=torch.float16, hidden=32, inner=48):
    """A block without weights: calls reach its checks and its row operators' plans."""
    ff = CompressedFeedForward.__new__(CompressedFeedForward)
    ff.hidden, ff.inner, ff.dtype, ff.eps, ff._plans = hidden, inner, dtype, 1e-6, _Plans()
    ff.gamma = torch.ones(hidden, dtype=dtype)
    return ff


X, ACC = torch.zeros((4, 32), dtype=torch.float16), torch.zeros((4, 32), dtype=torch.int32)
ROW, COL = torch.ones(4), torch.ones(32)


@pytest.mark.parametrize("bad", [
    Rows(ACC), Rows(ACC, ROW), Rows(ACC, None, COL), Rows(X, ROW, COL), Rows(X, None, COL), Rows(X, ROW), X.bfloat16(),
    X.float(), X[:, :16], X[0], X[None], Rows(ACC[:, :16], ROW, COL[:16]),
])
def test_refused_before_a_plan_is_made(bad):
    ff = block()
    with pytest.raises(ValueError):
        ff(bad)
    assert len(ff._plans) == 0


def test_a_plan_follows_the_type_of_the_values():
    ff = block()
    for op, cols in (("rmsnorm", 32), ("swiglu", 48)):
        for values, scales, dtype in ((ACC, (ROW, COL), torch.int32), (X, (), torch.float16), (ACC, (), torch.int32)):
            plan = ff._rows(op, 4, cols, Rows(values, *scales))
            assert plan.x_dtype is dtype and plan is ff._rows(op, 4, cols, Rows(values, *scales))


def test_plans_of_the_latest_calls_are_kept():
    ff = block()
    first = ff._rows("rmsnorm", 1, 32, Rows(X))
    for n in range(2, 2 * MOST_PLANS):
        ff._rows("rmsnorm", n, 32, Rows(X))
        assert ff._rows("rmsnorm", 1, 32, Rows(X)) is first            # used between the others
        assert len(ff._plans) <= MOST_PLANS
    last = ff._rows("rmsnorm", 2 * MOST_PLANS - 1, 32, Rows(X))
    assert ff._rows("rmsnorm", 2 * MOST_PLANS - 1, 32, Rows(X)) is last and len(ff._plans) == MOST_PLANS


def test_a_plan_that_cannot_be_made_is_not_kept():
    plans = _Plans()
    with pytest.raises(ZeroDivisionError):
        plans.get(1, lambda: 1 // 0)
    assert len(plans) == 0 and plans.get(1, lambda: 5) == 5 and plans.get(1, lambda: 6) == 5


def test_operands_that_want_a_gradient_are_refused():
    ff, wants = block(), X.clone().requires_grad_()
    for x, residual in ((wants, None), (X, wants), (Rows(ACC, ROW.clone().requires_grad_(), COL), None), (Rows(wants), X)):
        with pytest.raises(RuntimeError, match="gradient"):
            ff(x, residual)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):    # past that check, and on to the next: host tensors
            ff(x, residual)
