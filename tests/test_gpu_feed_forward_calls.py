"""The feed-forward block's calls: a refused call leaves later calls as they were, plans are kept for the latest
numbers of tokens only, and operands that want a gradient are refused."""
import pytest
import torch

from structured_sparse_gemm_nm_amd.feed_forward import MOST_PLANS, CompressedFeedForward, Rows
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


def test_plans_are_kept_for_the_latest_numbers_of_tokens():
    ff, _, _ = block(32, 48, torch.bfloat16)
    x, r = inputs(700, 32, torch.bfloat16)
    first, _ = ff(x[:3], r[:3])
    for n in range(1, 701):
        ff(x[:n], r[:n], few=True)
        if n % 7 == 0:
            ff(x[:n], r[:n], few=False)
    for plans in (ff._plans, ff.gate_up._plans, ff.down._plans):
        assert 0 < len(plans) <= MOST_PLANS
    again, _ = ff(x[:3], r[:3])
    assert torch.equal(again.values, first.values)


def test_inputs_that_want_a_gradient_are_refused():
    ff, _, _ = block(64, 96, torch.float16)
    x, r = inputs(3, 64, torch.float16)
    want, h = ff(x, r)
    wants = x.clone().requires_grad_()
    for a, b in ((wants, r), (x, wants), (Rows(wants), None)):
        with pytest.raises(RuntimeError, match="gradient"):
            ff(a, b)
    with torch.no_grad():
        y, hh = ff(wants, r)
    assert torch.equal(y.values, want.values) and torch.equal(hh, h)


def test_the_block_keeps_gamma_as_a_constant():
    _, gate_up, down = block(64, 96, torch.float16)
    gamma = torch.nn.Parameter(torch.ones(64, dtype=torch.float16, device="cuda"))
    ff = CompressedFeedForward(gamma, torch.nn.Parameter(gate_up), torch.nn.Parameter(down))
    y, h = ff(*inputs(3, 64, torch.float16))
    assert not (ff.gamma.requires_grad or y.values.requires_grad or h.requires_grad)
