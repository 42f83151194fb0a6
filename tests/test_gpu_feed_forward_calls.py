"""The feed-forward block's calls: a refused call leaves later calls as they were, plans are kept for the latest
numbers of tokens only, operands that want a gradient are refused, and small weights keep their values."""
import pytest
import torch

from structured_sparse_gemm_nm_amd.feed_forward import MOST_PLANS, CompressedFeedForward, Rows, _Weight
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


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-4, 1e-5, 1e-6, 1e-7])
def test_small_weights_keep_their_values(size, dtype):
    """Sixteen steps a row: an error of half a step, a seventh of the largest weight or f16's smallest step."""
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(48, 64, generator=g, device="cuda") * size).to(dtype)
    w[5] = 0
    packed = _Weight(w)
    d, o = packed.dense().double(), w.double()
    kept = d.new_zeros(48, 16, 4).scatter_(2, o.abs().reshape(48, 16, 4).sort(dim=2, descending=True, stable=True).indices[:, :, :2],
                                           1.0).reshape(48, 64) > 0
    assert (d[~kept] == 0).all() and (d[5] == 0).all()
    step = o.abs().amax(1, keepdim=True) / 7
    least = 2.0 ** -24 if dtype == torch.float16 else 0.0
    # the scale's own rounding moves the largest weight by 8 half steps of it
    half = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    bound = (step + least) / 2 + 8 * half * step
    assert ((d - o).abs() <= bound)[kept].all()
    # both products multiply by the same integers and scales
    codes = torch.randint(-127, 128, (4, 64), generator=g, device="cuda", dtype=torch.int32).to(torch.int8)
    scale = torch.full((4,), 1.0 / size, device="cuda")
    few, many = packed.product(codes, scale, True), packed.product(codes, scale, False)
    want = many.values.double() * scale.double()[:, None] * packed.scale.double()
    sizes = codes.double().abs() @ d.abs().t() * scale.double()[:, None]
    assert ((few.values.double() - want).abs() <= half * want.abs() + 32 * 2.0 ** -24 * sizes + 2.0 ** -25).all()
