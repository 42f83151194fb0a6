"""The 4-bit product at the ends of bf16's range, against the same 64-bit computation and with the same tolerances
as tests/test_gpu_layer_ops.py. A sum over a group that fp32 holds stays finite, with zero points and without."""
import pytest
import torch

from tests.test_gpu_layer_ops import close, w4_exact, w4_inputs, w4_run, w4_tolerance

pytestmark = pytest.mark.gpu


def large(m, n, k, group, x, sparse, zeros):
    """One strong activation every 256 columns, which meets codes 0 and 15 in the kept positions."""
    s = w4_inputs(m, n, k, group, "bf16", x, sparse, zeros, 31)
    if zeros:
        s["zeros"] = torch.full_like(s["zeros"], 8)
    if sparse:
        s["pairs"][:, :, 0], s["pairs"][:, :, 1] = 0, 2
    half = 2 if sparse else 1
    s["x"] = torch.zeros_like(s["x"])
    s["x"][:, ::256] = 127 if x == "i8" else 2.0 ** 122
    s["x"][1:, 256::512] *= -1                                     # the second token's meet with both signs
    s["q"][:, ::256 // half] = torch.randint(0, 2, s["q"][:, ::256 // half].shape, generator=torch.Generator().manual_seed(5),
                                             dtype=torch.uint8) * 15
    return s


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("group", [0, 128, 256, 512])
def test_strong_activations(group, sparse, zeros):
    """8 * 2^122 and its sums fit fp32, sixteen times that does not; the scales bring y down to 2^110 and less."""
    for m, n in ((48, 2), (4100, 2), (40, 9), (33, 20)):
        s = large(m, n, 1300, group, "16", sparse, zeros)
        s["scales"] = torch.full_like(s["scales"], 2.0 ** -16)
        y, size = w4_exact(s, 1300, group)
        got = w4_run(s, m, n, 1300, group, "bf16", "16")
        assert torch.isfinite(got).all()
        close(got, y, w4_tolerance(y, size, 1300, "bf16"), "y")


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("group", [0, 256, 512])
def test_strong_scales(group, sparse, zeros):
    """8-bit activations: sums of scale * whole number up to 2^127, brought down by the token's scale."""
    for m, n in ((48, 2), (4100, 2), (40, 9), (33, 20)):
        s = large(m, n, 1300, group, "i8", sparse, zeros)
        s["scales"] = torch.full_like(s["scales"], 2.0 ** 114)     # at most 6 strong columns: 6 * 8 * 127 * 2^114 < 2^127
        s["x_scale"] = torch.full((n,), 2.0 ** -30)
        y, size = w4_exact(s, 1300, group)
        got = w4_run(s, m, n, 1300, group, "bf16", "i8")
        assert torch.isfinite(got).all()
        close(got, y, w4_tolerance(y, size, 1300, "bf16"), "y")


@pytest.mark.parametrize("x", ["16", "i8"])
@pytest.mark.parametrize("sparse", [False, True])
def test_small_scales_are_not_lost(x, sparse):
    """Scales at bf16's smallest values, activations that bring y back: nothing is flushed on the way."""
    group = 256
    for m, n in ((48, 2), (40, 9)):
        s = large(m, n, 1300, group, x, sparse, False)
        s["scales"] = torch.full_like(s["scales"], 2.0 ** -126)
        if x == "i8":
            s["x_scale"] = torch.full((n,), 2.0 ** 60)
        y, size = w4_exact(s, 1300, group)
        assert (y.abs() > 0).any()
        close(w4_run(s, m, n, 1300, group, "bf16", x), y, w4_tolerance(y, size, 1300, "bf16"), "y")


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("power", [-110, -122, -126])
def test_weak_activations(power, sparse, zeros):
    """Products down to the smallest normal bf16 value times a code, brought back by the scales."""
    for m, n, group in ((48, 2, 0), (4100, 2, 128), (40, 9, 64), (33, 20, 256)):
        s = w4_inputs(m, n, 1300, group, "bf16", "16", sparse, zeros, 32)
        s["x"] = (torch.sign(s["x"].float()) * (1 + s["x"].float().abs() % 1) * 2.0 ** power).bfloat16()
        s["scales"] = torch.full_like(s["scales"], 2.0 ** 110)
        y, size = w4_exact(s, 1300, group)
        # fp32's smallest step, 2^-149, half of it in each of the sums of products before a scale
        close(w4_run(s, m, n, 1300, group, "bf16", "16"), y,
              w4_tolerance(y, size, 1300, "bf16") + 1300 * 2.0 ** -150 * 2.0 ** 110 * 16, "y")
