"""What infinities and NaN leave in a row of the row operators, and the range of 8-bit codes; tolerances as in
tests/test_gpu_layer_ops.py."""
import pytest
import torch

from tests.test_gpu_layer_ops import CODE, close, row_exact, row_inputs, row_run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["rmsnorm", "swiglu"])
@pytest.mark.parametrize("cols", [72, 3000, 17000, 40000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_an_infinity_or_nan_leaves_in_its_row(op, cols, bad):
    """The formula's value in 16 bits; in 8 bits a scale that is no number or infinite, codes from -127 to 127,
    and no number where the code and the scale are multiplied."""
    s = row_inputs(op, 3, cols, "bf16", "16", False, 40)
    s["x"][1, cols // 2] = bad
    got, _, _ = row_run(op, s, 3, cols, "bf16", None, 0, 1e-6, False)
    value = float(got[1, cols // 2])
    if op == "swiglu" and bad == float("inf"):
        assert value == float(torch.sign(s["x"][1, cols + cols // 2].float())) * float("inf")
    else:
        assert value != value                                       # NaN, inf / inf, -inf * 0
    codes, scale, _ = row_run(op, s, 3, cols, "bf16", "i8", 0, 1e-6, False)
    assert int(codes.int().abs().max()) == 127                      # of the two rows beside it
    assert not torch.isfinite(scale[1]) and torch.isfinite(scale[[0, 2]]).all()
    assert torch.isnan(codes[1, cols // 2].float() * scale[1])


def test_codes_stay_within_127_where_the_largest_is_rounded_down():
    """127 / a times a may round past 127, never to 128 or -128."""
    g = torch.Generator().manual_seed(41)
    for rows, cols in ((4000, 96), (64, 9000)):
        x = (torch.randn(rows, cols, generator=g) * torch.logspace(-3, 3, rows)[:, None]).bfloat16()
        s = dict(x=x, residual=None, gamma=(1 + 0.2 * torch.randn(cols, generator=g)).bfloat16(), row_scale=None, col_scale=None)
        codes, scale, _ = row_run("rmsnorm", s, rows, cols, "bf16", "i8", 0, 1e-6, False)
        v, _, size = row_exact("rmsnorm", s, cols, 1e-6)
        c = codes.int().cpu()
        assert int(c.max()) <= 127 and int(c.min()) >= -127 and (c.abs().amax(1) == 127).all()
        close(c.double() * scale.double().cpu()[:, None], v, (CODE * v.abs().amax(1) / 127)[:, None] + 2.0 ** -17 * size, "y")
