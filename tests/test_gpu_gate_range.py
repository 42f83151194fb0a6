"""The gated SiLU product of gates whose exponential fp32 does not hold, against large up values.

Tolerances. A rounding to 16 bits is off by half a step at most, HALF relative, or half the smallest step.
|gate| log2(e) / 4 is off by two roundings (2 steps of 2^-24 of its size), which the fourth power of its
exponential turns into 2 |gate| steps: 500 at |gate| = 250, and under 12 for the exponential itself, its powers,
1 / (1 + e) and the products: 2^-15 = 512 steps. fp32's own smallest values are rounded by half of 2^-149 in each
of the products: 2^-147 in all."""
import pytest
import torch

from tests.test_gpu_layer_ops import HALF, TINY, close, row_exact, row_run

pytestmark = pytest.mark.gpu

REL = 2.0 ** -15


@pytest.mark.parametrize("x", ["16", "i32"])
@pytest.mark.parametrize("power", [0, 20, 40, 80, 120])
def test_gates_far_below_zero_meet_large_up_values(power, x):
    gate = -torch.arange(20.0, 212.0, 0.25)
    gate[::16] *= -0.25                                             # some gates above zero between them
    up = torch.where(torch.arange(gate.numel()) % 2 == 0, 1.0, -1.5) * 2.0 ** power
    s = dict(x=torch.stack((gate, up), 0), row_scale=None, col_scale=None)
    if x == "i32":                                                  # whole numbers times powers of two: exact
        s["x"] = torch.cat((gate * 16, torch.sign(up) * up.abs() / 2.0 ** power * 2), 0)[None].to(torch.int32)
        s["row_scale"] = torch.ones(1)
        s["col_scale"] = torch.cat((torch.full_like(gate, 2.0 ** -4), torch.full_like(up, 2.0 ** (power - 1))))
    else:
        s["x"] = torch.cat((gate, up), 0)[None].bfloat16()
    cols = gate.numel()
    v, _, _ = row_exact("swiglu", s, cols, 0.0)
    v = torch.where(v.abs() > torch.finfo(torch.bfloat16).max, v.sign() * float("inf"), v)
    assert torch.isfinite(v).all() or power == 120
    got, _, _ = row_run("swiglu", s, 1, cols, "bf16", None, 0, 0.0, False)
    fin = torch.isfinite(v)
    assert torch.equal(torch.isfinite(got.cpu()), fin)
    close(got.cpu()[fin], v[fin], (HALF["bf16"] + REL * 1.01) * v.abs()[fin] + TINY["bf16"] + 2.0 ** -147, "y")


@pytest.mark.parametrize("gate,power", [(-95, 20), (-100, 20), (-104, 40), (-120, 60), (-150, 100)])
def test_codes_of_gates_far_below_zero(gate, power):
    """A row that only such products fill: its scale and codes are theirs."""
    g = torch.full((1, 64), float(gate)).bfloat16()
    up = ((torch.arange(64) - 63).double() * 2.0 ** power).bfloat16()[None]   # no ties: k 127 / 63 is never half a whole number
    s = dict(x=torch.cat((g, up), 1), row_scale=None, col_scale=None)
    got, scale, _ = row_run("swiglu", s, 1, 64, "bf16", "i8", 0, 0.0, False)
    v, _, _ = row_exact("swiglu", s, 64, 0.0)
    assert torch.equal(got[0].double().cpu(), torch.round(v[0] / v.abs().max() * 127))
    assert float(scale[0]) == pytest.approx(float(v.abs().max()) / 127, rel=REL)
