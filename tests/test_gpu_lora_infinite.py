"""Adapters where a token's inner product A x is infinite, or past the 16-bit type's largest value: the row is what the
formula gives, infinities with their signs and NaN where infinities of both signs meet."""
import pytest
import torch

from tests.test_gpu_layer_ops import HALF
from tests.test_gpu_lora import inputs, plain, run

pytestmark = pytest.mark.gpu
INF = float("inf")


def formula(s, r, j):
    """Row j in 64 bits."""
    a, m = int(s["index"][j]), s["base"].shape[1]
    x = s["x"][j].double() * (1 if s["x_scale"] is None else s["x_scale"][j].double())
    base = s["base"][j].double()
    if s["row_scale"] is not None:
        base = base * s["row_scale"][j].double() * s["col_scale"].double()
    t = (s["a"][a * r:(a + 1) * r].double() * x).sum(1)
    return base + s["scale"][a].double() * (s["b"][a * m:(a + 1) * m].double() * t).sum(1)


def same(got, want, what):
    got = got.double().cpu()
    assert torch.equal(got.isnan(), want.isnan()), what
    some = want.isinf()
    assert some.any() and torch.equal(got[some], want[some]) and torch.equal(got.isinf(), some), what


def signs(s, r, a):
    """B of adapter a: rows of positive, of negative and of mixed values."""
    m = s["base"].shape[1]
    b = s["b"][a * m:(a + 1) * m]
    b.abs_().clamp_min_(0.01)
    b[1::3] *= -1
    b[2::3, ::2] *= -1


@pytest.mark.parametrize("base", ["16", "i32"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,r", [(5, 8), (5, 48), (70, 16), (70, 128)])
@pytest.mark.parametrize("k,at", [(128, 0), (128, 127), (136, 135), (131, 130), (131, 124), (131, 5), (4100, 4099), (4100, 4093)])
def test_an_infinite_x(k, at, n, r, dtype, base):
    s = inputs(n, k, 70, r, 3, dtype, base=base, seed=k + n)
    s["index"][2], s["index"][4] = 1, 1
    signs(s, r, 1)
    clean = run(s, r)
    s["a"][r:2 * r, at] = s["a"][r:2 * r, at].abs() + 0.01
    before = run(s, r)
    s["x"][2, at], s["x"][4, at] = INF, -INF
    y = run(s, r)
    for j in (2, 4):
        same(y[j], formula(s, r, j), j)
    rest = torch.tensor([j not in (2, 4) for j in range(n)], device="cuda")
    assert torch.equal(y[rest], before[rest]) and clean.isfinite().all()


@pytest.mark.parametrize("x", ["16", "i8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,r", [(5, 8), (70, 40)])
@pytest.mark.parametrize("k", [128, 131])
def test_an_infinite_sum_beside_large_ones(k, n, r, dtype, x):
    """One rank's sum is infinite; others are finite, one of them past f16's largest value and against it in sign."""
    s = inputs(n, k, 70, r, 3, dtype, x, seed=k + n)
    s["index"][3] = 2
    signs(s, r, 2)
    s["x"][3, :8] = 100
    s["a"][2 * r + 1, :8] = 1000                       # 8e5 and more, before an int8 token's scale
    s["a"][2 * r, k - 1] = -INF
    s["x"][3, k - 1] = 3
    y = run(s, r)
    want = formula(s, r, 3)
    assert not want.isnan().any()
    same(y[3], want, "one infinite sum")


@pytest.mark.parametrize("base", ["16", "i32"])
def test_a_sum_past_the_largest_of_the_type(base):
    """bf16: A x between the type's largest value and fp32's is no infinity. Terms are powers of two, so that the tolerance
    is that of one rounding and of the two parts."""
    k, m, r = 128, 40, 8
    s = inputs(2, k, m, r, 1, "bf16", base=base)
    s["index"][:] = 0
    s["x"][:], s["a"][:], s["b"][:] = 0, 0, 0
    s["x"][0, 3], s["x"][0, 90], s["x"][1, 3], s["x"][1, 90] = 2.0 ** 64, 2.0 ** 64, -2.0 ** 64, -2.0 ** 64
    s["a"][5, 3], s["a"][5, 90] = 2.0 ** 63 * 1.9921875, 2.0 ** 63 * 0.005859375          # together 1.998 * 2^127
    s["b"][:, 5], s["scale"][0] = 2.0 ** -60, 2.0 ** -60
    y = run(s, r)
    want = plain(s, r)[0]
    assert want.abs().max() > 250 and y.isfinite().all()
    assert ((y.double().cpu() - want).abs() <= (HALF["bf16"] + HALF["bf16"] ** 2 * 2 + 2.0 ** -20) * (want.abs() + 256)).all()
