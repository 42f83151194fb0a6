"""The 4-bit product where blocks take several row tiles, against the same 64-bit
computation and with the same tolerances as tests/test_gpu_layer_ops.py."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from tests.test_gpu_layer_ops import (Out, TORCH, close, groups, strided, w4_check, w4_exact, w4_inputs, w4_pack,
                                      w4_plan, w4_run, w4_tolerance)

pytestmark = pytest.mark.gpu


# row tiles: 257 and 511 (two a block), 513 and 768 (three), 1000 (four), 1376 (three, in rounds), 2001
@pytest.mark.parametrize("m", [4097, 8170, 8209, 12288, 16000, 22016, 32003])
@pytest.mark.parametrize("x,sparse", [("16", False), ("16", True), ("i8", False), ("i8", True)])
def test_row_counts(m, x, sparse):
    dtype = ("f16", "bf16")[m % 2]
    w4_check(m, 1, 1024, 256, dtype, x, sparse, False)
    w4_check(m, 5, 772, 0, dtype, x, sparse, True, pad=16)


@pytest.mark.parametrize("n", [2, 7, 16, 17, 31, 33, 48, 50])
@pytest.mark.parametrize("x,sparse", [("16", False), ("16", True), ("i8", True)])
def test_token_counts(n, x, sparse):
    w4_check(16500, n, 1284, 256, "f16", x, sparse, n % 2 == 0)
    w4_check(5000, n, 516, groups(x, sparse)[1], "bf16", x, sparse, n % 2 == 1)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("k", [4, 252, 256, 516, 2048, 4100])
def test_many_sparse_rows(dtype, zeros, k):
    for i, (group, n) in enumerate(((0, 1), (64, 3), (128, 16), (192, 8), (256, 2), (512, 1))):
        w4_check((16400, 17003, 24576)[i % 3], n, k, group, dtype, "16", True, zeros, pad=16 * (i % 2), seed=i)


def test_k_in_more_pieces_than_scales_at_a_time():
    """Rows of 33 tiles and more: a wave fetches its scales several times."""
    w4_check(16400, 1, 16388, 64, "f16", "16", True, True)
    w4_check(16400, 2, 9000, 128, "bf16", "16", True, False)


def test_many_rows_keep_tokens_apart():
    """A token with a NaN leaves the other tokens' results bit for bit; so does what lies past k."""
    s = w4_inputs(17000, 6, 516, 128, "f16", "16", True, True, 2)
    a = w4_run(s, 17000, 6, 516, 128, "f16", "16")
    s["x"][5, 515] = float("nan")
    b = w4_run(s, 17000, 6, 516, 128, "f16", "16")
    assert torch.equal(a[:5], b[:5])
    meets = (s["pairs"][:, 128].long() == 3).any(1)                # rows whose kept weights meet column 515
    assert torch.equal(torch.isnan(b[5]).cpu(), meets)


def test_many_rows_repeat_bit_for_bit():
    s = w4_inputs(22016, 4, 1028, 128, "bf16", "16", True, False, 3)
    plan = w4_plan(s, 22016, 4, 1028, 128, "bf16", "16")
    packed, x = w4_pack(plan, s), strided(s["x"], plan._strides[0], 0)[0]
    outs = [Out(4, 22016, plan._strides[1], TORCH["bf16"]) for _ in range(4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        with torch.cuda.stream(side if i % 2 else torch.cuda.current_stream()):
            nm.nm_w4_matvec(plan, packed, x, o.t)
    torch.cuda.synchronize()
    for o in outs:
        o.check()
        assert torch.equal(o.t, outs[0].t)


@pytest.mark.parametrize("m", [64, 17000])
@pytest.mark.parametrize("x", ["16", "i8"])
def test_infinite_scales_stay_in_their_rows(m, x):
    """k ends inside the last tile: what lies past it meets no scale."""
    group = 128 if x == "16" else 256
    s = w4_inputs(m, 2, 1284, group, "f16", x, True, False, 4)
    s["x"] = s["x"].abs().clamp_min(1)
    s["q"][3] = 9                                                  # all positive: the sum is +inf, never a NaN
    want = w4_run(s, m, 2, 1284, group, "f16", x)
    s["scales"][3, -1] = float("inf")
    got = w4_run(s, m, 2, 1284, group, "f16", x)
    assert (got[:, 3] == float("inf")).all()
    rows = torch.arange(m) != 3
    assert torch.equal(got[:, rows], want[:, rows])


def test_strides_of_an_odd_number_of_rows():
    """y's rows on every alignment a plan allows: stores of four rows need whole 8 bytes."""
    for m, ldy in ((5, 5), (7, 9), (6, 7), (17, 24), (16403, 16408)):
        s = w4_inputs(m, 3, 260, 0, "f16", "16", True, False, 5)
        plan = nm.nm_w4_plan_init(m, 3, 260, group=0, sparse=True, ldx=272, ldy=ldy)
        out = Out(3, m, ldy, torch.float16)
        nm.nm_w4_matvec(plan, w4_pack(plan, s), strided(s["x"], 272, float("nan"))[0], out.t)
        torch.cuda.synchronize()
        out.check()
        y, size = w4_exact(s, 260, 0)
        close(out.t, y, w4_tolerance(y, size, 260, "f16"), "y")




def test_no_columns_and_many_rows():
    """k = 0 has nothing to load, and sums of nothing."""
    plan = nm.nm_w4_plan_init(17000, 2, 0, group=0, sparse=True, ldx=16)
    y = torch.full((2, 17000), 7.0, dtype=torch.float16, device="cuda")
    nm.nm_w4_matvec(plan, plan.empty_packed(), torch.zeros((2, 0), dtype=torch.float16, device="cuda"), y)
    torch.cuda.synchronize()
    assert (y == 0).all()


def test_more_than_64_kilobytes_of_lds():
    """Sixteen tokens that eight waves turn for three row tiles."""
    w4_check(16400, 8, 3840, 128, "bf16", "16", True, True)
    w4_check(12288, 16, 2560, 128, "f16", "16", True, False)
