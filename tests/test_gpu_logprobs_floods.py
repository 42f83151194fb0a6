"""Alternatives of rows most of whose logits are one value, wherever in the row it begins: the lowest columns, against a
stable sort, in a time near that of a row where it begins at the start."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm

pytestmark = pytest.mark.gpu


def rows_of(kind, rows, cols, low, value, dtype):
    x = torch.full((rows, (cols + 7) // 8 * 8), low, dtype=dtype, device="cuda")[:, :cols]
    at = torch.arange(cols, device="cuda")
    if kind == "early":
        x[:] = value
    elif kind == "late":
        x[:, cols * 3 // 4 + 5:] = value
    elif kind == "last":
        x[:, cols - 40:] = value
    elif kind == "spread":
        x[:, at % 997 == 996] = value                  # one or two in a hundred places of every thread's
    elif kind == "ends of slices":
        x[:, at % 4096 >= 4090] = value
    x[:, cols // 2] = value + 1                        # one is larger
    return x


def run(plan, x, work=None):
    lp, index = torch.empty((x.shape[0], plan.top), device="cuda"), torch.empty((x.shape[0], plan.top), dtype=torch.int64, device="cuda")
    nm.nm_logprobs(plan, x, top_logprob=lp, top_index=index, workspace=work if work is not None else plan.empty_workspace())
    return lp, index


@pytest.mark.parametrize("kind", ["early", "late", "last", "spread", "ends of slices"])
@pytest.mark.parametrize("dtype,low", [("f16", -65504.0), ("f32", -float("inf"))])
@pytest.mark.parametrize("rows,cols", [(1, 520), (1, 32003), (3, 131072), (2, 1 << 20), (1, 1 << 22), (1030, 2049), (1025, 8199)])
@pytest.mark.parametrize("top", [1, 5, 32])
def test_the_lowest_columns(rows, cols, kind, dtype, low, top):
    x = rows_of(kind, rows, cols, low, -1.5, {"f16": torch.float16, "f32": torch.float32}[dtype])
    plan = nm.nm_logprobs_plan_init(rows, cols, dtype=dtype, top=top, ldx=x.stride(0))
    lp, index = run(plan, x)
    one = x[0].float().cpu()
    want = torch.sort(one, descending=True, stable=True)[1][:top]
    assert torch.equal(index.cpu(), want.expand(rows, top))
    exact = torch.log_softmax(one.double(), 0)[want]
    # a logit's distance from the largest, fp32: half a step of it, twice; and the log of a sum of up to 2^22 terms
    fine = exact.isinf() | ((lp.cpu().double() - exact).abs() < 1e-4 + 2.0 ** -23 * exact.abs())
    assert fine.all() and torch.equal(lp.cpu().isinf(), exact.isinf().expand(rows, top))


def test_ties_that_begin_late_take_no_scan_of_the_row():
    rows, cols = 4, 1 << 21
    plan = nm.nm_logprobs_plan_init(rows, cols, dtype="f16", top=20)
    work, times = plan.empty_workspace(), {}
    for kind in ("early", "late"):
        x = rows_of(kind, rows, cols, -65504.0, -1.5, torch.float16)
        run(plan, x, work)
        best = 1e9
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            run(plan, x, work)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times[kind] = best
    assert times["late"] < 12 * times["early"], times      # 2.6 times; a scan by one wave took 110
