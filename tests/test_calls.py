"""The call extension of the operators around the product: what it takes by itself, and what it leaves to the checks in Python."""
import ctypes

import pytest
import torch

import structured_sparse_gemm_nm_amd as nm

F16, F32 = torch.float16, torch.float32
M = (F16, (4, 8), 8)
V = (F32, (4,), None)


def make(specs=(M, V, M, V), main=0, fn=0x1000, plan=0x1000):
    nm.lib()
    return nm._calls.Call(fn, plan, main, specs)


@pytest.mark.parametrize("kw,error", [
    (dict(specs=(M, V, M)), ValueError), (dict(specs=(M,) * 9), ValueError), (dict(main=4), ValueError),
    (dict(main=-1), ValueError), (dict(fn=0), ValueError), (dict(plan=0), ValueError),
    (dict(specs=((F16, (4,), 8), V, M, V)), ValueError), (dict(specs=((F16, (4, 8), None), V, M, V)), ValueError),
    (dict(specs=((F16, (4, 8), -8), V, M, V)), ValueError), (dict(specs=(("f16", (4, 8), 8), V, M, V)), TypeError),
    (dict(specs=((F16, ("4", 8), 8), V, M, V)), TypeError), (dict(specs=((F16, 4, 8), V, M, V)), TypeError),
    (dict(fn="x"), TypeError),
])
def test_descriptions_are_checked(kw, error):
    with pytest.raises(error):
        make(**kw)


def test_what_is_no_gpu_tensor_is_left_to_python():
    call, x, v = make(), torch.zeros((4, 8), dtype=F16), torch.zeros(4)
    assert call(x, v, x, v, 0) == -1
    assert call(None, v, x, v, 0) == -1
    assert call(0x1000, v, x, v, 0) == -1
    assert call("x", v, x, v, None) == -1


@pytest.mark.parametrize("args", [(), (None,) * 4, (None,) * 6])
def test_every_operand_and_the_stream_are_given(args):
    with pytest.raises(TypeError):
        make()(*args)
    with pytest.raises(TypeError):
        make()(None, None, None, None, stream=0)


def test_plans_hold_the_call_of_their_operator_until_they_are_destroyed():
    norm, gate, product = nm.nm_rows_plan_init(8, 64), nm.nm_rows_plan_init(8, 64, op="swiglu"), nm.nm_w4_plan_init(64, 4, 256)
    assert norm._norm_call and not norm._gate_call and gate._gate_call and not gate._norm_call and product._product_call
    for p in (norm, gate, product):
        p.destroy()
        assert not (p._norm_call or p._gate_call or p._product_call)


def test_a_plan_of_the_other_operator_is_refused():
    with pytest.raises(nm.NmError, match="other row operator"):
        nm.nm_swiglu(nm.nm_rows_plan_init(8, 64), 0x10000, 0x10000, stream=0)


@pytest.mark.gpu
def test_the_checks_are_those_of_python_on_the_gpu():
    """A recording entry point: the addresses that arrive are the operands', and every unfit operand is left to Python."""
    seen = []
    entry = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * 6)(lambda *a: seen.append(a) or 7)
    call = make(fn=ctypes.cast(entry, ctypes.c_void_p).value, plan=0x1234, main=2)
    x, y, v = torch.zeros((4, 8), dtype=F16, device="cuda"), torch.zeros((4, 8), dtype=F16, device="cuda"), torch.zeros(4, device="cuda")
    assert call(x, v, y, None, 99) == 7
    assert seen[-1] == (0x1234, x.data_ptr(), v.data_ptr(), y.data_ptr(), None, 99)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert call(torch.nn.Parameter(x), v, y, v, None) == 7
    assert seen[-1][-1] == side.cuda_stream
    n = len(seen)
    wide = torch.zeros((4, 16), dtype=F16, device="cuda")
    for bad in (x.cpu(), x.bfloat16(), x[:3], x.t(), x[:, :4], wide[:, :8], wide[:, ::2], x[0], x[None], v):
        assert call(bad, v, y, v, 0) == -1 and call(x, v, bad, v, 0) == -1
    for bad in (v.cpu(), v.half(), v[:3], v[None], torch.zeros(8, device="cuda")[::2], x):
        assert call(x, bad, y, v, 0) == -1
    assert call(x, v, y, v, side) == -1            # a stream object: Python reads its handle
    assert len(seen) == n
    one = make(specs=((F16, (1, 8), 24), V, M, V), fn=ctypes.cast(entry, ctypes.c_void_p).value)
    assert one(x[:1], v, y, v, 0) == 7             # one row: its stride says nothing
