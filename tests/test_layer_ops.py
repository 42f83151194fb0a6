"""Host side of the operators around the product (RMS norm, gated SiLU product,
4-bit product): plans, sizes and refusals, all before any device call."""
import ctypes

import pytest
import torch

import structured_sparse_gemm_nm_amd as nm

FAKE = 0x10000      # never dereferenced: the calls below fail before anything is enqueued
ODD = 0x10008


def rows(**kw):
    return nm.nm_rows_plan_init(**dict(dict(rows=8, cols=64, op="rmsnorm", dtype="f16"), **kw))


def w4(**kw):
    return nm.nm_w4_plan_init(**dict(dict(m=64, n=4, k=256, group=128, dtype="f16"), **kw))


def refused(call, status, text=""):
    with pytest.raises(nm.NmError) as e:
        call()
    assert e.value.status == status and text in str(e.value), str(e.value)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), nm.NM_ERR_SHAPE), (dict(cols=-1), nm.NM_ERR_SHAPE), (dict(rows=1 << 24), nm.NM_ERR_SHAPE),
    (dict(cols=(1 << 30) + 16, ldx=1 << 31, ldy=1 << 31, ldr=1 << 31, ldh=1 << 31), nm.NM_ERR_SHAPE),
    (dict(dtype="i8"), nm.NM_ERR_INVALID_ARG), (dict(x_dtype="bf16"), nm.NM_ERR_INVALID_ARG),
    (dict(x_dtype="i8"), nm.NM_ERR_INVALID_ARG), (dict(y_dtype="i32"), nm.NM_ERR_INVALID_ARG),
    (dict(eps=-1e-6), nm.NM_ERR_INVALID_ARG), (dict(eps=float("nan")), nm.NM_ERR_INVALID_ARG),
    (dict(eps=float("inf")), nm.NM_ERR_INVALID_ARG),
    (dict(ldx=32), nm.NM_ERR_SHAPE), (dict(ldy=32), nm.NM_ERR_SHAPE), (dict(ldr=32), nm.NM_ERR_SHAPE),
    (dict(ldh=32), nm.NM_ERR_SHAPE), (dict(ldx=68), nm.NM_ERR_ALIGN), (dict(y_dtype="i8", ldy=72), nm.NM_ERR_ALIGN),
    (dict(x_dtype="i32", ldx=66), nm.NM_ERR_ALIGN), (dict(ldh=66), nm.NM_ERR_ALIGN),
    (dict(op="swiglu", ldx=64), nm.NM_ERR_SHAPE),             # x holds both halves
])
def test_rows_plan_refuses(kw, status):
    refused(lambda: rows(**kw), status)


def test_rows_plan_accepts():
    rows(op="swiglu", ldr=1, ldh=1, eps=-1.0)                  # not read by this operator
    rows(cols=7, ldx=7, ldy=9, ldr=11, ldh=7)                  # short rows start anywhere
    rows(x_dtype="i32", ldx=68)
    rows(rows=0), rows(cols=0), rows(op="swiglu", cols=0)
    with pytest.raises(ValueError):
        rows(op="layernorm")
    with pytest.raises(ValueError):
        rows(dtype="f32")


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), nm.NM_ERR_SHAPE), (dict(n=-1), nm.NM_ERR_SHAPE), (dict(k=-1), nm.NM_ERR_SHAPE),
    (dict(m=(1 << 24) + 1), nm.NM_ERR_SHAPE), (dict(n=(1 << 20) + 1), nm.NM_ERR_SHAPE),
    (dict(k=(1 << 20) + 16), nm.NM_ERR_SHAPE),
    (dict(dtype="i8"), nm.NM_ERR_INVALID_ARG), (dict(x_dtype="bf16"), nm.NM_ERR_INVALID_ARG),
    (dict(x_dtype="i32"), nm.NM_ERR_INVALID_ARG),
    (dict(sparse=True, k=258, ldx=264), nm.NM_ERR_SHAPE),
    (dict(group=-32), nm.NM_ERR_SHAPE), (dict(group=16), nm.NM_ERR_SHAPE), (dict(group=100), nm.NM_ERR_SHAPE),
    (dict(group=32, x_dtype="i8"), nm.NM_ERR_SHAPE), (dict(group=32, sparse=True), nm.NM_ERR_SHAPE),
    (dict(group=64, sparse=True, x_dtype="i8"), nm.NM_ERR_SHAPE),
    (dict(ldx=128), nm.NM_ERR_SHAPE), (dict(ldy=32), nm.NM_ERR_SHAPE),
    (dict(ldx=260), nm.NM_ERR_ALIGN), (dict(x_dtype="i8", ldx=264), nm.NM_ERR_ALIGN), (dict(ldy=68), nm.NM_ERR_ALIGN),
])
def test_w4_plan_refuses(kw, status):
    refused(lambda: w4(**kw), status)


def test_w4_plan_refuses_flags_that_are_no_truth_values():
    p = nm.nm_w4_problem_t()
    p.m, p.n, p.k, p.ldx, p.ldy = 16, 1, 32, 32, 16
    h = ctypes.c_void_p()
    for name in ("sparse", "zeros"):
        setattr(p, name, 2)
        assert nm.lib().nm_w4_plan_init(ctypes.byref(h), ctypes.byref(p)) == nm.NM_ERR_INVALID_ARG
        assert h.value is None
        setattr(p, name, 0)
    assert nm.lib().nm_w4_plan_init(None, ctypes.byref(p)) == nm.NM_ERR_INVALID_ARG
    assert nm.lib().nm_w4_plan_init(ctypes.byref(h), None) == nm.NM_ERR_INVALID_ARG
    r = nm.nm_rows_problem_t()
    r.rows, r.cols, r.ldx, r.ldr, r.ldh, r.ldy = 1, 8, 8, 8, 8, 8
    r.op = 2
    assert nm.lib().nm_rows_plan_init(ctypes.byref(h), ctypes.byref(r)) == nm.NM_ERR_INVALID_ARG
    assert nm.lib().nm_rows_plan_init(None, ctypes.byref(r)) == nm.NM_ERR_INVALID_ARG
    assert nm.lib().nm_rows_plan_init(ctypes.byref(h), None) == nm.NM_ERR_INVALID_ARG


@pytest.mark.parametrize("m,k,group,sparse,zeros,x", [
    (64, 256, 128, False, False, None), (65, 257, 32, False, True, None), (1, 1, 0, False, True, "i8"),
    (100, 1032, 256, True, True, "i8"), (33, 4096, 64, True, False, None), (16, 96, 128, False, False, None),
    (16, 1000, 96, False, False, None),
])
def test_w4_sizes(m, k, group, sparse, zeros, x):
    p = w4(m=m, k=k, group=group, sparse=sparse, zeros=zeros, x_dtype=x, ldx=(k + 15) // 16 * 16, ldy=(m + 7) // 8 * 8)
    kept = k // 2 if sparse else k
    G = 1 if group == 0 else -(-k // group)
    assert (p.groups, p.code_ld) == (G, -(-kept // 2))
    assert p.meta_ld == ((-(-k // 8) + 15) // 16 * 16 if sparse else 0)
    blocks = -(-m // 16)
    codes = blocks * -(-kept // 128) * 1024                    # tiles of 16 rows x 128 kept values
    assert p.packed_bytes == codes + (codes // 2 if sparse else 0) + blocks * G * (48 if zeros else 32)
    assert w4(m=m, n=9, k=k, group=group, sparse=sparse, zeros=zeros, x_dtype=x, ldx=(k + 63) // 64 * 64,
              ldy=(m + 7) // 8 * 8 + 16).packed_bytes == p.packed_bytes


def test_calls_refuse_bad_arguments():
    L, bad, odd = nm.lib(), nm.NM_ERR_INVALID_ARG, nm.NM_ERR_ALIGN
    p, pi = rows(), rows(x_dtype="i32", y_dtype="i8")
    f, o = FAKE, ODD
    assert L.nm_rmsnorm(None, f, None, None, None, f, None, f, None, None) == bad
    assert L.nm_rmsnorm(p.handle, None, None, None, None, f, None, f, None, None) == bad      # no x
    assert L.nm_rmsnorm(p.handle, f, None, None, None, None, None, f, None, None) == bad      # no gamma
    assert L.nm_rmsnorm(p.handle, f, None, None, None, f, None, None, None, None) == bad      # no y
    assert L.nm_rmsnorm(p.handle, f, f, f, None, f, None, f, None, None) == bad               # scales of a 16-bit x
    assert L.nm_rmsnorm(p.handle, f, None, None, None, f, None, f, f, None) == bad            # scale of a 16-bit y
    assert L.nm_rmsnorm(pi.handle, f, f, None, None, f, None, f, f, None) == bad              # no column scales
    assert L.nm_rmsnorm(pi.handle, f, None, f, None, f, None, f, f, None) == bad              # no row scales
    assert L.nm_rmsnorm(pi.handle, f, f, f, None, f, None, f, None, None) == bad              # no y scales
    assert L.nm_swiglu(p.handle, f, None, None, f, None, None) == bad                         # a norm's plan
    assert "other row operator" in nm.nm_last_error()
    for i in (1, 4, 5, 6, 7):
        a = [p.handle, f, None, None, f, f, f, f, None, None]
        a[i] = o
        assert L.nm_rmsnorm(*a) == odd, i
    for i in (2, 3, 8):
        a = [pi.handle, f, f, f, None, f, None, f, f, None]
        a[i] = o
        assert L.nm_rmsnorm(*a) == odd, i
    s = rows(op="swiglu", x_dtype="i32", y_dtype="i8")
    assert L.nm_rmsnorm(s.handle, f, f, f, None, f, None, f, f, None) == bad
    assert L.nm_swiglu(s.handle, f, f, f, f, None, None) == bad
    for i in (1, 2, 3, 4, 5):
        a = [s.handle, f, f, f, f, f, None]
        a[i] = o
        assert L.nm_swiglu(*a) == odd, i
    w, wz = w4(), w4(x_dtype="i8", sparse=True, zeros=True, group=256)
    assert L.nm_w4_pack(None, f, f, None, None, f, None) == bad
    assert L.nm_w4_pack(w.handle, f, f, f, None, f, None) == bad                              # zeros of a plan without
    assert L.nm_w4_pack(w.handle, f, f, None, f, f, None) == bad                              # metadata of dense codes
    assert L.nm_w4_pack(wz.handle, f, f, None, f, f, None) == bad
    assert L.nm_w4_pack(wz.handle, f, f, f, None, f, None) == bad
    for i in (1, 2, 5):
        a = [wz.handle, f, f, f, f, f, None]
        a[i] = None
        assert L.nm_w4_pack(*a) == bad, i
    for i in range(1, 6):
        a = [wz.handle, f, f, f, f, f, None]
        a[i] = o
        assert L.nm_w4_pack(*a) == odd, i
    assert L.nm_w4_matvec(None, f, f, None, f, None) == bad
    assert L.nm_w4_matvec(w.handle, f, f, f, f, None) == bad                                  # scale of a 16-bit x
    assert L.nm_w4_matvec(wz.handle, f, f, None, f, None) == bad
    for i in (1, 2, 4):
        a = [w.handle, f, f, None, f, None]
        a[i] = None
        assert L.nm_w4_matvec(*a) == bad, i
    for i in range(1, 5):
        a = [wz.handle, f, f, f, f, None]
        a[i] = o
        assert L.nm_w4_matvec(*a) == odd, i
    assert L.nm_w4_sizes(None, None, None, None, None) == bad
    assert L.nm_w4_sizes(w.handle, None, None, None, None) == nm.NM_OK


def test_destroyed_plans_are_refused():
    p, w = rows(), w4()
    p.destroy(), w.destroy(), p.destroy(), w.destroy()
    refused(lambda: nm.nm_rmsnorm(p, FAKE, FAKE, FAKE, stream=0), nm.NM_ERR_INVALID_ARG, "plan is NULL")
    refused(lambda: nm.nm_w4_matvec(w, FAKE, FAKE, FAKE, stream=0), nm.NM_ERR_INVALID_ARG, "plan is NULL")


def test_empty_calls_enqueue_nothing():
    for kw in (dict(rows=0), dict(cols=0)):
        nm.nm_rmsnorm(rows(**kw), None, None, None, stream=0)
        nm.nm_rmsnorm(rows(x_dtype="i32", y_dtype="i8", **kw), None, None, None, stream=0)
        nm.nm_swiglu(rows(op="swiglu", **kw), None, None, stream=0)
    for kw in (dict(m=0), dict(n=0)):
        nm.nm_w4_matvec(w4(**kw), None, None, None, stream=0)
    for kw in (dict(m=0), dict(k=0)):
        nm.nm_w4_pack(w4(**kw), None, None, None, stream=0)


def test_host_tensors_are_refused():
    """A host tensor's address never reaches the library."""
    x, g = torch.zeros((8, 64), dtype=torch.float16), torch.zeros(64, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_rmsnorm(rows(), x, g, x.clone())
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_swiglu(rows(op="swiglu"), torch.zeros((8, 128), dtype=torch.float16), x)
    p = w4()
    packed = p.empty_packed(device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_w4_matvec(p, packed, torch.zeros((4, 256), dtype=torch.float16), torch.zeros((4, 64), dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_w4_pack(p, torch.zeros((64, 128), dtype=torch.uint8), torch.zeros((64, 2), dtype=torch.float16), packed)


@pytest.mark.parametrize("t,shape,ld", [
    (torch.zeros(4, 8), (4, 8), 8),                            # dtype
    (torch.zeros(4, 8, dtype=torch.float16), (4, 9), 8),       # shape
    (torch.zeros(8, dtype=torch.float16), (4, 8), 8),
    (torch.zeros(4, 8, dtype=torch.float16), (4, 8), 16),      # row stride
    (torch.zeros(4, 16, dtype=torch.float16)[:, ::2], (4, 8), 16),
    (torch.zeros(8, 4, dtype=torch.float16).t(), (4, 8), 8),
    (torch.zeros(16, dtype=torch.float16)[::2], (8,), None),
])
def test_operands_are_checked_against_the_plan(t, shape, ld):
    with pytest.raises(ValueError, match="operand"):
        nm._address(t, "operand", torch.float16, shape, ld, -1)


def test_operands_that_fit_the_plan_pass():
    f16 = torch.float16
    for t, shape, ld in ((torch.zeros(4, 8, dtype=f16), (4, 8), 8),
                         (torch.zeros(4, 16, dtype=f16)[:, :8], (4, 8), 16),
                         (torch.zeros(1, 8, dtype=f16), (1, 8), 24),        # one row: its stride says nothing
                         (torch.zeros(8, dtype=f16), (8,), None)):
        assert nm._address(t, "operand", f16, shape, ld, -1) == t.data_ptr()
    assert nm._address(None, "operand", f16, (4, 8), 8, 0) is None
    assert nm._address(FAKE, "operand", f16, (4, 8), 8, 0) == FAKE
