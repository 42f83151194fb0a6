"""Host side of the head norms with rotation: plans, sizes and refusals, all before any device call."""
import ctypes
import math

import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from structured_sparse_gemm_nm_amd.heads import rotation_table
from tests.test_layer_ops import FAKE, ODD, refused


def heads(**kw):
    return nm.nm_heads_plan_init(**dict(dict(rows=8, heads_q=4, heads_k=2, heads_v=2, head_dim=64, rotary_dim=64, table_rows=16), **kw))


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), nm.NM_ERR_SHAPE), (dict(rows=1 << 24), nm.NM_ERR_SHAPE), (dict(heads_q=0), nm.NM_ERR_SHAPE),
    (dict(heads_k=-1), nm.NM_ERR_SHAPE), (dict(heads_v=-1), nm.NM_ERR_SHAPE), (dict(heads_q=65537), nm.NM_ERR_SHAPE),
    (dict(head_dim=0), nm.NM_ERR_SHAPE), (dict(head_dim=60), nm.NM_ERR_SHAPE), (dict(head_dim=520), nm.NM_ERR_SHAPE),
    (dict(rotary_dim=-8), nm.NM_ERR_SHAPE), (dict(rotary_dim=72), nm.NM_ERR_SHAPE), (dict(rotary_dim=20), nm.NM_ERR_SHAPE),
    (dict(table_rows=0), nm.NM_ERR_SHAPE), (dict(table_rows=-1, rotary_dim=0), nm.NM_ERR_SHAPE),
    (dict(table_rows=(1 << 31) + 1), nm.NM_ERR_SHAPE),
    (dict(dtype="i8"), nm.NM_ERR_INVALID_ARG), (dict(x_dtype="bf16"), nm.NM_ERR_INVALID_ARG),
    (dict(x_dtype="i8"), nm.NM_ERR_INVALID_ARG), (dict(eps=-1e-6), nm.NM_ERR_INVALID_ARG),
    (dict(eps=math.nan), nm.NM_ERR_INVALID_ARG), (dict(eps=math.inf), nm.NM_ERR_INVALID_ARG),
    (dict(ldx=256), nm.NM_ERR_SHAPE), (dict(ldy=511), nm.NM_ERR_SHAPE), (dict(ldx=516), nm.NM_ERR_ALIGN),
    (dict(ldy=516), nm.NM_ERR_ALIGN), (dict(x_dtype="i32", ldx=514), nm.NM_ERR_ALIGN), (dict(ldx=(1 << 46) + 8), nm.NM_ERR_SHAPE),
])
def test_plan_refuses(kw, status):
    refused(lambda: heads(**kw), status)


def test_plan_accepts():
    heads(rotary_dim=0, table_rows=0), heads(heads_k=0, heads_v=0), heads(rows=0), heads(x_dtype="i32", ldx=516)
    heads(head_dim=512, rotary_dim=8, pairs="neighbours", dtype="bf16", ldy=4104)
    with pytest.raises(ValueError):
        heads(pairs="quarters")
    with pytest.raises(ValueError):
        heads(dtype="f64")
    p = nm.nm_heads_problem_t()
    p.rows, p.heads_q, p.head_dim, p.ldx, p.ldy, p.pairs = 1, 1, 8, 8, 8, 2
    h = ctypes.c_void_p()
    assert nm.lib().nm_heads_plan_init(ctypes.byref(h), ctypes.byref(p)) == nm.NM_ERR_INVALID_ARG and h.value is None
    p.pairs, p.type_io, p.type_x, p.zero_rows = 0, nm.NM_F16, nm.NM_F16, 2
    assert nm.lib().nm_heads_plan_init(ctypes.byref(h), ctypes.byref(p)) == nm.NM_ERR_INVALID_ARG and h.value is None
    assert nm.lib().nm_heads_plan_init(None, ctypes.byref(p)) == nm.NM_ERR_INVALID_ARG
    assert nm.lib().nm_heads_plan_init(ctypes.byref(h), None) == nm.NM_ERR_INVALID_ARG


def test_workspace():
    assert heads().workspace_bytes == 8 * 2 * 64 * 4 and 0 < heads(rows=1 << 20).workspace_bytes <= 1024 * 2 * 64 * 4
    assert heads(x_dtype="i32").workspace_bytes == 0
    assert nm.lib().nm_heads_workspace_size(None, None) == nm.NM_ERR_INVALID_ARG


def test_calls_refuse_bad_arguments():
    L, bad, odd = nm.lib(), nm.NM_ERR_INVALID_ARG, nm.NM_ERR_ALIGN
    p, a, none, k0 = heads(), heads(x_dtype="i32"), heads(rotary_dim=0, table_rows=0), heads(heads_k=0)
    f, o, four = FAKE, ODD, FAKE + 4
    fwd, back = L.nm_head_norm_rope, L.nm_head_norm_rope_backward
    # x, row_scale, col_scale, gamma_q, gamma_k, positions, table, y, stream
    good = [f, None, None, f, f, f, f, f, None]

    def forward(plan, **at):
        args = list(good)
        for i, v in at.items():
            args[int(i[1:])] = v
        return fwd(plan.handle if plan else None, *args)

    assert forward(None) == bad
    for i in (0, 3, 4, 5, 6, 7):
        assert forward(p, **{"a%d" % i: None}) == bad
        assert forward(p, **{"a%d" % i: four}) == odd
    assert forward(p, a1=f) == bad and forward(p, a1=f, a2=f) == bad and forward(a) == bad and forward(a, a1=f) == bad
    assert forward(a, a2=f) == bad and forward(a, a1=f, a2=o) == odd and forward(a, a1=f + 2, a2=f) == odd
    assert forward(p, a7=o) == odd and forward(p, a0=o) == odd and forward(p, a6=o) == odd
    # x, gamma_q, gamma_k, positions, table, grad_y, grad_x, dgamma_q, dgamma_k, workspace, stream
    gback = [f, f, f, f, f, f, f, f, f, f, None]

    def backward(plan, **at):
        args = list(gback)
        for i, v in at.items():
            args[int(i[1:])] = v
        return back(plan.handle if plan else None, *args)

    assert backward(None) == bad
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9):
        assert backward(p, **{"a%d" % i: None}) == bad
    assert backward(p, a7=None) == bad and backward(k0) == bad and backward(a) == nm.NM_ERR_UNSUPPORTED
    for i in (0, 1, 2, 4, 5, 6, 7, 8, 9):
        assert backward(p, **{"a%d" % i: o}) == odd
    assert backward(p, a3=four) == odd
    # nothing to do: no pointer is asked for
    z = heads(rows=0)
    assert fwd(z.handle, *[None] * 9) == nm.NM_OK and back(z.handle, *[None] * 11) == nm.NM_OK
    assert forward(none, a6=None, a7=None) == bad      # a missing table is none; y is missing


def test_host_tensors_are_refused():
    p = heads()
    x, g, at, table = torch.zeros((8, 512)).half(), torch.ones(64).half(), torch.zeros(8, dtype=torch.int64), torch.zeros((16, 64))
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_head_norm_rope(p, x, g, g, at, table, x)
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_head_norm_rope_backward(p, x, g, g, at, table, x, x)
    p.destroy()
    assert not (p._norm_call or p._back_call)


def test_rotation_table():
    t = rotation_table(70000, 16, base=500.0, device="cpu")
    assert t.shape == (70000, 16) and t.dtype is torch.float32
    for p in (0, 1, 65537, 69999):
        for i in range(8):
            a = p * 500.0 ** (-2 * i / 16)
            assert abs(t[p, i] - math.cos(a)) < 1e-7 and abs(t[p, 8 + i] - math.sin(a)) < 1e-7
    assert rotation_table(4, 0, device="cpu").shape == (4, 0)
    with pytest.raises(ValueError):
        rotation_table(4, 12, device="cpu")
