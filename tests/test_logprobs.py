"""Host side of the log probabilities: plans, sizes and refusals, all before any device call."""
import ctypes
import math

import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from tests.test_layer_ops import FAKE, ODD, refused


def plan(**kw):
    return nm.nm_logprobs_plan_init(**dict(dict(rows=4000, cols=64), **kw))


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), nm.NM_ERR_SHAPE), (dict(rows=1 << 24), nm.NM_ERR_SHAPE), (dict(cols=0), nm.NM_ERR_SHAPE),
    (dict(cols=(1 << 22) + 8), nm.NM_ERR_SHAPE), (dict(top=-1), nm.NM_ERR_SHAPE), (dict(top=33), nm.NM_ERR_SHAPE),
    (dict(cols=16, top=17), nm.NM_ERR_SHAPE), (dict(scale=0.0), nm.NM_ERR_INVALID_ARG), (dict(scale=-1.0), nm.NM_ERR_INVALID_ARG),
    (dict(scale=math.nan), nm.NM_ERR_INVALID_ARG), (dict(scale=math.inf), nm.NM_ERR_INVALID_ARG),
    (dict(scale=2.0 ** 127 * 1.01), nm.NM_ERR_INVALID_ARG),
    (dict(ldx=63), nm.NM_ERR_SHAPE), (dict(ldg=63), nm.NM_ERR_SHAPE), (dict(ldx=68), nm.NM_ERR_ALIGN),
    (dict(ldg=68), nm.NM_ERR_ALIGN), (dict(dtype="f32", ldx=66), nm.NM_ERR_ALIGN), (dict(cols=1003), nm.NM_ERR_ALIGN),
    (dict(ldx=1 << 47), nm.NM_ERR_SHAPE),
])
def test_plan_refuses(kw, status):
    refused(lambda: plan(**kw), status)


def test_plan_accepts():
    plan(scale=2.0 ** 127), plan(scale=2.0 ** -140), plan(cols=1), plan(cols=7, top=7), plan(rows=0), plan(dtype="f32", ldx=68), plan(dtype="i32", ldg=1), plan(cols=1 << 22, top=32)
    with pytest.raises(ValueError):
        plan(dtype="i8")
    p = nm.nm_logprobs_problem_t()
    p.rows, p.cols, p.ldx, p.ldg, p.scale, p.type_x = 1, 8, 8, 8, 1.0, nm.NM_I8
    h = ctypes.c_void_p()
    assert nm.lib().nm_logprobs_plan_init(ctypes.byref(h), ctypes.byref(p)) == nm.NM_ERR_INVALID_ARG and h.value is None
    assert nm.lib().nm_logprobs_plan_init(None, ctypes.byref(p)) == nm.NM_ERR_INVALID_ARG
    assert nm.lib().nm_logprobs_plan_init(ctypes.byref(h), None) == nm.NM_ERR_INVALID_ARG


def test_fp32_is_for_logits_only():
    for make, p in ((nm.lib().nm_rows_plan_init, nm.nm_rows_problem_t()), (nm.lib().nm_w4_plan_init, nm.nm_w4_problem_t()),
                    (nm.lib().nm_plan_init, nm.nm_problem_t()), (nm.lib().nm_heads_plan_init, nm.nm_heads_problem_t())):
        for name in ("type_io", "type_x", "type_y", "type_ab", "type_cd"):
            if hasattr(p, name):
                setattr(p, name, nm.NM_F32)
        if hasattr(p, "nm_n"):
            p.nm_n, p.nm_m, p.lda, p.ldb, p.ldc, p.ldd = 2, 4, 1, 1, 1, 1
        h = ctypes.c_void_p()
        assert make(ctypes.byref(h), ctypes.byref(p)) == nm.NM_ERR_INVALID_ARG


def test_workspace():
    assert plan().workspace_bytes == 0 and plan(top=5).workspace_bytes == 0
    for kw in (dict(rows=1, cols=1 << 20), dict(rows=16, cols=1 << 20, dtype="f32"), dict(rows=1, cols=1 << 22), dict(rows=5000, cols=1 << 22)):
        a, b = plan(**kw).workspace_bytes, plan(top=9, **kw).workspace_bytes
        assert a % (16 * kw["rows"]) == 0 and 1 < a // (16 * kw["rows"]) <= 64 and b > a and (b - a) // (4 * kw["rows"]) <= 2048
    assert nm.lib().nm_logprobs_workspace_size(None, None) == nm.NM_ERR_INVALID_ARG


def test_calls_refuse_bad_arguments():
    L, bad, odd = nm.lib(), nm.NM_ERR_INVALID_ARG, nm.NM_ERR_ALIGN
    p, a, t, long, none = plan(), plan(dtype="i32"), plan(top=3), plan(rows=1, cols=1 << 22), plan(rows=0)
    f, o = FAKE, ODD
    # x, row_scale, col_scale, tokens, logprob, entropy, stats, top_logprob, top_index, workspace, stream
    good = [f, None, None, f, f, f, f, None, None, None, None]

    def forward(plan, **at):
        args = list(good)
        for i, v in at.items():
            args[int(i[1:])] = v
        return L.nm_logprobs(plan.handle if plan else None, *args)

    assert forward(None) == bad and forward(p, a0=None) == bad and forward(p, a3=None) == bad and forward(p, a4=None) == bad
    assert forward(p, a1=f) == bad and forward(p, a2=f) == bad and forward(a) == bad and forward(a, a1=f) == bad and forward(a, a2=f) == bad
    assert forward(p, a7=f) == bad and forward(p, a8=f) == bad and forward(p, a7=f, a8=f) == bad
    assert forward(t) == bad and forward(t, a7=f) == bad and forward(t, a8=f) == bad
    assert forward(long) == bad                                # no workspace
    for i in (0, 2, 9):
        assert forward(p, **{"a%d" % i: o}) == odd
    for i in (3, 8):
        assert forward(p, **{"a%d" % i: f + 4}) == odd
    for i in (1, 4, 5, 6, 7):
        assert forward(p, **{"a%d" % i: f + 2}) == odd
    assert L.nm_logprobs(none.handle, *[None] * 11) == nm.NM_OK
    # x, tokens, stats, entropy, g_logprob, g_entropy, grad_x, stream
    gback = [f, f, f, f, f, f, f, None]

    def backward(plan, **at):
        args = list(gback)
        for i, v in at.items():
            args[int(i[1:])] = v
        return L.nm_logprobs_backward(plan.handle if plan else None, *args)

    assert backward(None) == bad and backward(a) == nm.NM_ERR_UNSUPPORTED
    for i in (0, 1, 2, 3, 6):
        assert backward(p, **{"a%d" % i: None}) == bad
    assert backward(p, a4=None, a5=None) == bad
    assert backward(p, a0=o) == odd and backward(p, a6=o) == odd and backward(p, a1=f + 4) == odd
    for i in (2, 3, 4, 5):
        assert backward(p, **{"a%d" % i: f + 2}) == odd
    assert L.nm_logprobs_backward(none.handle, *[None] * 8) == nm.NM_OK


def test_host_tensors_are_refused():
    p = plan()
    x, at, row = torch.zeros((4000, 64)).half(), torch.zeros(4000, dtype=torch.int64), torch.zeros(4000)
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_logprobs(p, x, at, row)
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_logprobs_backward(p, x, at, torch.zeros((4000, 2)), x, g_logprob=row)
