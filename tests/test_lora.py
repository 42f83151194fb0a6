"""Host side of the low-rank adapters: plans, sizes and refusals, all before any device call."""
import ctypes

import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from tests.test_layer_ops import FAKE, ODD, refused


def plan(**kw):
    return nm.nm_lora_plan_init(**dict(dict(m=64, n=4, k=128, rank=16, adapters=3), **kw))


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), nm.NM_ERR_SHAPE), (dict(n=-1), nm.NM_ERR_SHAPE), (dict(k=15, ldx=16, lda=16), nm.NM_ERR_SHAPE), (dict(m=7), nm.NM_ERR_SHAPE), (dict(m=(1 << 24) + 8), nm.NM_ERR_SHAPE),
    (dict(n=(1 << 20) + 1), nm.NM_ERR_SHAPE), (dict(k=(1 << 20) + 16), nm.NM_ERR_SHAPE), (dict(rank=0), nm.NM_ERR_SHAPE),
    (dict(rank=12), nm.NM_ERR_SHAPE), (dict(rank=136), nm.NM_ERR_SHAPE), (dict(adapters=0), nm.NM_ERR_SHAPE),
    (dict(adapters=(1 << 20) + 1), nm.NM_ERR_SHAPE), (dict(dtype="i8"), nm.NM_ERR_INVALID_ARG), (dict(dtype="i32"), nm.NM_ERR_INVALID_ARG),
    (dict(x_dtype="bf16"), nm.NM_ERR_INVALID_ARG), (dict(x_dtype="i32"), nm.NM_ERR_INVALID_ARG),
    (dict(base_dtype="i8"), nm.NM_ERR_INVALID_ARG), (dict(base_dtype="bf16"), nm.NM_ERR_INVALID_ARG),
    (dict(ldx=64), nm.NM_ERR_SHAPE), (dict(lda=64), nm.NM_ERR_SHAPE), (dict(ldc=32), nm.NM_ERR_SHAPE), (dict(ldy=32), nm.NM_ERR_SHAPE),
    (dict(ldx=132), nm.NM_ERR_ALIGN), (dict(lda=132), nm.NM_ERR_ALIGN), (dict(ldy=68), nm.NM_ERR_ALIGN), (dict(ldc=68), nm.NM_ERR_ALIGN),
    (dict(x_dtype="i8", ldx=136), nm.NM_ERR_ALIGN), (dict(base_dtype="i32", ldc=66), nm.NM_ERR_ALIGN), (dict(lda=1 << 46), nm.NM_ERR_SHAPE),
])
def test_plan_refuses(kw, status):
    refused(lambda: plan(**kw), status)


def test_plan_accepts():
    plan(n=0), plan(k=16, m=8), plan(k=17, m=9, ldx=24, lda=24, ldc=16, ldy=16), plan(rank=128, dtype="bf16", x_dtype="i8", base_dtype="i32", ldc=68)
    with pytest.raises(ValueError):
        plan(dtype="f32")
    h = ctypes.c_void_p()
    assert nm.lib().nm_lora_plan_init(None, None) == nm.NM_ERR_INVALID_ARG
    assert nm.lib().nm_lora_plan_init(ctypes.byref(h), None) == nm.NM_ERR_INVALID_ARG


@pytest.mark.parametrize("n,k,r", [(1, 16, 8), (1, 4096, 16), (64, 11008, 64), (4096, 4096, 16), (1 << 20, 128, 128), (100, 1 << 20, 24)])
def test_workspace(n, k, r):
    b = plan(n=n, k=k, rank=r, ldx=(k + 7) // 8 * 8, lda=(k + 7) // 8 * 8).workspace_bytes
    assert b % (n * r * 4) == 0 and 1 <= b // (n * r * 4) <= (32 if n <= 8 else 16)
    assert plan(n=0).workspace_bytes == 0
    if n >= 4096:                         # tokens over 4 adapters and more are sorted by them: 8 bytes each
        more = plan(n=n, k=k, rank=r, ldx=(k + 7) // 8 * 8, lda=(k + 7) // 8 * 8, adapters=4).workspace_bytes
        assert more == b + 8 * n
    assert nm.lib().nm_lora_workspace_size(None, None) == nm.NM_ERR_INVALID_ARG


def test_calls_refuse_bad_arguments():
    L, bad, odd = nm.lib(), nm.NM_ERR_INVALID_ARG, nm.NM_ERR_ALIGN
    p, c, i = plan(), plan(x_dtype="i8"), plan(base_dtype="i32")
    f, o = FAKE, ODD
    # x, x_scale, A, B, scale, index, base, row_scale, col_scale, y, workspace, stream
    good = [f, None, f, f, f, f, f, None, None, f, f, None]

    def call(plan, **at):
        args = list(good)
        for n, v in at.items():
            args[int(n[1:])] = v
        return L.nm_lora(plan.handle if plan else None, *args)

    assert call(None) == bad
    for n in (0, 2, 3, 4, 5, 6, 9, 10):
        assert call(p, **{"a%d" % n: None}) == bad
    assert call(p, a1=f) == bad and call(c) == bad
    assert call(p, a7=f) == bad and call(p, a8=f) == bad and call(i) == bad and call(i, a7=f) == bad and call(i, a8=f) == bad
    for n in (0, 2, 3, 6, 8, 9, 10):
        assert call(p, **{"a%d" % n: o}) == odd
    assert call(p, a5=f + 4) == odd
    for n in (1, 4, 7):
        assert call(p, **{"a%d" % n: f + 2}) == odd
    assert L.nm_lora(plan(n=0).handle, *[None] * 12) == nm.NM_OK


def test_host_tensors_are_refused():
    p = plan()
    x, w = torch.zeros((4, 128)).half(), torch.zeros((48, 128)).half()
    with pytest.raises(ValueError, match="GPU"):
        nm.nm_lora(p, x, w, torch.zeros((192, 16)).half(), torch.ones(3), torch.zeros(4, dtype=torch.int64), x[:, :64], x[:, :64])
