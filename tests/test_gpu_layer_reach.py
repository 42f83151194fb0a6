"""Adapters, head norms and log probabilities where offsets pass 32 bits, on two streams at once, and without any token.
The same values in compact rows, or one call after the other, have to give the same bits."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from structured_sparse_gemm_nm_amd.heads import norm_rotate, rotation_table
from structured_sparse_gemm_nm_amd.logprobs import token_logprobs
from tests import test_gpu_heads as heads_of, test_gpu_logprobs as logprobs_of
from tests.test_gpu_lora import adapters

pytestmark = pytest.mark.gpu
FAR = (1 << 31) + 64          # elements from a row to the next


def far(t):
    """t's rows, FAR elements apart."""
    wide = torch.empty(((t.shape[0] - 1) * FAR + t.shape[1],), dtype=t.dtype, device="cuda").as_strided(t.shape, (FAR, 1))
    return wide.copy_(t)


def test_far_head_rows():
    s = heads_of.inputs(3, (3, 1, 1), 64, 64, "bf16", False)
    tail = s["gamma_q"].cuda(), s["gamma_k"].cuda(), s["positions"].cuda(), s["table"].cuda()
    x, dy = s["x"].cuda(), s["dy"].cuda()
    got = []
    for put, ld in ((lambda t: t.clone(), x.shape[1]), (far, FAR)):
        plan = nm.nm_heads_plan_init(3, 3, 1, 1, 64, 64, table_rows=97, dtype="bf16", ldx=ld, ldy=ld)
        a, y, dx = put(x), put(torch.zeros_like(x)), put(torch.zeros_like(x))
        dq, dk = torch.empty_like(tail[0]), torch.empty_like(tail[0])
        nm.nm_head_norm_rope(plan, a, *tail, y)
        nm.nm_head_norm_rope_backward(plan, a, *tail, put(dy), dx, dgamma_q=dq, dgamma_k=dk, workspace=plan.empty_workspace())
        got.append([t.clone() for t in (y, dx, dq, dk)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_far_angles():
    """Positions whose angles lie past 2^32 bytes of the table."""
    s = heads_of.inputs(5, (2, 1, 0), 512, 512, "f16", False)
    rows = (1 << 21) + 3
    table = torch.empty((rows, 512), device="cuda")
    table[-5:] = s["table"][:5].cuda()
    args = s["x"].cuda(), s["gamma_q"].cuda(), s["gamma_k"].cuda()
    at = torch.arange(5, device="cuda")
    want = norm_rotate(*args, at, s["table"].cuda(), (2, 1, 0))
    assert torch.equal(norm_rotate(*args, at + rows - 5, table, (2, 1, 0)), want)


def test_far_logits():
    s = logprobs_of.inputs(3, 5000, "bf16", 4)
    x, tokens = s["x"].cuda(), s["tokens"].cuda()
    got = []
    for put, ld in ((lambda t: t.clone(), 5000), (far, FAR)):
        plan = nm.nm_logprobs_plan_init(3, 5000, dtype="bf16", top=9, ldx=ld, ldg=ld)
        a, dx = put(x), put(torch.zeros_like(x))
        out = [torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty((3, 2), device="cuda"),
               torch.empty((3, 9), device="cuda"), torch.empty((3, 9), dtype=torch.int64, device="cuda")]
        nm.nm_logprobs(plan, a, tokens, out[0], entropy=out[1], stats=out[2], top_logprob=out[3], top_index=out[4],
                       workspace=plan.empty_workspace())
        nm.nm_logprobs_backward(plan, a, tokens, out[2], dx, g_logprob=s["g"].cuda(), g_entropy=s["h"].cuda(), entropy=out[1])
        got.append([t.clone() for t in (*out, dx)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_far_adapters_and_rows():
    m, k, rank, count, n = (1 << 20) + 8, 48, 128, 17, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x, base = torch.randn(n, k, generator=g, device="cuda").half(), torch.randn(n, m, generator=g, device="cuda").half()
    a = torch.randn(rank, k, generator=g, device="cuda").half()
    b, scale = (0.1 * torch.randn(m, rank, generator=g, device="cuda")).half(), torch.full((count,), 0.5, device="cuda")
    every = torch.empty((count * m, rank), dtype=torch.float16, device="cuda")       # 2.3e9 elements
    every[-m:] = b
    rows = torch.empty((count * rank, k), dtype=torch.float16, device="cuda")
    rows[-rank:] = a
    got = []
    for weights, names, put, ld in (((a, b), 1, lambda t: t.clone(), None), ((rows, every), count, far, FAR)):
        plan = nm.nm_lora_plan_init(m, n, k, rank, names, dtype="f16", ldx=ld, ldc=ld, ldy=ld)
        y = put(torch.zeros_like(base))
        index = torch.tensor([names - 1, -1, names - 1], device="cuda")
        nm.nm_lora(plan, put(x), *weights, scale[:names], index, put(base), y, workspace=plan.empty_workspace())
        got.append(y.clone())
    assert torch.equal(*got) and torch.equal(got[0][1], base[1]) and not torch.equal(got[0][2], base[2])


def test_two_streams_at_once():
    """One plan, two calls in flight: their workspaces are their own."""
    ad = adapters(40, 1024, 768, 16, torch.bfloat16, 2)
    g = torch.Generator(device="cuda").manual_seed(8)
    cases = []
    for n in (700, 700):
        x = torch.randn(n, 1024, generator=g, device="cuda").bfloat16()
        cases.append((x, torch.randint(-1, 40, (n,), generator=g, device="cuda"), torch.randn(n, 768, generator=g, device="cuda").bfloat16(),
                      torch.randn(3, 200000, generator=g, device="cuda"), torch.randint(0, 200000, (3,), generator=g, device="cuda")))
    gains = [torch.ones(64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table, at = rotation_table(700, 64), torch.arange(700, device="cuda")

    def run(x, index, base, logits, tokens):
        y = norm_rotate(ad.add(x, index, base), *gains, at, table, (8, 2, 2))
        return (y, *token_logprobs(logits, tokens, top=7, entropy=True))

    want = [run(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        got = []
        for c, stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                got.append(run(*c))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_no_tokens():
    x = torch.empty((0, 512), dtype=torch.float16, device="cuda", requires_grad=True)
    gains = [torch.ones(64, dtype=torch.float16, device="cuda", requires_grad=True) for _ in range(2)]
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    y = norm_rotate(x, *gains, none, rotation_table(4, 64), (4, 2, 2))
    out = token_logprobs(y, none, top=3, entropy=True)
    assert out.logprob.shape == (0,) and out.top_index.shape == (0, 3)
    (out.logprob.sum() + out.entropy.sum()).backward()
    assert x.grad.shape == (0, 512) and all((t.grad == 0).all() for t in gains)
    ad = adapters(3, 512, 96, 8, torch.float16, 1)
    assert ad.add(x.detach(), none, torch.empty((0, 96), dtype=torch.float16, device="cuda")).shape == (0, 96)
