"""Head norms with rotation on the GPU, and their gradients, against plain 64-bit computations.

Tolerances, in fp32 steps of 2^-24 beside half a step of the 16-bit result (HALF, and TINY under the smallest normal):

- forward: an accumulator's value takes 3; the sum of squares at most 8 in a lane's chain and 6 across lanes, half of
  that and 2 for the root and division behind it; the factor's products 2; the rotation 3, relative to |a c| + |b s|.
  Under 32: 2^-19 of that size.
- dx = f w - u f^3 / dim * sum(w u): the turned-back gradient 3, its sums at most 14, the factor 9 (three times in the
  second term), 6 products: under 64, 2^-18 of |f w| + |u| f^3 / dim * sum |w u|, sizes as above.
- dgamma: a term 20, a lane's chain of fp32 sums at most tokens a block times heads a group (under 40 here), the groups'
  64: under 128, 2^-17 of the sum of the terms' sizes."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from structured_sparse_gemm_nm_amd.feed_forward import Rows
from structured_sparse_gemm_nm_amd.heads import norm_rotate, rotation_table
from tests.test_gpu_layer_ops import HALF, TINY, TORCH, Out, close, gen, strided, up16

pytestmark = pytest.mark.gpu
FWD, BACK, GAIN = 2.0 ** -19, 2.0 ** -18, 2.0 ** -17


def inputs(rows, heads, dim, rotary, dtype, acc, table=97, seed=1, table_on="cuda"):
    g, cols = gen(seed), sum(heads) * dim
    s = {"row_scale": None, "col_scale": None, "heads": heads, "dim": dim, "rotary": rotary, "dtype": dtype}
    if acc:
        s["x"] = (torch.randn(rows, cols, generator=g) * 1e5).round().to(torch.int32)
        s["row_scale"] = 0.02 + 0.02 * torch.rand(rows, generator=g)
        s["col_scale"] = 2e-4 + 3e-4 * torch.rand(cols, generator=g)
    else:
        s["x"] = (2 * torch.randn(rows, cols, generator=g)).to(TORCH[dtype])
    s["gamma_q"], s["gamma_k"] = ((1 + 0.3 * torch.randn(dim, generator=g)).to(TORCH[dtype]) for _ in range(2))
    s["positions"] = torch.randint(0, table, (rows,), generator=g)
    s["table"] = rotation_table(table, rotary, device="cpu")
    s["dy"] = torch.randn(rows, cols, generator=g).to(TORCH[dtype])
    return s


def turn(v, c, sn, pairs, size=False):
    half = v.shape[-1] // 2
    a, b = (v[..., :half], v[..., half:]) if pairs == "halves" else (v[..., 0::2], v[..., 1::2])
    out = (a * c + b * sn, b * c + a * sn) if size else (a * c - b * sn, b * c + a * sn)
    return torch.cat(out, -1) if pairs == "halves" else torch.stack(out, -1).flatten(-2)


def plain(s, pairs, eps, gamma_q=None, gamma_k=None, x=None):
    """(y, size of its errors) in 64 bits, rows x heads x dim."""
    q, k, _ = s["heads"]
    dim, rot, rows = s["dim"], s["rotary"], s["x"].shape[0]
    u = s["x"].double() if x is None else x
    if s["row_scale"] is not None:
        u = u * s["row_scale"].double()[:, None] * s["col_scale"].double()
    u = u.reshape(rows, -1, dim)
    gq = s["gamma_q"].double() if gamma_q is None else gamma_q
    gk = s["gamma_k"].double() if gamma_k is None else gamma_k
    gamma = torch.cat((gq.expand(q, dim), gk.expand(k, dim)))
    t = s["table"].double()[s["positions"].clamp(0, s["table"].shape[0] - 1)][:, None]
    c, sn = t[..., :rot // 2], t[..., rot // 2:]
    qk = u[:, :q + k]
    v = qk * gamma / (qk.square().mean(-1, keepdim=True) + eps).sqrt()
    y = torch.cat((turn(v[..., :rot], c, sn, pairs), v[..., rot:]), -1)
    size = torch.cat((turn(v[..., :rot].abs(), c.abs(), sn.abs(), pairs, True), v[..., rot:].abs()), -1)
    return torch.cat((y, u[:, q + k:]), 1), torch.cat((size, u[:, q + k:].abs()), 1)


def plain_back(s, pairs, eps):
    """(dx, dgamma_q, dgamma_k) and the sizes of their errors."""
    q, k, _ = s["heads"]
    dim, rot, rows = s["dim"], s["rotary"], s["x"].shape[0]
    u = s["x"].double().reshape(rows, -1, dim)
    dy = s["dy"].double().reshape(rows, -1, dim)
    gamma = torch.cat((s["gamma_q"].double().expand(q, dim), s["gamma_k"].double().expand(k, dim)))
    t = s["table"].double()[s["positions"].clamp(0, s["table"].shape[0] - 1)][:, None]
    c, sn = t[..., :rot // 2], t[..., rot // 2:]
    qk, g = u[:, :q + k], dy[:, :q + k]
    gs = torch.cat((turn(g[..., :rot].abs(), c.abs(), sn.abs(), pairs, True), g[..., rot:].abs()), -1)
    g = torch.cat((turn(g[..., :rot], c, -sn, pairs), g[..., rot:]), -1)
    f = 1 / (qk.square().mean(-1, keepdim=True) + eps).sqrt()
    w, ws = g * gamma, gs * gamma.abs()
    dx = f * w - qk * f ** 3 / dim * (w * qk).sum(-1, keepdim=True)
    size = f * ws + qk.abs() * f ** 3 / dim * (ws * qk.abs()).sum(-1, keepdim=True)
    term, terms = g * qk * f, gs * qk.abs() * f
    token = (s["positions"] >= 0).double()[:, None, None]
    dx = torch.cat((dx, dy[:, q + k:]), 1) * token
    size = torch.cat((size, dy[:, q + k:].abs()), 1)
    term, terms = term * token, terms * token
    return (dx, term[:, :q].sum((0, 1)), term[:, q:].sum((0, 1))), (size, terms[:, :q].sum((0, 1)), terms[:, q:].sum((0, 1)))


def cuda(t):
    return None if t is None else t.cuda()


def run(s, pairs, eps=1e-6, pad=0, in_place=False, table=True, zero_rows=False):
    rows, cols = s["x"].shape
    ld, acc = up16(cols) + pad, s["row_scale"] is not None
    x, _ = strided(s["x"], ld, 77)
    plan = nm.nm_heads_plan_init(rows, *s["heads"], s["dim"], s["rotary"], pairs=pairs, table_rows=s["table"].shape[0],
                                 dtype=s["dtype"], x_dtype="i32" if acc else None, ldx=ld, ldy=ld, eps=eps, zero_rows=zero_rows)
    out = Out(rows, cols, ld, TORCH[s["dtype"]])
    y = x if in_place else out.t
    nm.nm_head_norm_rope(plan, x, s["gamma_q"].cuda(), s["gamma_k"].cuda(), s["positions"].cuda(),
                         s["table"].cuda() if s["rotary"] else None, y, row_scale=cuda(s["row_scale"]), col_scale=cuda(s["col_scale"]))
    torch.cuda.synchronize()
    out.check()
    return y, plan, x, ld


def check(s, pairs, eps=1e-6, **kw):
    y, plan, x, ld = run(s, pairs, eps, **kw)
    want, size = plain(s, pairs, eps)
    want, size = want.flatten(1), size.flatten(1)
    close(y, want, HALF[s["dtype"]] * want.abs() + FWD * size * (1 + HALF[s["dtype"]]) + TINY[s["dtype"]], "y")
    return plan, x, ld


SHAPES = [
    (1, (32, 8, 8), 128, 128), (3, (1, 0, 0), 8, 8), (5, (3, 1, 2), 40, 16), (130, (20, 5, 0), 80, 32), (17, (4, 4, 4), 64, 64),
    (9, (2, 1, 1), 96, 96), (7, (5, 2, 1), 256, 64), (2, (3, 1, 1), 264, 264), (300, (7, 3, 2), 512, 256), (33, (6, 2, 2), 128, 0),
    (1500, (9, 3, 0), 72, 72), (64, (70, 1, 1), 24, 8),
]


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("rows,heads,dim,rotary", SHAPES)
def test_forward(rows, heads, dim, rotary, acc, dtype, pairs):
    check(inputs(rows, heads, dim, rotary, dtype, acc, seed=rows + dim), pairs, pad=16 * (rows % 2))


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,heads,dim,rotary", SHAPES)
def test_backward(rows, heads, dim, rotary, dtype, pairs):
    s = inputs(rows, heads, dim, rotary, dtype, False, seed=rows + dim)
    s["positions"][rows // 2::5] = -1
    pad = 16 * (rows % 2)
    cols = s["x"].shape[1]
    ld = up16(cols) + pad
    x, _ = strided(s["x"], ld, 77)
    dy, _ = strided(s["dy"], ld, 77)
    plan = nm.nm_heads_plan_init(rows, *heads, dim, rotary, pairs=pairs, table_rows=97, dtype=dtype, ldx=ld, ldy=ld)
    dx, dt = Out(rows, cols, ld, TORCH[dtype]), TORCH[dtype]
    dq, dk = (torch.full((dim + 8,), 93.0, dtype=dt, device="cuda") for _ in range(2))
    ws = plan.empty_workspace()
    args = x, s["gamma_q"].cuda(), s["gamma_k"].cuda() if heads[1] else None, s["positions"].cuda(), s["table"].cuda() if rotary else None
    nm.nm_head_norm_rope_backward(plan, *args, dy, dx.t, dgamma_q=dq[:dim], dgamma_k=dk[:dim] if heads[1] else None, workspace=ws)
    torch.cuda.synchronize()
    dx.check()
    assert (dq[dim:] == 93).all() and (dk[dim if heads[1] else 0:] == 93).all()
    want, size = plain_back(s, pairs, 1e-6)
    half, tiny = HALF[dtype], TINY[dtype]
    close(dx.t, want[0].flatten(1), half * want[0].flatten(1).abs() + BACK * 2 * size[0].flatten(1) + tiny, "dx")
    assert (dx.t[s["positions"].cuda() < 0] == 0).all()
    for got, w, z, there in ((dq, want[1], size[1], True), (dk, want[2], size[2], heads[1])):
        if there:
            close(got[:dim], w, half * w.abs() + GAIN * 2 * z + tiny, "dgamma")
    # without the gains the rows' gradient is the same; it may take the output gradient's place; and it repeats bit for bit
    again = dy.clone() if ld == cols else strided(s["dy"], ld, 77)[0]
    nm.nm_head_norm_rope_backward(plan, *args, again, again)
    assert torch.equal(again, dx.t)
    dq2, dk2 = torch.empty_like(dq[:dim]), torch.empty_like(dk[:dim])
    ws.fill_(255)
    nm.nm_head_norm_rope_backward(plan, *args, dy, dx.t, dgamma_q=dq2, dgamma_k=dk2 if heads[1] else None, workspace=ws)
    assert torch.equal(dq2, dq[:dim]) and (not heads[1] or torch.equal(dk2, dk[:dim]))


def test_gradient_formula_against_differences():
    s = inputs(2, (2, 1, 1), 16, 8, "f16", False, seed=5)
    for pairs in ("halves", "neighbours"):
        x, gq, gk = s["x"].double(), s["gamma_q"].double(), s["gamma_k"].double()
        dy = s["dy"].double().reshape(2, -1, 16)
        f = lambda **kw: (plain(s, pairs, 1e-6, **kw)[0] * dy).sum()  # noqa: E731
        (dx, dq, dk), _ = plain_back(s, pairs, 1e-6)
        h = 1e-6
        for i in range(x.numel()):
            e = torch.zeros(x.numel(), dtype=torch.float64)
            e[i] = h
            e = e.view_as(x)
            assert abs((f(x=x + e) - f(x=x - e)) / (2 * h) - dx.reshape(-1)[i]) < 1e-7
        for i in range(16):
            e = torch.zeros(16, dtype=torch.float64)
            e[i] = h
            assert abs((f(gamma_q=gq + e) - f(gamma_q=gq - e)) / (2 * h) - dq[i]) < 1e-7
            assert abs((f(gamma_k=gk + e) - f(gamma_k=gk - e)) / (2 * h) - dk[i]) < 1e-7


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_in_place(dtype, pairs):
    s = inputs(70, (6, 2, 2), 80, 48, dtype, False)
    y, _, _, _ = run(s, pairs)
    z, _, _, _ = run(s, pairs, in_place=True)
    assert torch.equal(y, z)


@pytest.mark.parametrize("acc", [False, True])
def test_rows_without_a_token_stay_as_they_were(acc):
    s = inputs(40, (4, 2, 2), 64, 64, "bf16", acc)
    whole = run(s, "halves")[0].clone()
    s["positions"][[0, 7, 39]] = torch.tensor([-1, -(1 << 40), -100])
    y = run(s, "halves")[0]
    out = s["positions"].cuda() < 0
    assert (y[out] == 93).all() and torch.equal(y[~out], whole[~out])


@pytest.mark.parametrize("rows,heads,dim", [(3, (5, 1, 1), 80), (400, (20, 3, 2), 512), (70, (1, 0, 0), 8)])
@pytest.mark.parametrize("acc", [False, True])
def test_rows_without_a_token_become_zeros(rows, heads, dim, acc):
    s = inputs(rows, heads, dim, dim, "bf16", acc)
    y, _, _, _ = run(s, "halves")
    s["positions"][::2] = -1 - torch.arange(0, rows, 2) * (1 << 40)
    z, _, _, _ = run(s, "halves", zero_rows=True)
    assert (z[::2] == 0).all() and torch.equal(z[1::2], y[1::2])


def test_a_position_behind_the_table_is_nan():
    s = inputs(12, (2, 1, 1), 64, 32, "f16", False, table=50)
    want = run(s, "neighbours")[0].clone().view(12, 4, 64)
    s["positions"][3], s["positions"][8] = 50, 1 << 40
    y = run(s, "neighbours")[0].view(12, 4, 64)
    far = torch.zeros(12, dtype=torch.bool, device="cuda")
    far[[3, 8]] = True
    assert torch.equal(y[~far], want[~far])
    assert y[far][:, :3, :32].isnan().all() and torch.equal(y[far][:, :3, 32:], want[far][:, :3, 32:])
    assert torch.equal(y[far][:, 3], want[far][:, 3])


def test_what_is_not_finite_stays_in_its_head():
    s = inputs(6, (3, 2, 1), 128, 128, "bf16", False)
    want = run(s, "halves")[0].clone().view(6, 6, 128)
    s["x"][2, 128 + 5], s["x"][4, 5 * 128 + 3] = float("nan"), float("inf")
    y = run(s, "halves")[0].view(6, 6, 128)
    assert y[2, 1].isnan().all() and y[4, 5, 3] == float("inf")
    y[2, 1], want[2, 1] = 0, 0
    y[4, 5, 3] = want[4, 5, 3]
    assert torch.equal(y, want)


def test_heads_of_zeros_and_far_positions():
    s = inputs(3, (2, 1, 0), 64, 64, "f16", False, table=1 << 17)
    s["x"][:, :64] = 0
    s["positions"] = torch.tensor([(1 << 17) - 1, 0, 99999])
    check(s, "halves")
    y = run(s, "halves", eps=0.0)[0].view(3, 3, 64)
    assert y[:, 0].isnan().all() and y[:, 1:].isfinite().all()


def test_no_rows():
    plan = nm.nm_heads_plan_init(0, 2, 1, 1, 64, 64, table_rows=8)
    g, table = torch.ones(64, dtype=torch.float16, device="cuda"), rotation_table(8, 64)
    none, at = torch.empty((0, 256), dtype=torch.float16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    nm.nm_head_norm_rope(plan, none, g, g, at, table, none)
    dq, dk = torch.ones_like(g), torch.ones_like(g)
    nm.nm_head_norm_rope_backward(plan, none, g, g, at, table, none, none, dgamma_q=dq, dgamma_k=dk, workspace=plan.empty_workspace())
    assert (dq == 0).all() and (dk == 0).all()


def test_captured_and_on_another_stream():
    s = inputs(200, (8, 2, 2), 128, 128, "bf16", False)
    plan = nm.nm_heads_plan_init(200, 8, 2, 2, 128, 128, table_rows=97, dtype="bf16")
    x, dy = s["x"].cuda(), s["dy"].cuda()
    args = s["gamma_q"].cuda(), s["gamma_k"].cuda(), s["positions"].cuda(), s["table"].cuda()
    y, dx, dq, dk = torch.empty_like(x), torch.empty_like(x), torch.empty_like(args[0]), torch.empty_like(args[0])
    ws = plan.empty_workspace()

    def step():
        nm.nm_head_norm_rope(plan, x, *args, y)
        nm.nm_head_norm_rope_backward(plan, x, *args, dy, dx, dgamma_q=dq, dgamma_k=dk, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want = [t.clone() for t in (y, dx, dq, dk)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.mul_(-1 if i else 1)
        for t in (y, dx, dq, dk):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dq, dk)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, dx, dq, dk)))
        if i == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_wrapper_and_its_gradients():
    s = inputs(50, (4, 2, 2), 64, 64, "bf16", False)
    s["positions"][::7] = -1
    x = s["x"].cuda().requires_grad_()
    gq, gk = s["gamma_q"].cuda().requires_grad_(), s["gamma_k"].cuda().requires_grad_()
    at, table = s["positions"].cuda(), s["table"].cuda()
    y = norm_rotate(x, gq, gk, at, table, (4, 2, 2))
    with torch.no_grad():
        assert torch.equal(y, norm_rotate(x, gq, gk, at, table, (4, 2, 2))) and (y[at < 0] == 0).all()
    want, size = plain(s, "halves", 1e-6)
    ok = (s["positions"] >= 0)
    want, size = want.flatten(1)[ok], size.flatten(1)[ok]
    close(y[at >= 0], want, HALF["bf16"] * want.abs() + 2 * FWD * size + TINY["bf16"], "y")
    dy = s["dy"].cuda()
    (y.t() * dy.t()).sum().backward()                  # an output gradient of its own strides
    want, size = plain_back(s, "halves", 1e-6)
    for got, w, z, rel in ((x.grad, want[0].flatten(1), size[0].flatten(1), BACK), (gq.grad, want[1], size[1], GAIN),
                           (gk.grad, want[2], size[2], GAIN)):
        close(got, w, HALF["bf16"] * w.abs() + 2 * rel * z + TINY["bf16"], "gradient")
    # gains alone, rows alone, and rows that lie elsewhere
    gq.grad = None
    norm_rotate(x.detach(), gq, gk.detach(), at, table, (4, 2, 2)).backward(dy)
    close(gq.grad, want[1], HALF["bf16"] * want[1].abs() + 2 * GAIN * size[1] + TINY["bf16"], "gradient")
    wide = torch.zeros((50, 520), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:515] = x.detach()
    assert torch.equal(norm_rotate(wide[:, 3:515], gq.detach(), gk.detach(), at, table, (4, 2, 2)), y)


def test_wrapper_refuses():
    s = inputs(4, (2, 1, 1), 32, 32, "f16", True)
    gq, at, table = s["gamma_q"].cuda(), s["positions"].cuda(), s["table"].cuda()
    rows = Rows(s["x"].cuda(), s["row_scale"].cuda(), s["col_scale"].cuda())
    norm_rotate(rows, gq, gq, at, table, (2, 1, 1))
    for args in ((rows.values, gq, gq, at, table, (2, 1, 1)), (Rows(*rows[:2]), gq, gq, at, table, (2, 1, 1)),
                 (rows, gq, None, at, table, (2, 1, 1)), (rows, gq, gq, at, table, (2, 1, 2)), (rows, gq, gq, at, table, (2, 1)),
                 (rows, gq.float(), gq, at, table, (2, 1, 1)), (rows, gq, gq.bfloat16(), at, table, (2, 1, 1)),
                 (rows, gq, gq, at.int(), table, (2, 1, 1)), (rows, gq, gq, at[:3], table, (2, 1, 1)),
                 (rows, gq, gq, at.cpu(), table, (2, 1, 1)), (rows, gq, gq, at, table.half(), (2, 1, 1)),
                 (rows.dense(), gq, gq, at, table, (2, 1, 1))):
        with pytest.raises((ValueError, nm.NmError)):
            norm_rotate(*args)
    with pytest.raises(RuntimeError, match="gradient"):
        norm_rotate(rows, gq.clone().requires_grad_(), gq, at, table, (2, 1, 1))
    with pytest.raises(RuntimeError, match="gradient"):
        norm_rotate(rows, gq, gq, at, table.clone().requires_grad_(), (2, 1, 1))
    with pytest.raises(RuntimeError, match="gradient"):
        norm_rotate(rows.dense().half().requires_grad_(), gq, gq, at, table.clone().requires_grad_(), (2, 1, 1))


def test_gains_of_many_tokens():
    """40000 tokens: 79 of them a block, three chains of sums. Sums of squares of one sign are where a chain loses most."""
    rows = 40000
    s = inputs(rows, (2, 1, 0), 16, 0, "f16", False)
    s["x"] = s["x"].abs() + 0.5
    s["dy"] = s["dy"].abs() + 0.5
    s["gamma_q"], s["gamma_k"] = s["gamma_q"].abs() + 0.1, s["gamma_k"].abs() + 0.1
    plan = nm.nm_heads_plan_init(rows, 2, 1, 0, 16, 0, dtype="f16")
    x, dy = s["x"].cuda(), (s["dy"] / 16384).cuda()
    s["dy"] = dy.cpu()
    dx, dq, dk = torch.empty_like(x), torch.empty(16, dtype=torch.float16, device="cuda"), torch.empty(16, dtype=torch.float16, device="cuda")
    nm.nm_head_norm_rope_backward(plan, x, s["gamma_q"].cuda(), s["gamma_k"].cuda(), s["positions"].cuda(), None, dy, dx, dgamma_q=dq,
                                  dgamma_k=dk, workspace=plan.empty_workspace())
    want, size = plain_back(s, "halves", 1e-6)
    for got, w, z in ((dq, want[1], size[1]), (dk, want[2], size[2])):
        close(got, w, HALF["f16"] * w.abs() + GAIN * z + TINY["f16"], "dgamma")
