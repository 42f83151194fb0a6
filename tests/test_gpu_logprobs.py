"""Log probabilities on the GPU, and the logits' gradient, against plain 64-bit computations.

Tolerances, in fp32 steps of 2^-24. P is the number of pieces that a thread adds up.

- the sum of exponentials: a term's exponent takes 3 steps of its size, weighted by its probability at most 3 (log N + 1)
  < 50; each piece one addition and at most one change of the largest (4), the joins under 32, a few for the rest:
  5 P + 100, relative. A log probability adds 3 steps of |z - max| and 2 of |log sum|, the entropy's weighted sum 10:
  error(P) = (5 P + 160) 2^-24 (2 + log N + |value|) covers each.
- the gradient: p is off by error(P) relative, log p + H by two of them, then 4 products; half a step of the result's type
  (HALF, TINY)."""
import math

import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from structured_sparse_gemm_nm_amd.feed_forward import Rows
from structured_sparse_gemm_nm_amd.logprobs import token_logprobs
from tests.test_gpu_layer_ops import HALF as HALF16, TINY as TINY16, TORCH as TORCH16, Out, close, gen, strided, up16

pytestmark = pytest.mark.gpu
TORCH = dict(TORCH16, f32=torch.float32)
HALF = dict(HALF16, f32=2.0 ** -24)
TINY = dict(TINY16, f32=2.0 ** -149)
INF = math.inf


def inputs(rows, cols, dtype, seed, spread=2.5):
    g = gen(seed)
    s = {"row_scale": None, "col_scale": None, "dtype": dtype}
    if dtype == "i32":
        s["x"] = (torch.randn(rows, cols, generator=g) * 1e5).round().to(torch.int32)
        s["row_scale"] = 0.02 + 0.02 * torch.rand(rows, generator=g)
        s["col_scale"] = 2e-4 + 3e-4 * torch.rand(cols, generator=g)
    else:
        s["x"] = (spread * torch.randn(rows, cols, generator=g)).to(TORCH[dtype])
    s["tokens"] = torch.randint(0, cols, (rows,), generator=g)
    s["g"], s["h"] = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    return s


def logits(s):
    x = s["x"].float()
    return x if s["row_scale"] is None else (x * s["row_scale"][:, None]) * s["col_scale"]


def plain(s, scale):
    """log p (rows x cols) and entropy in 64 bits; rows without any weight and rows without a distribution by their rule."""
    z = logits(s).double() * float(torch.tensor(scale))
    top = z.amax(1, keepdim=True)
    bad = z.isnan().any(1) | (top[:, 0] == INF)
    none = top[:, 0] == -INF
    z = z - torch.where(top.isfinite(), top, 0.0)       # 64 bits lose the sum beside logits of 1e38
    logp = z - torch.logsumexp(z, 1, keepdim=True)
    logp[none] = -INF
    logp[bad] = math.nan
    p = logp.exp()
    H = -torch.where(p > 0, p * logp, torch.where(p.isnan(), p, 0.0)).sum(1)
    return logp, H, bad


def error(plan, cols, value):
    pieces = -(-cols // 8)
    return (5 * min(64, -(-pieces // 64)) + 160) * 2.0 ** -24 * (2 + math.log(cols) + value.abs().clamp(max=1e30))


def call(s, top=0, scale=1.0, entropy=True, stats=True, pad=0):
    rows, cols = s["x"].shape
    ld = up16(cols) + pad
    x, _ = strided(s["x"], ld, 77)
    plan = nm.nm_logprobs_plan_init(rows, cols, dtype=s["dtype"], top=top, scale=scale, ldx=ld, ldg=ld)
    raw = {"logprob": torch.full((rows + 8,), 93.0, device="cuda"), "entropy": torch.full((rows + 8,), 93.0, device="cuda"),
           "stats": torch.full((rows + 8, 2), 93.0, device="cuda")}
    out = {k: v[:rows] for k, v in raw.items()}
    out["top_logprob"] = torch.full((rows, top), 93.0, device="cuda") if top else None
    out["top_index"] = torch.full((rows, top), 93, dtype=torch.int64, device="cuda") if top else None
    work = plan.empty_workspace()
    if work is not None:
        work.fill_(255)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    nm.nm_logprobs(plan, x, s["tokens"].cuda(), out["logprob"], entropy=out["entropy"] if entropy else None,
                   stats=out["stats"] if stats else None, top_logprob=out["top_logprob"], top_index=out["top_index"],
                   row_scale=cuda(s["row_scale"]), col_scale=cuda(s["col_scale"]), workspace=work)
    torch.cuda.synchronize()
    for k in raw:
        assert (raw[k][rows:] == 93).all()
    return plan, x, out


def check(s, top=0, scale=1.0, pad=0, **kw):
    rows, cols = s["x"].shape
    plan, x, out = call(s, top, scale, pad=pad, **kw)
    logp, H, bad = plain(s, scale)
    t = s["tokens"]
    want = torch.where(t >= 0, logp.gather(1, t.clamp(0, cols - 1)[:, None])[:, 0], 0.0)
    want[t >= cols] = math.nan
    same(out["logprob"], want, error(plan, cols, want), "logprob")
    if kw.get("entropy", True):
        same(out["entropy"], H, error(plan, cols, H), "entropy")
    if top:
        order = torch.sort(logits(s), dim=1, descending=True, stable=True)[1][:, :top]
        order[bad] = -1
        assert torch.equal(out["top_index"].cpu(), order)
        best = torch.where(order >= 0, logp.gather(1, order.clamp_min(0)), math.nan)
        same(out["top_logprob"], best, error(plan, cols, best), "top")
    return plan, x, out


def same(got, want, tol, what):
    got = got.double().cpu()
    odd = ~want.isfinite()
    assert torch.equal(got[odd].isnan(), want[odd].isnan()) and torch.equal(got[odd].nan_to_num(), want[odd].nan_to_num()), what
    close(got[~odd], want[~odd], tol[~odd], what)


SHAPES = [(1, 1), (3, 5), (2, 7), (5, 8), (4, 9), (33, 63), (70, 513), (9, 2048), (5, 2049), (1, 32003), (3, 50001), (1100, 2500),
          (300, 9001), (1030, 4097), (2, 300000), (1, 1 << 20), (3, 1000003)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32", "i32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype):
    s = inputs(rows, cols, dtype, rows + cols)
    s["tokens"][rows // 3::4] = -1 - rows
    for top, scale, entropy in ((0, 1.0, True), (min(cols, 5), 0.7, False), (min(cols, 32), 1.5, True)):
        check(s, top, scale, pad=16 * (top % 2), entropy=entropy, stats=entropy)


@pytest.mark.parametrize("terms", ["logprob", "entropy", "both"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (4, 9), (33, 63), (5, 2049), (1, 32003), (40, 8192), (300, 9001), (2, 300000)])
def test_backward(rows, cols, dtype, terms):
    s = inputs(rows, cols, dtype, rows + cols, spread=1.5)
    s["tokens"][rows // 2::3] = -100
    scale, pad = 0.8, 16 * (rows % 2)
    plan, x, out = check(s, 0, scale, pad=pad)
    g = s["g"] if terms != "entropy" else None
    h = s["h"] if terms != "logprob" else None
    ld = up16(cols) + pad
    dx = Out(rows, cols, ld, TORCH[dtype])
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(g_logprob=cuda(g), g_entropy=cuda(h), entropy=out["entropy"] if h is not None else None)
    tokens = s["tokens"].cuda() if g is not None else None
    nm.nm_logprobs_backward(plan, x, tokens, out["stats"], dx.t, **kw)
    torch.cuda.synchronize()
    dx.check()
    logp, H, _ = plain(s, scale)
    p, f = logp.exp(), float(torch.tensor(scale))
    zero = torch.zeros(rows, dtype=torch.float64)
    gg = torch.where(s["tokens"] >= 0, g.double(), 0.0) if g is not None else zero
    hh = h.double() if h is not None else zero
    hit = torch.zeros_like(p).scatter_(1, s["tokens"].clamp_min(0)[:, None], 1.0)
    want = f * (gg[:, None] * (hit - p) - hh[:, None] * p * (logp + H[:, None]))
    e = error(plan, cols, logp.abs() + H[:, None])
    tol = f * p * ((e + 2.0 ** -21) * (gg.abs()[:, None] + hh.abs()[:, None] * (logp + H[:, None]).abs()) + 2 * e * hh.abs()[:, None])
    tol += f * hit * gg.abs()[:, None] * 2.0 ** -22 + 2.0 ** -140
    close(dx.t, want, tol * (1 + HALF[dtype]) + HALF[dtype] * want.abs() + TINY[dtype], "dx")
    nm.nm_logprobs_backward(plan, x, tokens, out["stats"], x, **kw)       # in the logits' place
    assert torch.equal(x, dx.t)


def test_gradient_formula_against_differences():
    s = inputs(3, 11, "f32", 4)
    s["x"], g, h, scale, d = s["x"].double(), s["g"].double(), s["h"].double(), 0.75, 1e-6

    def loss(x):
        z = x * scale
        logp = z - torch.logsumexp(z, 1, keepdim=True)
        return (g * logp.gather(1, s["tokens"][:, None])[:, 0] - h * (logp.exp() * logp).sum(1)).sum()

    z = s["x"] * scale
    logp = z - torch.logsumexp(z, 1, keepdim=True)
    p, H = logp.exp(), -(logp.exp() * logp).sum(1)
    hit = torch.zeros_like(p).scatter_(1, s["tokens"][:, None], 1.0)
    want = scale * (g[:, None] * (hit - p) - h[:, None] * p * (logp + H[:, None]))
    for i in range(33):
        e = torch.zeros(33, dtype=torch.float64)
        e[i] = d
        e = e.view(3, 11)
        assert abs((loss(s["x"] + e) - loss(s["x"] - e)) / (2 * d) - want.reshape(-1)[i]) < 1e-8


def backward(s, plan, x, out, g=True, h=True):
    dx = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    nm.nm_logprobs_backward(plan, x, s["tokens"].cuda() if g else None, out["stats"], dx, g_logprob=s["g"].cuda() if g else None,
                            g_entropy=s["h"].cuda() if h else None, entropy=out["entropy"] if h else None)
    return dx


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(6, 40), (6, 2500), (1100, 4100)])
def test_masks(rows, cols, dtype):
    """Logits ruled out by -infinity and by the type's lowest value; rows of nothing else; infinities and NaN."""
    s = inputs(rows, cols, dtype, 3)
    x, low = s["x"], torch.finfo(TORCH[dtype]).min
    x[0, 3:] = -INF                      # three are left, fewer than the alternatives
    x[1] = -INF                          # nothing is left
    x[2, 1::2] = low
    x[3] = low                           # all alike
    x[4, cols // 2] = math.nan
    x[5, cols // 3] = INF
    s["tokens"][:6] = torch.tensor([1, 2, cols - 1, 0, 0, cols // 3])
    plan, xg, out = check(s, top=min(cols, 20))
    assert out["logprob"][1] == -INF and out["entropy"][1] == 0
    assert out["logprob"][4:6].isnan().all() and out["entropy"][4:6].isnan().all()
    assert (out["top_index"][4:6] == -1).all() and out["top_logprob"][4:6].isnan().all()
    dx = backward(s, plan, xg, out)
    assert (dx[0, 3:] == 0).all() and (dx[1] == 0).all() and (dx[2, 1:-1:2] == 0).all()
    assert dx[4:6].isnan().all() and dx[:4].isfinite().all() and dx[6:].isfinite().all()
    s["tokens"][4] = -1
    assert call(s, 4)[2]["logprob"][4] == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 513), (1, 32003), (7, 2048), (3, 140001), (1100, 4100)])
def test_alternatives_among_logits_ruled_out(rows, cols, dtype):
    """Few logits are left, or all but the last columns' are equal, or two low values mix: the lowest columns come next."""
    s = inputs(rows, cols, dtype, cols)
    x, low = s["x"], torch.finfo(TORCH[dtype]).min
    g = gen(5)
    for row in range(min(rows, 7)):
        kept = torch.randperm(cols, generator=g)[:(0, 1, 3, 19, 20, 40, 7)[row]]
        values = x[row, kept].clone()
        x[row] = -INF if row % 2 else low
        if row == 4:
            x[row, cols // 2:] = -INF
        if row == 5:
            x[row, cols - 9:] = low                     # the larger of the low ones come last
        if row == 6:
            x[row] = -1.5
            x[row, :cols // 3] = -INF                   # ties begin far from the row's start
        x[row, kept] = values
    check(s, top=20)
    check(s, top=1)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [5, 2500])
def test_padded_rows_have_gradient_zero(cols, dtype):
    """Whatever lies in them: their tokens are none, and the entropy's gradient is 0 or left out."""
    s = inputs(6, cols, dtype, 3)
    s["x"][1], s["x"][3, cols // 2], s["x"][4, 0] = math.nan, INF, math.nan
    s["tokens"][1:5], s["h"][1:5] = torch.tensor([-1, -100, -1, -1]), torch.tensor([0.0, 0.0, -0.0, 0.0])
    plan, xg, out = call(s)
    for h in (False, True):
        dx = backward(s, plan, xg, out, h=h)
        assert (dx[1:5] == 0).all() and (dx[0] != 0).any() and (dx[5] != 0).any()


@pytest.mark.parametrize("scale", [2.0 ** 127, 2.0 ** -126])
def test_the_scale_at_its_bounds(scale):
    """Nothing but the largest logit is left, or all alike; the next logits are 1 below it, times 2^127 still finite."""
    x = torch.tensor([[0.0, -1.0, -2.0 ** -20, -1.0] * 100, [3.0] + [2.0] * 399], device="cuda")
    plan = nm.nm_logprobs_plan_init(2, 400, dtype="f32", scale=scale)
    out, H, at = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.tensor([4, 0], device="cuda")
    nm.nm_logprobs(plan, x, at, out, entropy=H, workspace=plan.empty_workspace())
    want = torch.tensor([100.0, 1.0] if scale > 1 else [400.0, 400.0]).log()
    assert torch.allclose(out.cpu(), -want, rtol=1e-6, atol=1e-6) and torch.allclose(H.cpu(), want, rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("scale", [1.0, 3.0])
def test_a_token_ruled_out(scale):
    s = inputs(4, 100, "f32", 8)
    s["x"][:, 50:] = -INF
    s["tokens"][:] = torch.tensor([49, 50, 99, 100])
    plan, x, out = check(s, 3, scale)
    assert out["logprob"][1] == -INF and out["logprob"][2] == -INF and out["logprob"][3].isnan()
    dx = backward(s, plan, x, out)
    assert dx[:3].isfinite().all() and dx[3].isnan().all()


@pytest.mark.parametrize("dtype", ["f16", "f32", "i32"])
@pytest.mark.parametrize("order", ["alike", "rising", "falling", "few values", "signed zeros", "one lane"])
@pytest.mark.parametrize("rows,cols", [(1, 70001), (2, 4096), (1050, 3001)])
def test_alternatives_of_every_order(rows, cols, order, dtype):
    s = inputs(rows, cols, dtype, 5)
    at = torch.arange(cols, dtype=torch.float64)
    if order == "alike":
        v = torch.full((cols,), 3.0)
    elif order == "rising":
        v = at / cols * 200 - 100
    elif order == "falling":
        v = 100 - at / cols * 200
    elif order == "few values":
        v = (at * 7 % 5) - 2
    elif order == "signed zeros":
        v = torch.where(at % 3 == 0, 0.0, torch.where(at % 3 == 1, -0.0, -1.0))
    else:                                # the largest all meet in one thread
        v = torch.where(at // 8 % 256 == 17, at, -1.0) / cols
    if dtype == "i32":
        s["x"] = (v * 1000).round().to(torch.int32).expand(rows, cols).contiguous()
        s["row_scale"][:], s["col_scale"][:] = 1.0, 2.0 ** -10
    else:
        s["x"] = v.to(TORCH[dtype]).expand(rows, cols).contiguous()
    for top in (1, 20, 32):
        check(s, top)


def test_scores_far_from_zero():
    s = inputs(8, 3001, "f32", 6)
    s["x"] += torch.tensor([1e4, -1e4, 3e5, 0, 1e-30, 0, 2e38, -2e38])[:, None]
    check(s, 7)
    check(s, 7, scale=1e-3)


def test_nothing_to_do():
    plan = nm.nm_logprobs_plan_init(0, 100, dtype="f32", top=3)
    none, at = torch.empty((0, 100), device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    row = torch.empty(0, device="cuda")
    nm.nm_logprobs(plan, none, at, row, entropy=row, top_logprob=torch.empty((0, 3), device="cuda"),
                   top_index=torch.empty((0, 3), dtype=torch.int64, device="cuda"), workspace=plan.empty_workspace())
    nm.nm_logprobs_backward(plan, none, at, torch.empty((0, 2), device="cuda"), none, g_logprob=row)
    s = inputs(5, 64, "f16", 1)           # alternatives and entropy alone
    plan = nm.nm_logprobs_plan_init(5, 64, top=2)
    lp, at = torch.empty((5, 2), device="cuda"), torch.empty((5, 2), dtype=torch.int64, device="cuda")
    nm.nm_logprobs(plan, s["x"].cuda(), top_logprob=lp, top_index=at)
    assert torch.equal(at.cpu(), torch.sort(s["x"].float(), dim=1, descending=True, stable=True)[1][:, :2])


def test_tokens_that_start_off_the_16_bytes():
    """Shifted labels, as a language model's loss reads them."""
    s = inputs(20, 500, "bf16", 2)
    plan = nm.nm_logprobs_plan_init(19, 500, dtype="bf16", ldx=504)
    x = strided(s["x"], 504, 0)[0]
    ids, lp = torch.cat((s["tokens"][:1], s["tokens"])).cuda(), torch.empty(20, device="cuda")
    nm.nm_logprobs(plan, x[:19], ids[1:20], lp[1:])
    want = plain(s, 1.0)[0].gather(1, s["tokens"][:, None])[:19, 0]
    close(lp[1:], want, error(plan, 500, want), "logprob")


def test_captured_and_on_another_stream():
    s = inputs(3, 700001, "bf16", 12)
    plan = nm.nm_logprobs_plan_init(3, 700001, dtype="bf16", top=20, ldx=700016, ldg=700016)
    x = strided(s["x"], 700016, 0)[0]
    assert plan.workspace_bytes > 0
    out = [torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), torch.empty((3, 2), device="cuda"),
           torch.empty((3, 20), device="cuda"), torch.empty((3, 20), dtype=torch.int64, device="cuda"),
           torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")]
    ws, tokens, g, h = plan.empty_workspace(), s["tokens"].cuda(), s["g"].cuda(), s["h"].cuda()

    def step():
        nm.nm_logprobs(plan, x, tokens, out[0], entropy=out[1], stats=out[2], top_logprob=out[3], top_index=out[4], workspace=ws)
        nm.nm_logprobs_backward(plan, x, tokens, out[2], out[5], g_logprob=g, g_entropy=h, entropy=out[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.mul_(-1 if i else 1)
        for t in out:
            t.fill_(7)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, out))
        assert i or all(torch.equal(a, b) for a, b in zip(got, want))


def test_wrapper_and_its_gradients():
    s = inputs(30, 1003, "bf16", 21)
    s["tokens"][::6] = -100
    x, tokens = s["x"].cuda().requires_grad_(), s["tokens"].cuda()          # rows off the 16 bytes: copied
    out = token_logprobs(x, tokens, temperature=0.5, top=4, entropy=True)
    with torch.no_grad():
        again = token_logprobs(x, tokens, temperature=0.5, top=4, entropy=True)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    assert not out.top_logprob.requires_grad and out.logprob.requires_grad
    (-out.logprob.mean() + 0.3 * out.entropy.sum()).backward()
    logp, H, _ = plain(s, 2.0)
    p, hit = logp.exp(), torch.zeros_like(logp).scatter_(1, s["tokens"].clamp_min(0)[:, None], 1.0)
    g = torch.where(s["tokens"] >= 0, -1 / 30, 0.0).double()[:, None]
    want = 2 * (g * (hit - p) - 0.3 * p * (logp + H[:, None]))
    close(x.grad, want, HALF["bf16"] * want.abs() + 2.0 ** -14 * p * (1 + logp.abs()) + 2.0 ** -24 * hit, "gradient")
    x.grad = None
    token_logprobs(x, tokens).logprob[3:9].sum().backward()                 # no entropy; some rows have no gradient
    assert (x.grad[9:] == 0).all() and (x.grad[:3] == 0).all() and (x.grad[6] == 0).all() and (x.grad[5] != 0).any()
    x.grad = None
    token_logprobs(x, tokens, entropy=True).entropy.sum().backward()
    assert x.grad.isfinite().all() and (x.grad != 0).any()
    a = inputs(6, 500, "i32", 2)
    acc = Rows(a["x"].cuda(), a["row_scale"].cuda(), a["col_scale"].cuda())
    got = token_logprobs(acc, a["tokens"].cuda(), top=3)
    want = plain(a, 1.0)[0].gather(1, a["tokens"][:, None])[:, 0]
    close(got.logprob, want, 2.0 ** -14 * (1 + want.abs()), "logprob")
    assert got.entropy is None


def test_wrapper_refuses():
    x, at = torch.zeros((4, 32), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    scales = torch.ones(4, device="cuda"), torch.ones(32, device="cuda")
    token_logprobs(x, at)
    for args, kw in (((x.double(), at), {}), ((x[0], at), {}), ((x, at.int()), {}), ((x, at[:3]), {}), ((x, at.cpu()), {}),
                     ((x.int(), at), {}), ((Rows(x, *scales), at), {}), ((x, at), dict(temperature=0)), ((x, at), dict(top=33)),
                     ((x, at), dict(temperature=math.nan)), ((x, at), dict(top=-1)), ((x[:, :0], at), {}), ((x, None), {})):
        with pytest.raises((ValueError, nm.NmError)):
            token_logprobs(*args, **kw)
    with pytest.raises(RuntimeError, match="gradient"):
        token_logprobs(Rows(x.int(), scales[0].clone().requires_grad_(), scales[1]), at)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_past_the_caches_give_the_same(dtype):
    """512 MB and more are read past the caches: a row's results do not depend on that."""
    rows, cols = (2048, 131072) if dtype == "bf16" else (1100, 131000)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (2 * torch.randn((rows, cols), generator=g, device="cuda")).to(TORCH[dtype])
    tokens = torch.randint(0, cols, (rows,), generator=g, device="cuda")
    gl, ge = torch.randn(rows, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")
    got = []
    for n in (rows, 1030):
        plan = nm.nm_logprobs_plan_init(n, cols, dtype=dtype, top=7)
        assert plan.workspace_bytes == 0
        out = [torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty((n, 2), device="cuda"),
               torch.empty((n, 7), device="cuda"), torch.empty((n, 7), dtype=torch.int64, device="cuda"), torch.empty_like(x[:n])]
        nm.nm_logprobs(plan, x[:n], tokens[:n], out[0], entropy=out[1], stats=out[2], top_logprob=out[3], top_index=out[4])
        nm.nm_logprobs_backward(plan, x[:n], tokens[:n], out[2], out[5], g_logprob=gl[:n], g_entropy=ge[:n], entropy=out[1])
        got.append(out)
    for a, b in zip(*got):
        assert torch.equal(a[:1030], b)
    logp = torch.log_softmax(x[-3:].double(), 1)
    close(got[0][0][-3:], logp.gather(1, tokens[-3:, None])[:, 0].cpu(), torch.full((3,), 1e-4, dtype=torch.float64), "logprob")
