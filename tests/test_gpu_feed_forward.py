"""The feed-forward block on 4-bit 2:4 weights against 64-bit computations from its own weights.

Bounds, elementwise. The 8-bit codes are off by half a step of their scale, s / 2
(0.505 of it with fp32 errors): a product's error is at most the sum of |w| times
that, and a 16-bit rounding of it (few tokens). The activation's slope is below 1.1,
so its error is at most 1.1 |up| Eg + (|silu| + 1.1 Eg) Eu for errors Eg, Eu of the
halves. fp32 sums of exact products add under 2^-12 of the sums of magnitudes.
Root mean square: a rounding's error is s / sqrt(12); with the largest of a row at
most 6 times its mean square's root, s <= 6 / 127 of that, each of the two
quantisations (the first meets both halves) adds at most 1.4 % and all three 2.4 %,
and the 16-bit roundings 0.4 % each: 4 % in all."""
import pytest
import torch

from structured_sparse_gemm_nm_amd.feed_forward import FEW_TOKENS, CompressedFeedForward, Rows

pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def block(hidden, inner, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    gamma = (1 + 0.2 * torch.randn(hidden, generator=g, device="cuda")).to(dtype)
    gate_up = (torch.randn(2 * inner, hidden, generator=g, device="cuda") / hidden ** 0.5).to(dtype)
    down = (torch.randn(hidden, inner, generator=g, device="cuda") / inner ** 0.5).to(dtype)
    return CompressedFeedForward(gamma, gate_up, down), gate_up, down


def inputs(n, hidden, dtype, seed=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, hidden, generator=g, device="cuda").to(dtype),
            (2 * torch.randn(n, hidden, generator=g, device="cuda")).to(dtype))


def exact(ff, x, r, dtype, few):
    """(y, bound of its error, h) in 64 bits."""
    cpu = lambda t: t.double().cpu()  # noqa: E731
    w1, w2, gamma = cpu(ff.gate_up.dense()), cpu(ff.down.dense()), cpu(ff.gamma)
    h = cpu(x) + (cpu(r) if r is not None else 0)
    v = h / (h.square().mean(1, keepdim=True) + ff.eps).sqrt() * gamma
    half = HALF[dtype] if few else 0.0
    step = v.abs().amax(1, keepdim=True) / 127 * 0.505
    p, size = v @ w1.t(), v.abs() @ w1.abs().t()
    e = step * w1.abs().sum(1) + 2.0 ** -12 * size
    e = e + half * (p.abs() + e)
    gate, up = p.split(ff.inner, 1)
    eg, eu = e.split(ff.inner, 1)
    silu = gate * torch.sigmoid(gate)
    a = silu * up
    ea = 1.1 * up.abs() * eg + (silu.abs() + 1.1 * eg) * eu + 2.0 ** -14 * a.abs()
    step = (a.abs() + ea).amax(1, keepdim=True) / 127 * 0.505
    y, size = a @ w2.t(), a.abs() @ w2.abs().t()
    ey = (ea + step) @ w2.abs().t() + 2.0 ** -12 * size
    return y, ey + half * (y.abs() + ey), h


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,few", [(1, True), (5, True), (48, True), (1, False), (16, False), (49, False), (130, False)])
def test_block(n, few, dtype):
    ff, _, _ = block(256, 688, dtype)
    x, r = inputs(n, 256, dtype)
    y, h = ff(x, r, few=few)
    want, bound, hw = exact(ff, x, r, dtype, few)
    got = y.dense().double().cpu()
    assert (y.row_scale is None) == few
    assert ((got - want).abs() <= bound).all()
    assert ((got - want).norm() / want.norm()) < 0.04
    assert ((h.double().cpu() - hw).abs() <= HALF[dtype] * hw.abs() + 2.0 ** -22 * (x.double().abs() + r.double().abs()).cpu()).all()


def test_the_number_of_tokens_picks_the_product():
    ff, _, _ = block(64, 96, torch.float16)
    for n, few in ((1, True), (FEW_TOKENS, True), (FEW_TOKENS + 1, False)):
        y, _ = ff(*inputs(n, 64, torch.float16))
        assert (y.row_scale is None) == few


@pytest.mark.parametrize("n", [1, 17, 48])
def test_both_products_multiply_by_the_same_integers(n):
    """The gate/up products of the same codes differ by the 16-bit rounding alone."""
    ff, _, _ = block(512, 352, torch.float16)
    codes = torch.randint(-127, 128, (n, 512), dtype=torch.int32).to(torch.int8).cuda()
    scale = torch.rand(n, device="cuda") * 0.05
    few, many = ff.gate_up.product(codes, scale, True), ff.gate_up.product(codes, scale, False)
    want = many.values.double() * scale.double()[:, None] * ff.gate_up.scale.double()
    size = codes.double().abs() @ ff.gate_up.dense().double().abs().t() * scale.double()[:, None]
    # fp32: one step a tile of k and a few for the joining of sums and the scales
    assert ((few.values.double() - want).abs() <= HALF[torch.float16] * want.abs() + 32 * 2.0 ** -24 * size + 2.0 ** -25).all()


def test_blocks_chain_on_accumulators():
    """A prompt through two blocks: the second's norm reads the first's accumulators and residual."""
    a, _, _ = block(128, 256, torch.bfloat16, 3)
    b, _, _ = block(128, 256, torch.bfloat16, 4)
    x, r = inputs(64, 128, torch.bfloat16)
    y, h = a(x, r, few=False)
    assert isinstance(y, Rows) and y.values.dtype == torch.int32
    z, h2 = b(y, h, few=False)
    y16 = y.dense().to(torch.bfloat16)
    u = y.dense().double() + h.double()
    assert ((h2.double() - u).abs() <= HALF[torch.bfloat16] * u.abs() + 2.0 ** -22 * (u.abs() + h.double().abs())).all()
    want, _, _ = exact(b, y.dense(), h, torch.bfloat16, False)
    assert ((z.dense().double().cpu() - want).norm() / want.norm()) < 0.04
    z16, _ = b(y16, h, few=False)
    assert ((z16.dense() - z.dense()).norm() / z.dense().norm()) < 0.04


def test_weights_are_the_largest_two_of_four_in_sixteen_steps():
    ff, gate_up, down = block(64, 48, torch.float16)
    for w, orig in ((ff.gate_up, gate_up), (ff.down, down)):
        d, o = w.dense(), orig.float()
        four = o.abs().reshape(o.shape[0], -1, 4)
        two = four.sort(dim=2, descending=True, stable=True).indices[:, :, :2]          # equal magnitudes: the first
        kept = torch.zeros_like(four, dtype=torch.bool).scatter_(2, two, True).reshape(o.shape)
        assert (d[~kept] == 0).all()
        # a step is the scale; the scale's own 16-bit rounding moves the largest by 8 half steps of it
        assert ((d - o).abs()[kept] <= (0.5 * w.scale[:, None] + 2.0 ** -10 * o.abs()).expand_as(o)[kept]).all()


@pytest.mark.parametrize("n", [3, 64, 128])
def test_captured_calls_repeat(n):
    ff, _, _ = block(128, 256, torch.float16)
    x, r = inputs(n, 128, torch.float16)
    first, h = ff(x, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, hh = ff(x, r)
    for _ in range(4):
        y.values.zero_(), hh.zero_()
        graph.replay()
        again, _ = ff(x, r)
        torch.cuda.synchronize()
        assert torch.equal(y.values, first.values) and torch.equal(hh, h) and torch.equal(again.values, first.values)


def test_refusals():
    gamma, gate_up, down = (torch.zeros(s, dtype=torch.float16, device="cuda") for s in ((32,), (64, 32), (32, 32)))
    for bad in ((gamma.cpu(), gate_up, down), (gamma, gate_up.float(), down), (gamma, gate_up.bfloat16(), down),
                (gamma, gate_up[:60], down), (gamma[:24], gate_up, down), (gamma, gate_up, down.t()[:, :16]),
                (gamma[None], gate_up, down), (gamma, gate_up, down.cpu())):
        with pytest.raises(ValueError):
            CompressedFeedForward(*bad)
    with pytest.raises(ValueError):
        CompressedFeedForward(gamma[:24], torch.zeros((64, 24), dtype=torch.float16, device="cuda"),
                              torch.zeros((24, 32), dtype=torch.float16, device="cuda"))
    ff = CompressedFeedForward(gamma, gate_up, down)
    x = torch.zeros((4, 32), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        ff(x.bfloat16())
    with pytest.raises(ValueError):
        ff(x, residual=x[:2])
