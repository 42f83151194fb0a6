"""Low-rank adapters on the GPU against plain 64-bit computations.

Tolerances. HALF is half a step of the 16-bit type, fp32 steps are 2^-24; the matrix unit may cut instead of round, 2^-23.

- t = A x: k / 32 instructions in a chain at most, 32 products in each, 16 parts: (k / 32 + 64) 2^-23 of sum |A| |x|.
- t as two parts, each off by HALF of what it rounds: HALF^2 of |t|, of the token's largest |t| where f16 is scaled to it.
- B t: up to 8 instructions of 32 products: 48 of 2^-23 of sum |B| |t|.
- the factor takes 3 steps, the accumulator's value 3, the sum 1: 8 steps of what meets there."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from structured_sparse_gemm_nm_amd.adapters import Adapters
from structured_sparse_gemm_nm_amd.feed_forward import Rows
from tests.test_gpu_feed_forward import block, inputs as block_inputs
from tests.test_gpu_layer_ops import HALF, TINY, TORCH, Out, close, gen, strided, up16

pytestmark = pytest.mark.gpu


def inputs(n, k, m, r, count, dtype, x="16", base="16", seed=1, mix="scattered"):
    g, dt = gen(seed), TORCH[dtype]
    s = {"dtype": dtype, "row_scale": None, "col_scale": None, "x_scale": None}
    v = torch.randn(n, k, generator=g)
    if x == "i8":
        s["x_scale"] = v.abs().amax(1).clamp_min(1e-3) / 127
        s["x"] = (v / s["x_scale"][:, None]).round().to(torch.int8)
    else:
        s["x"] = v.to(dt)
    s["a"] = (torch.randn(count * r, k, generator=g) / k ** 0.5).to(dt)
    s["b"] = (0.3 * torch.randn(count * m, r, generator=g)).to(dt)
    s["scale"] = 0.5 + torch.rand(count, generator=g)
    s["index"] = torch.randint(-1, count, (n,), generator=g)
    if mix == "runs":
        s["index"] = s["index"][:max(1, n // 37)].repeat_interleave(37)[:n] if n > 37 else s["index"]
        s["index"] = torch.cat((s["index"], s["index"].new_full((n - s["index"].numel(),), 0)))
    if base == "i32":
        s["base"] = (torch.randn(n, m, generator=g) * 1e5).round().to(torch.int32)
        s["row_scale"], s["col_scale"] = 0.02 + 0.02 * torch.rand(n, generator=g), 2e-4 + 3e-4 * torch.rand(m, generator=g)
    else:
        s["base"] = torch.randn(n, m, generator=g).to(dt)
    return s


def plain(s, r):
    """y and the tolerance of each of its values."""
    n, k = s["x"].shape
    m, dtype = s["base"].shape[1], s["dtype"]
    x, base = s["x"].double(), s["base"].double()
    if s["row_scale"] is not None:
        base = base * s["row_scale"].double()[:, None] * s["col_scale"].double()
    at = s["index"].clamp_min(0)
    y, tol = base.clone(), 2.0 ** -22 * base.abs()
    for a in sorted(set(s["index"].tolist()) - {-1}):
        mine = s["index"] == a
        A, B = s["a"][a * r:(a + 1) * r].double(), s["b"][a * m:(a + 1) * m].double()
        f = s["scale"][a].double() * (s["x_scale"][mine].double() if s["x_scale"] is not None else torch.ones(int(mine.sum())).double())
        t, size = x[mine] @ A.t(), x[mine].abs() @ A.t().abs()
        part = HALF[dtype] ** 2 * (t.abs().amax(1, keepdim=True).expand_as(t) if dtype == "f16" else t.abs())
        dt = (k / 32 + 64) * 2.0 ** -23 * size + 2 * part
        y[mine] += f[:, None] * (t @ B.t())
        tol[mine] += f[:, None] * (dt @ B.t().abs() + (48 * 2.0 ** -23 + 2.0 ** -21) * (t.abs() @ B.t().abs()))
    assert at.max() * r < s["a"].shape[0]
    return y, tol * (1 + HALF[dtype]) + HALF[dtype] * y.abs() + TINY[dtype]


def cuda(t):
    return None if t is None else t.cuda()


def run(s, r, pad=0, in_place=False, index=None):
    n, k = s["x"].shape
    m, count = s["base"].shape[1], s["scale"].numel()
    x, _ = strided(s["x"], up16(k) + pad, 77)
    a, _ = strided(s["a"], up16(k), 77)
    base, _ = strided(s["base"], up16(m) + pad, 77)
    plan = nm.nm_lora_plan_init(m, n, k, r, count, dtype=s["dtype"], x_dtype="i8" if s["x_scale"] is not None else None,
                                base_dtype="i32" if s["row_scale"] is not None else None, ldx=up16(k) + pad, lda=up16(k),
                                ldc=up16(m) + pad, ldy=up16(m) + pad)
    out = Out(n, m, up16(m) + pad, TORCH[s["dtype"]])
    y = base if in_place else out.t
    work = torch.full((plan.workspace_bytes + 64,), 255, dtype=torch.uint8, device="cuda")
    nm.nm_lora(plan, x, a, s["b"].cuda(), s["scale"].cuda(), (s["index"] if index is None else index).cuda(), base, y,
               x_scale=cuda(s["x_scale"]), row_scale=cuda(s["row_scale"]), col_scale=cuda(s["col_scale"]),
               workspace=work[:plan.workspace_bytes])
    torch.cuda.synchronize()
    out.check()
    assert (work[plan.workspace_bytes:] == 255).all()
    return y


def check(s, r, **kw):
    y = run(s, r, **kw)
    want, tol = plain(s, r)
    close(y, want, tol, "y")
    return y


SHAPES = [  # n, k, m, rank, adapters, mix
    (1, 64, 64, 8, 1, "scattered"), (1, 4096, 1000, 16, 5, "scattered"), (3, 17, 9, 8, 2, "scattered"), (2, 16, 8, 128, 3, "scattered"), (20, 47, 31, 16, 4, "scattered"),
    (16, 1000, 513, 24, 9, "scattered"), (17, 333, 300, 32, 40, "scattered"), (37, 2000, 777, 64, 24, "scattered"),
    (64, 136, 256, 40, 64, "scattered"), (65, 129, 65, 72, 3, "scattered"), (200, 520, 260, 128, 7, "scattered"),
    (130, 4100, 96, 16, 30, "scattered"), (300, 1024, 512, 16, 4, "runs"), (1000, 700, 130, 48, 6, "runs"), (33, 11008, 320, 96, 1, "runs"),
]


@pytest.mark.parametrize("x", ["16", "i8"])
@pytest.mark.parametrize("base", ["16", "i32"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,k,m,r,count,mix", SHAPES)
def test_product(n, k, m, r, count, mix, dtype, base, x):
    check(inputs(n, k, m, r, count, dtype, x, base, seed=n + k, mix=mix), r, pad=16 * (n % 2))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [5, 100])
def test_in_place_and_tokens_without_an_adapter(n, dtype):
    s = inputs(n, 320, 200, 16, 6, dtype)
    s["index"][::3] = -1 - torch.arange(len(s["index"][::3])) * (1 << 33)
    named = s["index"].clone()
    s["index"] = s["index"].clamp_min(-1)
    y = check(s, 16)
    assert torch.equal(run(s, 16, in_place=True, index=named), y)
    none = s["index"] < 0
    assert torch.equal(y.cpu()[none], s["base"][none])


@pytest.mark.parametrize("base", ["16", "i32"])
@pytest.mark.parametrize("n", [4, 90])
def test_an_adapter_that_does_not_exist_is_nan(n, base):
    s = inputs(n, 320, 200, 16, 6, "f16", base=base)
    y, far = run(s, 16), s["index"].clone()
    far[1], far[n - 1] = 6, 1 << 40
    z, hit = run(s, 16, index=far), torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[[1, n - 1]] = True
    assert z[hit].isnan().all() and torch.equal(z[~hit], y[~hit])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [6, 70])
def test_what_is_not_finite_stays_with_its_token_and_adapter(n, dtype):
    s = inputs(n, 200, 300, 16, 4, dtype)
    s["index"] = torch.arange(n) % 4
    y = run(s, 16)
    s["x"][2, 7], s["x"][1, 3] = float("nan"), float("inf")
    s["a"][3 * 16 + 5, 9], s["b"][0 * 300 + 11, 2] = float("nan"), float("inf")
    z = run(s, 16)
    assert z[2].isnan().all() and not z[1].isfinite().any()
    row = torch.arange(n) % 4
    assert z[row == 3].isnan().all()
    zero = row == 0
    assert not z[zero][:, 11].isfinite().any()
    z[zero, 11] = y[zero, 11]
    rest = (row == 0) | (row == 1) | (row == 2)
    rest[[1, 2]] = False
    assert torch.equal(z[rest], y[rest])


@pytest.mark.parametrize("x,k,up", [("16", 256, 1.0), ("16", 256, 2.0 ** -12), ("16", 4096, 2.0 ** 9), ("i8", 4096, 1.0)])
def test_f16_inner_products_beyond_f16(x, k, up):
    """t passes 65504, or lies under the smallest normal value; the factor brings y back."""
    s = inputs(9, k, 64, 16, 3, "f16", x=x)
    s["a"] = (s["a"].float() * up * (60 if x == "i8" else 1)).clamp(-60000, 60000).half()
    if up > 1:
        s["x"] = (s["x"].float() * 500).half()
    s["scale"] /= up * (500 if up > 1 else 1)
    check(s, 16)
    s["x"] = torch.zeros_like(s["x"])
    check(s, 16)


@pytest.mark.parametrize("n,k,m,r,count,mix", [
    (256, 130, 65, 8, 32, "scattered"), (300, 300, 130, 16, 64, "scattered"), (2048, 64, 40, 40, 4, "scattered"),
    (2047, 100, 72, 16, 5, "runs"), (4096, 32, 33, 8, 9, "scattered"), (4097, 32, 33, 24, 9, "scattered"), (9000, 48, 24, 8, 200, "runs"),
    (700, 16, 8, 8, 9000, "scattered")])
@pytest.mark.parametrize("dtype,x,base", [("f16", "i8", "i32"), ("bf16", "16", "16")])
def test_tokens_sorted_by_their_adapters(n, k, m, r, count, mix, dtype, x, base):
    s = inputs(n, k, m, r, count, dtype, x, base, seed=n, mix=mix)
    if count == 9000:                     # adapters that share a bin of the sort
        s["index"] = torch.where(s["index"] < 0, s["index"], s["index"] % 3 * 4096 + 5)
        s["index"][s["index"] >= count] = 4101
    y = check(s, r)
    assert torch.equal(run(s, r), y)
    named, far = s["index"].clone(), torch.arange(n) % 11 == 3
    named[far] = count + torch.arange(int(far.sum())) * (1 << 40)
    named[~far & (s["index"] < 0)] = -(1 << 50)
    z = run(s, r, index=named)
    assert z[far.cuda()].isnan().all() and torch.equal(z[~far.cuda()], y[~far.cuda()])


@pytest.mark.parametrize("n", [150, 1700])
def test_a_token_does_not_depend_on_the_others(n):
    s = inputs(n, 700, 300, 32, 5, "bf16")
    y = run(s, 32)
    order = torch.randperm(n, generator=gen(3))
    for name in ("x", "index", "base"):
        s[name] = s[name][order]
    assert torch.equal(run(s, 32), y[order.cuda()])
    s["index"][n // 2:] = -1              # the others' adapters leave
    assert torch.equal(run(s, 32)[:n // 2], y[order.cuda()][:n // 2])


def test_nothing_to_do():
    n, m = 0, 64
    plan = nm.nm_lora_plan_init(m, n, 64, 16, 2)
    x, a = torch.zeros((n, 64), dtype=torch.float16, device="cuda"), torch.zeros((32, 64), dtype=torch.float16, device="cuda")
    y = torch.zeros((n, m), dtype=torch.float16, device="cuda")
    nm.nm_lora(plan, x, a, torch.zeros((2 * m, 16), dtype=torch.float16, device="cuda"), torch.ones(2, device="cuda"),
               torch.zeros(n, dtype=torch.int64, device="cuda"), y, y, workspace=plan.empty_workspace())
    torch.cuda.synchronize()


def test_captured_and_on_another_stream():
    s = inputs(40, 2048, 600, 16, 8, "bf16", x="i8", base="i32")
    plan = nm.nm_lora_plan_init(600, 40, 2048, 16, 8, dtype="bf16", x_dtype="i8", base_dtype="i32")
    t = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    y, ws = torch.empty((40, 600), dtype=torch.bfloat16, device="cuda"), plan.empty_workspace()

    def step():
        nm.nm_lora(plan, t["x"], t["a"], t["b"], t["scale"], t["index"], t["base"], y, x_scale=t["x_scale"],
                   row_scale=t["row_scale"], col_scale=t["col_scale"], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want, tol = plain(s, 16)
    close(y, want, tol, "y")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        t["index"].copy_((t["index"] + 1) % 8 - 1)             # other requests, the same graph
        t["x"].neg_()
        y.fill_(7)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y)


def adapters(count, in_f, out_f, rank, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = (torch.randn((count, rank, in_f), generator=g, device="cuda") / in_f ** 0.5).to(dtype)
    b = (0.3 * torch.randn((count, out_f, rank), generator=g, device="cuda")).to(dtype)
    return Adapters(a, b, 0.5 + torch.rand(count, generator=g, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_wrapper(dtype):
    ad = adapters(5, 100, 60, 12, dtype, 3)             # a rank and widths that are padded
    x, base = torch.randn((9, 100), device="cuda").to(dtype), torch.randn((9, 60), device="cuda").to(dtype)
    index = torch.tensor([0, -1, 4, 4, 2, 1, -7, 3, 0], device="cuda")
    y = ad.add(x, index, base)
    want = base.double() + torch.einsum("nmk,nk->nm", ad.dense(index).double(), x.double())
    assert y.dtype is dtype and (y.double() - want).abs().max() < 0.05
    assert torch.equal(y[1], base[1]) and torch.equal(y[6], base[6])
    with pytest.raises(RuntimeError, match="backward"):
        ad.add(x.clone().requires_grad_(), index, base)
    with pytest.raises(RuntimeError, match="backward"):
        ad.add(x, index, base, out=torch.empty((9, 64), dtype=dtype, device="cuda", requires_grad=True)[:, :60])
    for bad in (dict(x=x.float()), dict(x=x[:, :50]), dict(index=index.int()), dict(index=index[:3]), dict(base=base[:, :30]),
                dict(base=base.float()), dict(x=x.cpu()), dict(base=Rows(base, index.float(), None)), dict(x=x[0])):
        with pytest.raises((ValueError, nm.NmError)):
            ad.add(**dict(dict(x=x, index=index, base=base), **bad))
    a, b = ad.a.reshape(5, 16, -1), ad.b.reshape(5, 60, 16)
    for args in ((a, b.float(), ad.scale), (a, b[:4], ad.scale), (a.cpu(), b, ad.scale), (a, b, ad.scale.half()), (a[0], b, ad.scale),
                 (a, b, ad.scale[:3]), (a.repeat(1, 9, 1), b.repeat(1, 1, 9), ad.scale)):
        with pytest.raises(ValueError):
            Adapters(*args)


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_feed_forward_block_with_adapters(dtype, few):
    hidden, inner, n = 64, 96, 21
    ff, _, _ = block(hidden, inner, dtype)
    x, r = block_inputs(n, hidden, dtype)
    index = (torch.arange(n, device="cuda") * 5) % 4 - 1
    up, down = adapters(3, hidden, 2 * inner, 8, dtype, 1), adapters(3, inner, hidden, 16, dtype, 2)
    plain_y, plain_h = ff(x, r, few=few)
    same, h = ff(x, r, few=few, adapters=(index, None, None))
    assert torch.equal(same.values, plain_y.values) and torch.equal(h, plain_h)
    none, _ = ff(x, r, few=few, adapters=(torch.full_like(index, -1), up, down))
    close(none.dense(), plain_y.dense().double().cpu(), 0.02 * (1 + plain_y.dense().double().cpu().abs()), "without an adapter")
    y, h = ff(x, r, few=few, adapters=(index, up, down))
    assert torch.equal(h, plain_h) and y.values.dtype is dtype
    # the block in fp64 on the weights that it multiplies by; 8-bit activations leave a few hundredths
    u = (x.double() + r.double())
    norm = u / (u.square().mean(1, keepdim=True) + ff.eps).sqrt() * ff.gamma.double()
    both = norm @ ff.gate_up.dense().double().t().contiguous() + torch.einsum("nmk,nk->nm", up.dense(index).double(), norm)
    act = both[:, :inner] * torch.sigmoid(both[:, :inner]) * both[:, inner:]
    want = act @ ff.down.dense().double().t().contiguous() + torch.einsum("nmk,nk->nm", down.dense(index).double(), act)
    err = (y.dense().double() - want).abs().amax() / want.abs().amax()
    assert err < 0.05, err
    with pytest.raises(ValueError, match="features"):
        ff(x, r, few=few, adapters=(index, down, up))
