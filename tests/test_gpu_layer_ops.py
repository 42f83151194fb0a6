"""The operators around the product on the GPU, against plain 64-bit computations.

Tolerances. A rounding to a type is off by at most half a step, HALF[type]
relative (f16: 2^-11, bf16: 2^-8; results under the smallest normal f16 by half
of its smallest step, 2^-25). fp32 steps are counted below by 2^-24 each:

- row operators: an accumulator's value takes 3 (its conversion and two
  products), absolute to its size where the residual is added; the sum of
  squares at most 224 in a chain (160 columns a thread for 40000 columns and a
  wave's and the block's sums), half of that after the square root, and under
  16 for the rest: 2^-17 = 128 steps. The gated product's exponential has an
  argument off by at most 4 steps of its size (<= 90 where it is not flushed):
  360 steps, and a few for itself: 2^-15 = 512 steps.
- 8-bit codes: half a step of the scale, and the 127 steps of a code times the
  relative error above: 0.5 + 127 * 2^-15 < 0.505 of the scale.
- the 4-bit product: products are exact in fp32 (4 + 11 bits), a group's sum
  takes at most 128 additions, then one step per scale application (2 per tile
  of 128: the scale's product and the sum, fused, and at most 4 applications a
  tile) and 16 for the waves' sums; the matrix unit may cut instead of round:
  2^-23 each, relative to the sum of magnitudes. Sums of 8-bit x are exact in a
  group."""
import math

import pytest
import torch

import structured_sparse_gemm_nm_amd as nm

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}
CODE = 0.505


def up16(n):
    return (n + 15) // 16 * 16


def strided(t, ld, fill):
    """t in rows ld apart on the GPU; what lies between and past the rows is `fill`."""
    raw = torch.full((t.shape[0] * ld + 64,), fill, dtype=t.dtype, device="cuda")
    v = raw[:t.shape[0] * ld].view(t.shape[0], ld)[:, :t.shape[1]]
    v.copy_(t)
    return v, raw


class Out:
    """An output in rows ld apart whose surroundings must stay as they were."""

    def __init__(self, rows, cols, ld, dtype):
        self.fill = 93
        self.t, self.raw = strided(torch.full((rows, cols), self.fill, dtype=dtype), ld, self.fill)
        self.rows, self.cols, self.ld = rows, cols, ld

    def check(self):
        body = self.raw[:self.rows * self.ld].view(self.rows, self.ld)[:, self.cols:]
        assert (body == self.fill).all() and (self.raw[self.rows * self.ld:] == self.fill).all(), "write outside the rows"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, want, tol, what):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %g of tolerance" % (
        what, int(bad.sum()), bad.numel(), float((err / tol.clamp_min(1e-300)).max()))


# ------------------------------------------------------------------ row operators

def row_inputs(op, rows, cols, dtype, x, residual, seed):
    g, width = gen(seed), cols * (2 if op == "swiglu" else 1)
    s = {"row_scale": None, "col_scale": None, "residual": None}
    if x == "i32":
        s["x"] = (torch.randn(rows, width, generator=g) * 1e5).round().to(torch.int32)
        s["row_scale"] = 0.02 + 0.02 * torch.rand(rows, generator=g)
        s["col_scale"] = 2e-4 + 3e-4 * torch.rand(width, generator=g)
    else:
        s["x"] = (2 * torch.randn(rows, width, generator=g)).to(TORCH[dtype])
    if op == "rmsnorm":
        s["gamma"] = (1 + 0.2 * torch.randn(cols, generator=g)).to(TORCH[dtype])
        if residual:
            s["residual"] = (3 * torch.randn(rows, cols, generator=g)).to(TORCH[dtype])
    return s


def row_exact(op, s, cols, eps):
    """(v * f, u) in 64 bits, and the magnitude that fp32 errors are relative to."""
    x = s["x"].double()
    if s["row_scale"] is not None:
        x = x * s["row_scale"].double()[:, None] * s["col_scale"].double()
    if op == "swiglu":
        gate, up = x[:, :cols], x[:, cols:]
        v = gate * torch.sigmoid(gate) * up
        return v, None, v.abs()
    size = x.abs()
    if s["residual"] is not None:
        x, size = x + s["residual"].double(), size + s["residual"].double().abs()
    f = 1 / (x.square().mean(1, keepdim=True) + eps).sqrt()
    gamma = s["gamma"].double()
    return x * f * gamma, x, size * f * gamma.abs()


def row_run(op, s, rows, cols, dtype, y, pad, eps, want_h, in_place=False):
    ld = up16(cols) + pad
    width = s["x"].shape[1]
    x, _ = strided(s["x"], up16(width) + pad, 77)
    plan = nm.nm_rows_plan_init(rows, cols, op=op, dtype=dtype, x_dtype="i32" if s["row_scale"] is not None else None,
                                y_dtype=y, ldx=up16(width) + pad, ldr=ld, ldh=ld, ldy=ld, eps=eps)
    out = Out(rows, cols, ld, torch.int8 if y == "i8" else TORCH[dtype])
    scale = torch.full((rows + 8,), 93.0, device="cuda") if y == "i8" else None
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    kw = dict(y_scale=None if scale is None else scale[:rows], row_scale=cuda(s["row_scale"]), col_scale=cuda(s["col_scale"]))
    h = None
    if op == "rmsnorm":
        res = None if s["residual"] is None else strided(s["residual"], ld, 77)[0]
        if want_h:
            h = Out(rows, cols, ld, TORCH[dtype])
            ht = h.t
            if in_place:
                h = None
                ht = res
        nm.nm_rmsnorm(plan, x, s["gamma"].cuda(), out.t, residual=res, h=ht if want_h else None, **kw)
    else:
        nm.nm_swiglu(plan, x, out.t, **kw)
    torch.cuda.synchronize()
    out.check()
    if h is not None:
        h.check()
    if scale is not None:
        assert (scale[rows:] == 93).all()
    return out.t, None if scale is None else scale[:rows], (ht if op == "rmsnorm" and want_h else None)


def row_check(op, s, rows, cols, dtype, y, pad=0, eps=1e-6, want_h=True, in_place=False):
    got, scale, h = row_run(op, s, rows, cols, dtype, y, pad, eps, want_h, in_place)
    v, u, size = row_exact(op, s, cols, eps)
    rel = 2.0 ** -17 if op == "rmsnorm" else 2.0 ** -15
    if y == "i8":
        top = v.abs().amax(1)
        want = top / 127
        # the largest magnitude is off by its own error, absolute to the sizes that met in it
        close(scale, want, rel * size.amax(1) / 127 + 1e-44, "y_scale")
        codes = got.double().cpu()
        assert codes.abs().max() <= 127
        assert (codes.abs().amax(1)[top > 0] == 127).all()
        close(codes * scale.double().cpu()[:, None], v, (CODE * want)[:, None] + rel * size, "y")
    else:
        close(got, v, HALF[dtype] * v.abs() + rel * size * (1 + HALF[dtype]) + TINY[dtype], "y")
    if h is not None:
        hs = s["x"].double().abs() if s["row_scale"] is None else u.abs() + (0 if s["residual"] is None else s["residual"].double().abs())
        close(h, u, HALF[dtype] * u.abs() + 4 * 2.0 ** -24 * (hs + u.abs()) * 2 + TINY[dtype], "h")


COLS = [1, 2, 7, 8, 9, 31, 64, 65, 127, 200, 511, 512, 513, 1000, 1023, 1024, 2047, 2048, 2056, 4096, 5120, 8191, 8192,
        11008, 16384, 16385, 40000]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("op", ["rmsnorm", "swiglu"])
def test_rows_every_width(op, cols):
    for i, (x, y) in enumerate([("16", None), ("16", "i8"), ("i32", None), ("i32", "i8")]):
        dtype = ("f16", "bf16")[(i + cols) % 2]
        for rows in (1, 3):
            s = row_inputs(op, rows, cols, dtype, x, residual=(i + rows) % 2 == 0, seed=1000 + cols + i)
            row_check(op, s, rows, cols, dtype, y, pad=16 * (i % 2), want_h=rows == 3 or i % 2 == 0)


@pytest.mark.parametrize("rows", [2, 5, 64, 255, 1025, 5000])
@pytest.mark.parametrize("op", ["rmsnorm", "swiglu"])
def test_rows_many(op, rows):
    for i, cols in enumerate((40, 264, 513)):
        for x, y in (("16", "i8"), ("i32", None)):
            dtype = ("f16", "bf16")[i % 2]
            row_check(op, row_inputs(op, rows, cols, dtype, x, True, 7 + i), rows, cols, dtype, y, pad=32)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("cols", [96, 4096, 40000])
def test_norm_writes_the_residual_in_place(dtype, cols):
    s = row_inputs("rmsnorm", 4, cols, dtype, "16", True, 5)
    row_check("rmsnorm", s, 4, cols, dtype, "i8", in_place=True)
    s = row_inputs("rmsnorm", 4, cols, dtype, "i32", True, 6)
    row_check("rmsnorm", s, 4, cols, dtype, None, in_place=True)


@pytest.mark.parametrize("y", [None, "i8"])
@pytest.mark.parametrize("cols", [40, 4096, 20000])
def test_norm_of_zero_rows(cols, y):
    s = row_inputs("rmsnorm", 3, cols, "f16", "16", False, 8)
    s["x"][1] = 0
    got, scale, _ = row_run("rmsnorm", s, 3, cols, "f16", y, 0, 1e-6, False)
    assert (got[1] == 0).all()
    if y:
        assert scale[1] == 0 and scale[0] > 0 and scale[2] > 0
    # eps = 0 on a row of zeros: 0 / 0, as the formula says; its codes are still zero
    got, scale, _ = row_run("rmsnorm", s, 3, cols, "f16", y, 0, 0.0, False)
    if y:
        assert torch.isnan(scale[1]) and (got[1] == 0).all()
    else:
        assert torch.isnan(got[1]).all()


def test_eps_decides_small_rows():
    s = row_inputs("rmsnorm", 2, 512, "bf16", "16", False, 9)
    s["x"] = (s["x"].float() * 1e-4).to(torch.bfloat16)
    for eps in (0.0, 1e-12, 1e-6, 1.0):
        row_check("rmsnorm", s, 2, 512, "bf16", None, eps=eps)


@pytest.mark.parametrize("op", ["rmsnorm", "swiglu"])
@pytest.mark.parametrize("cols", [72, 3000, 17000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_rows_keep_infinities_and_nan_to_their_row(op, cols, bad):
    clean = row_inputs(op, 3, cols, "bf16", "16", False, 10)
    s = dict(clean, x=clean["x"].clone())
    s["x"][1, cols // 2] = bad
    for y in (None, "i8"):
        a, sa, _ = row_run(op, clean, 3, cols, "bf16", y, 0, 1e-6, False)
        b, sb, _ = row_run(op, s, 3, cols, "bf16", y, 0, 1e-6, False)
        for r in (0, 2):
            assert torch.equal(a[r], b[r]) and (y is None or sa[r] == sb[r])
        if y is None:
            value = b[1].float().cpu()
        else:
            assert not torch.isfinite(sb[1]) and int(b[1].abs().max()) <= 127
            value = b[1].float().cpu() * sb[1].cpu()
        assert not torch.isfinite(value[cols // 2]) or bad == float("-inf") or op == "rmsnorm" and y is None
        # the plain formula's NaNs are the 16-bit output's
        if y is None:
            v, _, _ = row_exact(op, s, cols, 1e-6)
            assert torch.equal(torch.isnan(value), torch.isnan(v[1]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_swiglu_over_the_range_of_the_gate(dtype):
    gate = torch.linspace(-120, 120, 2400).to(TORCH[dtype])[None]
    s = dict(x=torch.cat((gate, torch.ones_like(gate)), 1), row_scale=None, col_scale=None)
    row_check("swiglu", s, 1, 2400, dtype, None)
    top = torch.finfo(TORCH[dtype]).max
    edge = torch.tensor([[0.0, -0.0, top, -top, float("inf"), 1e-7, -1e-7, 88.0]]).to(TORCH[dtype])
    s["x"] = torch.cat((edge, torch.ones_like(edge)), 1)
    got, _, _ = row_run("swiglu", s, 1, 8, dtype, None, 0, 0.0, False)
    e = edge.double()
    want = (e * torch.sigmoid(e)).to(TORCH[dtype])
    assert torch.equal(got[0, [0, 1, 2, 3, 4, 7]].cpu(), want[0, [0, 1, 2, 3, 4, 7]])


def test_codes_round_half_to_even_and_reach_127():
    v = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 3.0]]).half()
    s = dict(x=v, residual=None, gamma=torch.ones(8).half(), row_scale=None, col_scale=None)
    got, scale, _ = row_run("rmsnorm", s, 1, 8, "f16", "i8", 0, 0.0, False)
    assert got[0].tolist() == [127, 0, 2, 2, 0, -2, -126, 3]
    f = 1 / math.sqrt(float(v.double().square().mean()))
    assert abs(float(scale[0]) / f - 1) < 2.0 ** -20


@pytest.mark.parametrize("op", ["rmsnorm", "swiglu"])
def test_rows_far_apart(op):
    """Offsets past 2^31 elements and 2^32 bytes."""
    ld, cols = (1 << 30) + 16, 520
    width = cols * (2 if op == "swiglu" else 1)
    s = row_inputs(op, 3, cols, "f16", "16", True, 11)
    raw = torch.empty(2 * ld + width, dtype=torch.float16, device="cuda")
    x = raw.as_strided((3, width), (ld, 1))
    x.copy_(s["x"])
    yraw = torch.empty(2 * ld + cols, dtype=torch.float16, device="cuda")
    y = yraw.as_strided((3, cols), (ld, 1))
    plan = nm.nm_rows_plan_init(3, cols, op=op, ldx=ld, ldy=ld, ldr=cols, ldh=cols)
    if op == "rmsnorm":
        nm.nm_rmsnorm(plan, x, s["gamma"].cuda(), y, residual=s["residual"].cuda())
    else:
        nm.nm_swiglu(plan, x, y)
    v, _, size = row_exact(op, s, cols, 1e-6)
    close(y, v, HALF["f16"] * v.abs() + 2.0 ** -15 * size + TINY["f16"], "y")


# ------------------------------------------------------------------ 4-bit product

def w4_inputs(m, n, k, group, dtype, x, sparse, zeros, seed):
    g = gen(seed)
    kept, G = (k // 2 if sparse else k), (1 if group == 0 or k == 0 else -(-k // group))
    s = {"q": torch.randint(0, 16, (m, kept), generator=g, dtype=torch.uint8),
         "scales": (0.004 + 0.012 * torch.rand(m, G, generator=g)).to(TORCH[dtype]),
         "zeros": torch.randint(0, 16, (m, G), generator=g, dtype=torch.uint8) if zeros else None,
         "pairs": None, "x_scale": None}
    if sparse:
        table = torch.tensor([[a, b] for a in range(4) for b in range(a + 1, 4)], dtype=torch.uint8)
        s["pairs"] = table[torch.randint(0, 6, (m, k // 4), generator=g)]          # kept offsets of each four
    v = torch.randn(n, k, generator=g) * (1 + 7 * (torch.rand(1, k, generator=g) < 0.02))
    if x == "i8":
        s["x"] = torch.randint(-127, 128, (n, k), generator=g, dtype=torch.int32).to(torch.int8)
        s["x_scale"] = 0.01 + 0.05 * torch.rand(n, generator=g)
    else:
        s["x"] = v.to(TORCH[dtype])
    return s


def w4_exact(s, k, group):
    """y (n x m) and the sum of magnitudes, in 64 bits."""
    m, kept = s["q"].shape
    per = (group or max(1, k)) // (2 if s["pairs"] is not None else 1)
    z = s["zeros"].double() if s["zeros"] is not None else torch.full(s["scales"].shape, 8.0, dtype=torch.float64)
    w = s["q"].double() - z.repeat_interleave(per, 1)[:, :kept]
    w = w * s["scales"].double().repeat_interleave(per, 1)[:, :kept]
    if s["pairs"] is not None:
        at = (s["pairs"].long() + 4 * torch.arange(k // 4)[None, :, None]).reshape(m, -1)
        w = torch.zeros(m, k, dtype=torch.float64).scatter_(1, at, w)
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double()[:, None]
    return x @ w.t(), x.abs() @ w.abs().t()


def nibbles(q, bytes_a_row):
    m, kept = q.shape
    out = torch.zeros(m, 2 * bytes_a_row, dtype=torch.uint8)
    out[:, :kept] = q
    return out[:, 0::2] | out[:, 1::2] << 4


def w4_plan(s, m, n, k, group, dtype, x, pad=0):
    return nm.nm_w4_plan_init(m, n, k, group=group, dtype=dtype, x_dtype="i8" if x == "i8" else None,
                              sparse=s["pairs"] is not None, zeros=s["zeros"] is not None, ldx=up16(k) + pad + 16 * (k == 0),
                              ldy=up16(m) + pad + 16 * (m == 0))


def w4_pack(plan, s):
    meta = None
    if s["pairs"] is not None:
        nib = (s["pairs"][..., 0] | s["pairs"][..., 1] << 2)
        meta = nibbles(nib, plan.meta_ld).cuda()
    raw = torch.full((plan.packed_bytes + 256,), 93, dtype=torch.uint8, device="cuda")
    packed = raw[:plan.packed_bytes]
    nm.nm_w4_pack(plan, nibbles(s["q"], plan.code_ld).cuda(), s["scales"].cuda(), packed,
                  zeros=None if s["zeros"] is None else s["zeros"].cuda(), meta=meta)
    torch.cuda.synchronize()
    assert (raw[plan.packed_bytes:] == 93).all()
    return packed


def w4_run(s, m, n, k, group, dtype, x, pad=0):
    plan = w4_plan(s, m, n, k, group, dtype, x, pad)
    packed = w4_pack(plan, s)
    xt, _ = strided(s["x"], plan._strides[0], 113 if x == "i8" else float("nan"))   # past k: what must not be read
    out = Out(n, m, plan._strides[1], TORCH[dtype])
    xs = None if s["x_scale"] is None else s["x_scale"].cuda()
    nm.nm_w4_matvec(plan, packed, xt, out.t, x_scale=xs)
    torch.cuda.synchronize()
    out.check()
    return out.t


def w4_tolerance(y, size, k, dtype):
    steps = 128 + 8 * (k // 128 + 1) + 16 + 4
    return HALF[dtype] * y.abs() + (1 + HALF[dtype]) * steps * 2.0 ** -23 * size + TINY[dtype]


def w4_check(m, n, k, group, dtype, x, sparse, zeros, pad=0, seed=0):
    s = w4_inputs(m, n, k, group, dtype, x, sparse, zeros, seed + m + n + k)
    got = w4_run(s, m, n, k, group, dtype, x, pad)
    y, size = w4_exact(s, k, group)
    close(got, y, w4_tolerance(y, size, k, dtype), "y %s" % ((m, n, k, group, dtype, x, sparse, zeros),))


def groups(x, sparse):
    least = 32 * (2 if sparse else 1) * (2 if x == "i8" else 1)
    return [0, least, 2 * least, 3 * least, 4 * least, 512]


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("x", ["16", "i8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_groups_and_tails(dtype, x, sparse, zeros):
    ks = (4, 28, 128, 252, 256, 260, 516, 1032, 2048) if sparse else (1, 7, 31, 32, 127, 128, 129, 257, 1000, 1024, 2048)
    for i, k in enumerate(ks):
        for j, group in enumerate(groups(x, sparse)):
            w4_check((16, 37, 64, 80)[(i + j) % 4], (1, 2, 5, 16)[(i + 2 * j) % 4], k, group, dtype, x, sparse, zeros,
                     pad=16 * (j % 3))


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("x", ["16", "i8"])
@pytest.mark.parametrize("n", [1, 2, 3, 15, 16, 17, 32, 33, 40, 48, 49, 100])
def test_w4_tokens(n, x, sparse):
    for dtype in ("f16", "bf16"):
        w4_check(48, n, 700, 128 if not (sparse and x == "i8") else 256, dtype, x, sparse, n % 2 == 0, pad=16)
        w4_check(33, n, 516, groups(x, sparse)[1], dtype, x, sparse, n % 2 == 1)


@pytest.mark.parametrize("m", [1, 2, 3, 4, 7, 15, 16, 17, 31, 129, 1000, 5000])
def test_w4_rows(m):
    w4_check(m, 3, 384, 128, "f16", "16", False, True)
    w4_check(m, 1, 384, 64, "bf16", "16", False, False, pad=16)
    w4_check(m, 2, 512, 128, "bf16", "i8", True, True)


@pytest.mark.parametrize("k", [4096, 11008, 16388])
def test_w4_long_rows(k):
    for dtype, x, sparse in (("f16", "16", False), ("bf16", "16", True), ("f16", "i8", True), ("bf16", "i8", False)):
        w4_check(48, 4, k, 128, dtype, x, sparse, True)
        w4_check(20, 1, k, 0, dtype, x, sparse, False)


def test_w4_is_exact_where_sums_are():
    """Small integers and scales of 1: every sum is a whole number that f16 holds."""
    for x, sparse, zeros in (("16", False, False), ("16", True, True), ("i8", False, True), ("i8", True, False)):
        group = 256 if sparse and x == "i8" else 128
        s = w4_inputs(40, 5, 260, group, "f16", x, sparse, zeros, 3)
        s["scales"] = torch.ones_like(s["scales"])
        s["x"] = torch.randint(-1, 2, (5, 260), generator=gen(4)).to(s["x"].dtype)
        if x == "i8":
            s["x_scale"] = torch.ones(5)
        got = w4_run(s, 40, 5, 260, group, "f16", x)
        y, _ = w4_exact(s, 260, group)
        assert y.abs().max() < 2048 and torch.equal(got.double().cpu(), y)


def test_w4_every_code_and_zero_point():
    """One weight a row: all 16 codes times all 16 zero points, exactly."""
    for dtype in ("f16", "bf16"):
        for x in ("16", "i8"):
            for at in range(8):          # every nibble of a dword
                k = 64
                s = w4_inputs(256, 1, k, 64, dtype, x, False, True, 1)
                s["scales"] = torch.ones(256, 1).to(TORCH[dtype])
                s["zeros"] = (torch.arange(256) // 16).to(torch.uint8)[:, None]
                s["q"] = s["zeros"].repeat(1, k)
                s["q"][:, at] = (torch.arange(256) % 16).to(torch.uint8)
                s["x"] = torch.ones(1, k).to(s["x"].dtype)
                if x == "i8":
                    s["x_scale"] = torch.ones(1)
                got = w4_run(s, 256, 1, k, 64, dtype, x)[0].double().cpu()
                assert torch.equal(got, (torch.arange(256) % 16 - torch.arange(256) // 16).double()), (dtype, x, at)


def test_w4_tokens_do_not_meet():
    """A token with a NaN and one with an infinity leave the other tokens' results bit for bit."""
    for dtype in ("f16", "bf16"):
        s = w4_inputs(64, 6, 300, 128, dtype, "16", False, True, 2)
        a = w4_run(s, 64, 6, 300, 128, dtype, "16")
        s["x"][1, 17], s["x"][4, 299] = float("nan"), float("inf")
        b = w4_run(s, 64, 6, 300, 128, dtype, "16")
        for j in (0, 2, 3, 5):
            assert torch.equal(a[j], b[j])
        assert torch.isnan(b[1]).all() and not torch.isfinite(b[4]).any()
        # an infinity times a code at its zero point is NaN, any other keeps its sign
        z = s["zeros"][:, 2].long()
        d = s["q"][:, 299].long() - z
        want = torch.where(d == 0, torch.tensor(float("nan")), torch.sign(d.float()) * float("inf"))
        assert torch.equal(torch.nan_to_num(b[4].float().cpu(), nan=0.5, posinf=2, neginf=-2),
                           torch.nan_to_num(want, nan=0.5, posinf=2, neginf=-2))


def test_w4_pruned_columns_do_not_count():
    """2:4: an activation that no kept weight meets may be anything."""
    s = w4_inputs(32, 2, 256, 0, "f16", "16", True, False, 5)
    s["pairs"][:, :, 0], s["pairs"][:, :, 1] = 0, 2
    a = w4_run(s, 32, 2, 256, 0, "f16", "16")
    s["x"][:, 1::2] = float("nan")
    assert torch.equal(a, w4_run(s, 32, 2, 256, 0, "f16", "16"))


@pytest.mark.parametrize("x,sparse", [("16", False), ("i8", True)])
def test_w4_without_columns(x, sparse):
    """k = 0: sums of nothing."""
    s = w4_inputs(20, 3, 0, 0, "f16", x, sparse, False, 6)
    plan = w4_plan(s, 20, 3, 0, 0, "f16", x)
    y = torch.full((3, 32), 7.0, dtype=torch.float16, device="cuda")
    nm.nm_w4_matvec(plan, plan.empty_packed(), s["x"].cuda(), y[:, :20],
                    x_scale=None if s["x_scale"] is None else s["x_scale"].cuda())
    torch.cuda.synchronize()
    assert (y[:, :20] == 0).all() and (y[:, 20:] == 7).all()


def test_w4_reads_the_library_metadata():
    """2:4 weights from nm_prune and nm_compress: the product's offsets are nm_compress's bytes."""
    m, k, n = 64, 512, 4
    a = torch.randn(m, k, generator=gen(12)).half().cuda()
    cp = nm.nm_plan_init(m, n, k, 2, 4, dtype="f16")
    pruned, values, meta = torch.empty_like(a), cp.empty_values(), cp.empty_meta()
    nm.nm_prune(cp, a, pruned)
    nm.nm_compress(cp, pruned, values, meta)
    kept = values[:, :k // 2].double().cpu()
    scales = (kept.abs().amax(1, keepdim=True) / 7).half()
    q = (kept / scales.double()).round().clamp(-8, 7)
    plan = nm.nm_w4_plan_init(m, n, k, group=0, sparse=True)
    assert plan.meta_ld == cp.meta_ld
    packed = plan.empty_packed()
    nm.nm_w4_pack(plan, nibbles((q + 8).to(torch.uint8), plan.code_ld).cuda(), scales.cuda(), packed, meta=meta)
    x = torch.randn(n, k, generator=gen(13)).half()
    y = torch.empty(n, m, dtype=torch.float16, device="cuda")
    nm.nm_w4_matvec(plan, packed, x.cuda(), y)
    w = torch.zeros(m, k, dtype=torch.float64)
    w[pruned.cpu() != 0] = (q * scales.double()).reshape(-1)        # kept values lie in order in each row
    want, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    close(y, want, w4_tolerance(want, size, k, "f16"), "y")


def test_w4_far_apart_tokens_and_large_weights():
    """Token strides past 2^31 elements; packed weights past 2^32 bytes."""
    ld = (1 << 30) + 16
    s = w4_inputs(32, 3, 256, 128, "f16", "16", False, False, 14)
    raw = torch.empty(2 * ld + 256, dtype=torch.float16, device="cuda")
    x = raw.as_strided((3, 256), (ld, 1))
    x.copy_(s["x"])
    yraw = torch.empty(2 * ld + 32, dtype=torch.float16, device="cuda")
    y = yraw.as_strided((3, 32), (ld, 1))
    plan = nm.nm_w4_plan_init(32, 3, 256, group=128, ldx=ld, ldy=ld)
    nm.nm_w4_matvec(plan, w4_pack(plan, s), x, y)
    want, size = w4_exact(s, 256, 128)
    close(y, want, w4_tolerance(want, size, 256, "f16"), "y")
    del raw, yraw, x, y
    m, k, G = 140000, 65536, 512
    codes = torch.randint(0, 256, (m, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((m, G), 0.0078125, dtype=torch.float16, device="cuda")
    plan = nm.nm_w4_plan_init(m, 1, k, group=128, x_dtype="i8")
    packed = plan.empty_packed()
    assert packed.numel() > 1 << 32
    nm.nm_w4_pack(plan, codes, scales, packed)
    x8 = torch.randint(-127, 128, (1, k), dtype=torch.int32).to(torch.int8)
    y = torch.empty(1, m, dtype=torch.float16, device="cuda")
    nm.nm_w4_matvec(plan, packed, x8.cuda(), y, x_scale=torch.full((1,), 2.0 ** -10, device="cuda"))
    rows = torch.tensor([0, 1, 70000, 131072, m - 1])
    c = codes[rows.cuda()].cpu()
    q = torch.stack((c & 15, c >> 4), 2).reshape(5, -1).double() - 8
    want = (x8.double() @ q.t()) * 2.0 ** -17
    close(y[:, rows.cuda()], want, w4_tolerance(want, (x8.double().abs() @ q.abs().t()) * 2.0 ** -17, k, "f16"), "y")


# ------------------------------------------------------------------ all of them

def test_calls_repeat_bit_for_bit_on_other_streams_and_in_graphs():
    """The same bits again, on a side stream and from a captured graph replayed between eager calls."""
    s = row_inputs("rmsnorm", 7, 1000, "bf16", "16", True, 20)
    norm = nm.nm_rows_plan_init(7, 1000, dtype="bf16", y_dtype="i8", ldy=1008)
    x, r, g = s["x"].cuda(), s["residual"].cuda(), s["gamma"].cuda()
    t = w4_inputs(96, 7, 1000, 128, "bf16", "i8", False, True, 21)
    prod = nm.nm_w4_plan_init(96, 7, 1000, group=128, dtype="bf16", x_dtype="i8", zeros=True, ldx=1008)
    packed = w4_pack(prod, t)
    act = nm.nm_rows_plan_init(7, 48, op="swiglu", dtype="bf16", y_dtype="i8")

    def step(o):
        nm.nm_rmsnorm(norm, x, g, o["q"][:, :1000], y_scale=o["qs"], residual=r, h=o["h"])
        nm.nm_w4_matvec(prod, packed, o["q"][:, :1000], o["y"], x_scale=o["qs"])
        nm.nm_swiglu(act, o["y"], o["a"], y_scale=o["as"])

    def outs():
        i8, b16 = dict(dtype=torch.int8, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        return {"q": torch.zeros(7, 1008, **i8), "qs": torch.zeros(7, device="cuda"), "h": torch.zeros(7, 1000, **b16),
                "y": torch.zeros(7, 96, **b16), "a": torch.zeros(7, 48, **i8), "as": torch.zeros(7, device="cuda")}

    first, second, third = outs(), outs(), outs()
    step(first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(second)
    side.synchronize()
    assert all(torch.equal(first[k], second[k]) for k in first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(third)
    for _ in range(4):
        for k in third:
            third[k].zero_()
        graph.replay()
        step(second)
        torch.cuda.synchronize()
        assert all(torch.equal(first[k], third[k]) and torch.equal(first[k], second[k]) for k in first)


def test_operands_on_the_host_or_unlike_the_plan_are_refused():
    x, g = torch.zeros((8, 64), dtype=torch.float16, device="cuda"), torch.zeros(64, dtype=torch.float16, device="cuda")
    plan = nm.nm_rows_plan_init(8, 64)
    with pytest.raises(ValueError, match="gamma"):
        nm.nm_rmsnorm(plan, x, g.cpu(), x.clone())
    with pytest.raises(ValueError, match="y must"):
        nm.nm_rmsnorm(plan, x, g, x.clone().float())
    with pytest.raises(ValueError, match="residual"):
        nm.nm_rmsnorm(plan, x, g, x.clone(), residual=x[:4])
    with pytest.raises(ValueError, match="x must"):
        nm.nm_swiglu(nm.nm_rows_plan_init(8, 64, op="swiglu"), x, x.clone())
    w = nm.nm_w4_plan_init(64, 8, 64, group=64)
    with pytest.raises(ValueError, match="packed"):
        nm.nm_w4_matvec(w, w.empty_packed()[:-1], x, x.clone())
