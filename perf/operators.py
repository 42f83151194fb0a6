"""Cases of the operators that serve a layer with compressed weights.

Three operators, which follow each other in a block whose weights the library
holds in 8 or 4 bits:

- ``rmsnorm``: root-mean-square norm of x + residual, written in 8 bits with one
  scale a token (or in 16 bits). x is 16-bit, or the int32 accumulators of an
  int8 product with a scale for each token and each channel.
- ``swiglu``: silu(gate) * up of the joint gate/up product, in 8 or 16 bits, from
  the same two kinds of input.
- ``w4``: y = x W^T for few tokens, W in 4 bits with a scale (and an optional
  zero point) for each group along k, W dense or 2:4 with the library's
  metadata, x in 16 bits or in 8 bits with one scale a token.

With ``own`` false ``run`` computes them from elementary torch operations, with
``own`` true by the library's entry points. Codes of 8 bits are returned as the
values they stand for, in the layer's 16-bit type.
"""
import math

import torch

own = False

_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a chat, hidden size 4096: the smallest call, all latency
        {"name": "norm_i8_1x4096", "op": "rmsnorm", "rows": 1, "cols": 4096, "dtype": "f16", "x": "16", "y": "i8",
         "residual": True, "pad": 0},
        # a prompt of 8192 tokens before an int8 product
        {"name": "norm_i8_8192x4096", "op": "rmsnorm", "rows": 8192, "cols": 4096, "dtype": "bf16", "x": "16", "y": "i8",
         "residual": True, "pad": 0},
        # the same prompt after an int8 product: its accumulators come in, the next layer's 16-bit input goes out
        {"name": "norm_acc_4096x4096", "op": "rmsnorm", "rows": 4096, "cols": 4096, "dtype": "bf16", "x": "i32", "y": "16",
         "residual": True, "pad": 0},
        # odd width and a row stride of its own: a norm over the heads' joint width, no residual
        {"name": "norm_odd_777x1023", "op": "rmsnorm", "rows": 777, "cols": 1023, "dtype": "f16", "x": "16", "y": "i8",
         "residual": False, "pad": 16},
        # a decode batch of 16 after a 4-bit gate/up product
        {"name": "swiglu_i8_16x11008", "op": "swiglu", "rows": 16, "cols": 11008, "dtype": "f16", "x": "16", "y": "i8",
         "pad": 0},
        # a prompt of 4096 tokens after the int8 2:4 gate/up product
        {"name": "swiglu_acc_4096x11008", "op": "swiglu", "rows": 4096, "cols": 11008, "dtype": "bf16", "x": "i32",
         "y": "i8", "pad": 0},
        # the smallest 4-bit product: one token, a 1024 x 1024 projection
        {"name": "w4_1024x1024_n1", "op": "w4", "m": 1024, "k": 1024, "n": 1, "group": 128, "dtype": "f16", "x": "16",
         "sparse": False, "zeros": False, "pad": 0},
        # one token through a square projection, zero points
        {"name": "w4_4096x4096_n1", "op": "w4", "m": 4096, "k": 4096, "n": 1, "group": 128, "dtype": "bf16", "x": "16",
         "sparse": False, "zeros": True, "pad": 0},
        # a vocabulary-sized head with an odd number of rows, a batch of 5, fine groups
        {"name": "w4_32003x4096_n5", "op": "w4", "m": 32003, "k": 4096, "n": 5, "group": 64, "dtype": "f16", "x": "16",
         "sparse": False, "zeros": False, "pad": 16},
        # the 2:4 gate/up product for one token, 16-bit activations
        {"name": "w4_24_22016x4096_n1", "op": "w4", "m": 22016, "k": 4096, "n": 1, "group": 128, "dtype": "bf16",
         "x": "16", "sparse": True, "zeros": False, "pad": 0},
        # the 2:4 down product for a full batch of 16, 8-bit activations
        {"name": "w4a8_24_4096x11008_n16", "op": "w4", "m": 4096, "k": 11008, "n": 16, "group": 128, "dtype": "f16",
         "x": "i8", "sparse": True, "zeros": False, "pad": 0},
        # weights that no cache holds, 8-bit activations, a batch of 4
        {"name": "w4a8_32768x32768_n4", "op": "w4", "m": 32768, "k": 32768, "n": 4, "group": 128, "dtype": "bf16",
         "x": "i8", "sparse": False, "zeros": True, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rmsnorm", "swiglu", "w4", "w4"])
    dtype = rng.choice(["f16", "bf16"])
    pad = rng.choice([0, 0, 16, 64])
    if op == "w4":
        sparse = rng.random() < 0.5
        x = rng.choice(["16", "i8"])
        # the groups that a step of the matrix instructions covers whole
        least = 32 * (2 if sparse else 1) * (2 if x == "i8" else 1)
        group = rng.choice([g for g in (32, 64, 128, 256) if g >= least] + [0])
        n = rng.choice([1, 1, 2, 3, 4, 7, 8, 16, rng.randint(1, 16), rng.randint(17, 40)])
        m = _log_int(rng, 64, 32768)
        k = _log_int(rng, 128, 16384)
        if rng.random() < 0.7:  # most widths are whole groups, the others end inside one
            k = max(128, k // 128 * 128)
        if sparse:
            k = max(4, k // 4 * 4)
        return {"op": "w4", "m": m, "k": k, "n": n, "group": group, "dtype": dtype, "x": x, "sparse": sparse,
                "zeros": rng.random() < 0.5, "pad": pad}
    rows = _log_int(rng, 1, 8192)
    cols = _log_int(rng, 64, 16384)
    while rows * cols > 1 << 25:
        rows = max(1, rows // 2)
    if rng.random() < 0.6:
        cols = max(64, cols // 64 * 64)
    case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "x": rng.choice(["16", "i32"]),
            "y": rng.choice(["i8", "i8", "16"]), "pad": pad}
    if op == "rmsnorm":
        case["residual"] = rng.random() < 0.7
    return case


def _ld(width, pad, step=16):
    """A row stride that keeps rows on 16-byte boundaries for every element type."""
    return (width + step - 1) // step * step + pad


def _strided(t, pad):
    """The same values in rows that are _ld() apart."""
    out = torch.zeros((t.shape[0], _ld(t.shape[1], pad)), dtype=t.dtype, device=t.device)
    out[:, :t.shape[1]] = t
    return out[:, :t.shape[1]]


def _groups(case):
    return 1 if case["group"] == 0 else -(-case["k"] // case["group"])


def _inputs(case, seed):
    """The inputs of a case, drawn from its seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    dt = _TORCH[case["dtype"]]
    s = {}
    if case["op"] == "w4":
        m, n, k, G = case["m"], case["n"], case["k"], _groups(case)
        kept = k // 2 if case["sparse"] else k
        # codes as a quantiser leaves them: near the middle, seldom at the ends
        pair = (normal(m, -(-kept // 2)) * 2.5 + 8).round_().clamp_(0, 15).to(torch.uint8)
        pair += (normal(m, -(-kept // 2)) * 2.5 + 8).round_().clamp_(0, 15).to(torch.uint8) << 4
        if kept % 2:
            pair[:, -1] &= 15
        s["codes"] = pair
        s["scales"] = (0.004 + 0.012 * uniform(m, G)).to(dt)
        s["zeros"] = torch.randint(5, 12, (m, G), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        s["meta"] = None
        if case["sparse"]:
            # one nibble i0 | i1 << 2 a group of four columns, two to a byte, rows of whole 16 bytes
            table = torch.tensor([i0 | i1 << 2 for i0 in range(4) for i1 in range(i0 + 1, 4)], dtype=torch.uint8, device="cuda")
            nib = table[torch.randint(0, 6, (m, -(-k // 8) * 2), generator=g, device="cuda")]
            nib[:, k // 4:] = 0
            meta = torch.zeros((m, -(-k // 128) * 16), dtype=torch.uint8, device="cuda")
            meta[:, :-(-k // 8)] = nib[:, 0::2] | nib[:, 1::2] << 4
            s["meta"] = meta
        # activations after a norm: unit variance, a few strong channels
        x = normal(n, k) * (1 + 7 * (uniform(1, k) < 0.01))
        if case["x"] == "i8":
            s["x_scale"] = x.abs().amax(1) / 127
            s["x"] = _strided((x / s["x_scale"][:, None]).round_().to(torch.int8), case["pad"])
        else:
            s["x_scale"] = None
            s["x"] = _strided(x.to(dt), case["pad"])
        return s
    rows, cols = case["rows"], case["cols"]
    width = 2 * cols if case["op"] == "swiglu" else cols
    if case["x"] == "i32":
        # accumulators of an int8 product over a few thousand columns
        s["x"] = _strided((normal(rows, width) * 1e5).round_().to(torch.int32), case["pad"])
        s["row_scale"] = 0.02 + 0.02 * uniform(rows)
        s["col_scale"] = 2e-4 + 3e-4 * uniform(width)
    else:
        s["x"] = _strided((normal(rows, width) * (1 + 7 * (uniform(1, width) < 0.01))).to(dt), case["pad"])
        s["row_scale"] = s["col_scale"] = None
    if case["op"] == "rmsnorm":
        s["gamma"] = (1 + 0.2 * normal(cols)).to(dt)
        s["residual"] = _strided((3 * normal(rows, cols)).to(dt), case["pad"]) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import structured_sparse_gemm_nm_amd as nm
        s["nm"], dt = nm, _TORCH[case["dtype"]]
        if case["op"] == "w4":
            ldy = _ld(case["m"], case["pad"])
            plan = nm.nm_w4_plan_init(case["m"], case["n"], case["k"], group=case["group"], dtype=case["dtype"],
                                      x_dtype="i8" if case["x"] == "i8" else None, sparse=case["sparse"],
                                      zeros=case["zeros"], ldx=s["x"].stride(0), ldy=ldy)
            packed = plan.empty_packed()
            nm.nm_w4_pack(plan, s.pop("codes"), s.pop("scales"), packed, zeros=s.pop("zeros"), meta=s.pop("meta"))
            s["plan"], s["packed"] = plan, packed
            s["y"] = torch.empty((case["n"], ldy), dtype=dt, device="cuda")[:, :case["m"]]
            return s
        rows, cols = case["rows"], case["cols"]
        ld = _ld(cols, case["pad"])
        s["plan"] = nm.nm_rows_plan_init(rows, cols, op=case["op"], dtype=case["dtype"],
                                         x_dtype="i32" if case["x"] == "i32" else None,
                                         y_dtype="i8" if case["y"] == "i8" else None,
                                         ldx=s["x"].stride(0), ldr=ld, ldh=ld, ldy=ld, eps=1e-6)
        s["y"] = torch.empty((rows, ld), dtype=torch.int8 if case["y"] == "i8" else dt, device="cuda")[:, :cols]
        s["y_scale"] = torch.empty(rows, device="cuda") if case["y"] == "i8" else None
        s["value"] = torch.empty((rows, cols), dtype=dt, device="cuda") if case["y"] == "i8" else None
        if case["op"] == "rmsnorm":
            s["h"] = torch.empty((rows, ld), dtype=dt, device="cuda")[:, :cols] if case["residual"] else None
    return s


def _scaled(s):
    x = s["x"].float()
    return x * s["row_scale"][:, None] * s["col_scale"] if s["row_scale"] is not None else x


def _in_8_bits(v, amax, scale, dt):
    """Codes of v with the row's largest magnitude at 127, as the values they stand for."""
    q = (v * (127.0 / amax)[:, None]).round()
    return (q * scale[:, None]).to(dt)


def _plain_rmsnorm(s, case, dt):
    x = _scaled(s)
    out = {}
    if s["residual"] is not None:
        x = x + s["residual"].float()
        out["h"] = x.to(dt)
    inv = torch.rsqrt((x * x).mean(1) + 1e-6)
    v = x * s["gamma"].float()
    if case["y"] == "i8":
        amax = v.abs().amax(1)
        out["scale"] = amax * inv / 127.0
        out["y"] = _in_8_bits(v, amax, out["scale"], dt)
    else:
        out["y"] = (v * inv[:, None]).to(dt)
    return out


def _plain_swiglu(s, case, dt):
    x = _scaled(s)
    gate, up = x[:, :case["cols"]], x[:, case["cols"]:]
    v = gate / (1 + torch.exp(-gate)) * up
    if case["y"] == "i8":
        amax = v.abs().amax(1)
        scale = amax / 127.0
        return {"y": _in_8_bits(v, amax, scale, dt), "scale": scale}
    return {"y": v.to(dt)}


def _plain_w4(s, case, dt):
    m, k = case["m"], case["k"]
    kept = k // 2 if case["sparse"] else k
    per = (case["group"] or k) // (2 if case["sparse"] else 1)  # kept values that share a scale
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), 2).reshape(m, -1)[:, :kept].float()
    q -= 8 if s["zeros"] is None else s["zeros"].float().repeat_interleave(per, 1)[:, :kept]
    q *= s["scales"].float().repeat_interleave(per, 1)[:, :kept]
    if case["sparse"]:
        nib = torch.stack((s["meta"] & 15, s["meta"] >> 4), 2).reshape(m, -1)[:, :k // 4]
        at = torch.stack((nib & 3, nib >> 2), 2).long()
        at += 4 * torch.arange(k // 4, device=at.device)[None, :, None]
        q = torch.zeros((m, k), device=q.device).scatter_(1, at.reshape(m, -1), q)
    y = s["x"].float() @ q.t()
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None]
    return {"y": y.to(dt)}


def run(state):
    s, case = state, state["case"]
    if own:
        nm = s["nm"]
        if case["op"] == "w4":
            nm.nm_w4_matvec(s["plan"], s["packed"], s["x"], s["y"], x_scale=s["x_scale"])
            return {"y": s["y"]}
        out = {}
        if case["op"] == "rmsnorm":
            nm.nm_rmsnorm(s["plan"], s["x"], s["gamma"], s["y"], y_scale=s["y_scale"], residual=s["residual"],
                          h=s["h"], row_scale=s["row_scale"], col_scale=s["col_scale"])
            if s["h"] is not None:
                out["h"] = s["h"]
        else:
            nm.nm_swiglu(s["plan"], s["x"], s["y"], y_scale=s["y_scale"], row_scale=s["row_scale"],
                         col_scale=s["col_scale"])
        if s["y_scale"] is None:
            out["y"] = s["y"]
        else:  # a layer's next product reads the codes; they are spelt out here to be compared
            out["scale"] = s["y_scale"]
            out["y"] = torch.mul(s["y"], s["y_scale"][:, None], out=s["value"])
        return out
    plain = {"rmsnorm": _plain_rmsnorm, "swiglu": _plain_swiglu, "w4": _plain_w4}[case["op"]]
    return plain(s, case, _TORCH[case["dtype"]])


def work(case):
    if case["op"] == "w4":
        m, n, k = case["m"], case["n"], case["k"]
        kept = k / 2 if case["sparse"] else k
        weights = m * kept / 2 + (m * k / 8 if case["sparse"] else 0)
        weights += m * _groups(case) * (3 if case["zeros"] else 2)
        x = n * k + 4 * n if case["x"] == "i8" else 2 * n * k
        return {"bytes": weights + x + 2 * n * m, "flops": 2 * m * n * kept}
    rows, cols = case["rows"], case["cols"]
    width = 2 * cols if case["op"] == "swiglu" else cols
    x = rows * width * 2 if case["x"] == "16" else 4 * (rows * width + rows + width)
    y = rows * cols + 4 * rows if case["y"] == "i8" else 2 * rows * cols
    if case["op"] == "rmsnorm":
        x += 2 * cols
        if case["residual"]:
            x += 2 * rows * cols
            y += 2 * rows * cols
    return {"bytes": x + y, "flops": 6 * rows * width}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "w4":
        return {"y": _exact_w4(s, case)}
    x = s["x"].double()
    if case["x"] == "i32":
        x = torch.einsum("rc,r,c->rc", x, s["row_scale"].double(), s["col_scale"].double())
    out = {}
    if case["op"] == "swiglu":
        gate, up = x.split(case["cols"], 1)
        v, per_row = torch.sigmoid(gate) * gate * up, torch.ones(case["rows"], dtype=torch.float64, device="cuda")
    else:
        if s["residual"] is not None:
            x = out["h"] = x + s["residual"].double()
        per_row = 1 / torch.sqrt(x.square().sum(1) / case["cols"] + 1e-6)
        v = x * s["gamma"].double()[None, :]
    if case["y"] == "i8":
        top = torch.linalg.vector_norm(v, ord=math.inf, dim=1)
        out["scale"] = top * per_row / 127
        out["y"] = torch.round(v / top[:, None] * 127) * out["scale"][:, None]
    else:
        out["y"] = v * per_row[:, None]
    return out


def _exact_w4(s, case):
    """Group by group: each group's codes times the columns of x that they meet."""
    m, n, k = case["m"], case["n"], case["k"]
    group = case["group"] or k
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double()[:, None]
    xt = x.t().contiguous()                                                  # k x n
    y = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    step = max(1, (1 << 26) // max(1, n * min(group, k)))                    # rows at a time
    for j in range(_groups(case)):
        c0, c1 = j * group, min(k, (j + 1) * group)
        half = 2 if case["sparse"] else 1
        p = torch.arange(c0 // half, c1 // half, device="cuda")              # kept positions of the group
        for r in range(0, m, step):
            rows = slice(r, min(m, r + step))
            q = (s["codes"][rows][:, p // 2] >> (4 * (p % 2)).to(torch.uint8)[None, :]) & 15
            z = s["zeros"][rows, j].double() if s["zeros"] is not None else 8.0 * torch.ones(q.shape[0], dtype=torch.float64, device="cuda")
            q = q.double() - z[:, None]
            if case["sparse"]:
                four = p // 2
                nib = (s["meta"][rows][:, four // 2] >> (4 * (four % 2)).to(torch.uint8)[None, :]) & 15
                at = 4 * four[None, :] + ((nib >> (2 * (p % 2)).to(torch.uint8)[None, :]) & 3).long()
                part = (q[:, :, None] * xt[at]).sum(1)
            else:
                part = q @ xt[c0:c1]
            y[rows] += part * s["scales"][rows, j].double()[:, None]
    return y.t()
