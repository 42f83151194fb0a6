"""Cases of the operators that take what a compressed layer's products hand on.

Three operators, each on 16-bit rows or on the int32 accumulators of an int8
product with a scale for each token and each channel:

- ``lora``: low-rank adapters of many requests beside a shared projection,
  y = base + s B (A x) with the adapter that each token names (or none). x is
  16-bit, or 8-bit codes with one scale a token; base is what the shared
  projection gave.
- ``heads``: the norms of queries and keys for each head and the rotation by
  position, in one pass over the joint query/key/value product; with ``step`` the
  gradients of x and of both gains too.
- ``logprobs``: log probabilities of given tokens, entropy and the most probable
  alternatives from rows of logits; with ``step`` the logits' gradient too.

With ``own`` false ``run`` computes them from elementary torch operations, with
``own`` true by the library's entry points.
"""
import math

import torch

own = False

_TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token of a chat through a square projection, its own adapter of 32 in memory: all latency
        {"name": "lora_1x4096x4096_r16", "op": "lora", "n": 1, "k": 4096, "m": 4096, "rank": 16, "adapters": 32,
         "dtype": "f16", "x": "16", "base": "16", "mix": "scattered", "pad": 0},
        # a decode batch of 16 requests on the joint gate/up projection of a block whose activations are 8-bit
        {"name": "lora_16x4096x22016_r16", "op": "lora", "n": 16, "k": 4096, "m": 22016, "rank": 16, "adapters": 64,
         "dtype": "bf16", "x": "i8", "base": "16", "mix": "scattered", "pad": 0},
        # 37 requests on the down projection, larger ranks, rows with strides of their own
        {"name": "lora_37x11008x4096_r64", "op": "lora", "n": 37, "k": 11008, "m": 4096, "rank": 64, "adapters": 24,
         "dtype": "f16", "x": "16", "base": "16", "mix": "scattered", "pad": 16},
        # prompts of several requests, 4096 tokens together, beside the int8 2:4 product's accumulators
        {"name": "lora_acc_4096x4096x6144_r16", "op": "lora", "n": 4096, "k": 4096, "m": 6144, "rank": 16, "adapters": 16,
         "dtype": "bf16", "x": "i8", "base": "i32", "mix": "runs", "pad": 0},
        # one token, 32 query heads and 8 key and value heads of 128: all latency
        {"name": "heads_1x48x128", "op": "heads", "rows": 1, "q": 32, "kh": 8, "v": 8, "dim": 128, "rotary": 128,
         "pairs": "halves", "table": 32768, "dtype": "f16", "x": "16", "step": False, "pad": 0},
        # an odd batch, a part of each head turned, neighbours in pairs, rows with a stride of their own
        {"name": "heads_777x25x80", "op": "heads", "rows": 777, "q": 20, "kh": 5, "v": 0, "dim": 80, "rotary": 32,
         "pairs": "neighbours", "table": 4096, "dtype": "f16", "x": "16", "step": False, "pad": 16},
        # a prompt of 4096 tokens after the int8 2:4 product: accumulators in, all heads in 16 bits out
        {"name": "heads_acc_4096x48x128", "op": "heads", "rows": 4096, "q": 32, "kh": 8, "v": 8, "dim": 128, "rotary": 128,
         "pairs": "halves", "table": 8192, "dtype": "bf16", "x": "i32", "step": False, "pad": 0},
        # a training step of 8192 tokens: forward and backward
        {"name": "heads_step_8192x48x128", "op": "heads", "rows": 8192, "q": 32, "kh": 8, "v": 8, "dim": 128, "rotary": 128,
         "pairs": "halves", "table": 8192, "dtype": "bf16", "x": "16", "step": True, "pad": 0},
        # one sampled token over an odd vocabulary, half of it ruled out by a grammar, five alternatives
        {"name": "logprobs_1x32003_top5", "op": "logprobs", "rows": 1, "cols": 32003, "dtype": "f16", "x": "16", "top": 5,
         "entropy": False, "temperature": 1.0, "mask": "inf", "step": False, "pad": 0},
        # a decode batch of 16 over a large vocabulary, logits in fp32 after penalties, 20 alternatives
        {"name": "logprobs_16x131072_top20", "op": "logprobs", "rows": 16, "cols": 131072, "dtype": "f32", "x": "16",
         "top": 20, "entropy": True, "temperature": 0.7, "mask": "none", "step": False, "pad": 0},
        # a prompt scored from the accumulators of an int8 head
        {"name": "logprobs_acc_2048x32768_top1", "op": "logprobs", "rows": 2048, "cols": 32768, "dtype": "f16", "x": "i32",
         "top": 1, "entropy": True, "temperature": 1.0, "mask": "none", "step": False, "pad": 0},
        # a training step of 4096 tokens: the loss of given tokens with an entropy term, and the logits' gradient
        {"name": "logprobs_step_4096x131072", "op": "logprobs", "rows": 4096, "cols": 131072, "dtype": "bf16", "x": "16",
         "top": 0, "entropy": True, "temperature": 1.0, "mask": "none", "step": True, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "heads", "logprobs"])
    pad = rng.choice([0, 0, 16, 64])
    dtype = rng.choice(["f16", "bf16"])
    x = rng.choice(["16", "16", "i32"])
    if op == "lora":
        n = rng.choice([1, 2, rng.randint(1, 16), rng.randint(17, 64), _log_int(rng, 64, 4096)])
        k, m = _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
        if rng.random() < 0.6:  # most widths are whole tiles
            k, m = max(64, k // 64 * 64), max(64, m // 64 * 64)
        while n * (k + 3 * m) > 4096 * (4096 + 3 * 6144):
            n = max(1, n // 2)
        return {"op": "lora", "n": n, "k": k, "m": m, "rank": rng.choice([8, 16, 24, 32, 64]),
                "adapters": _log_int(rng, 1, 64), "dtype": dtype, "x": rng.choice(["16", "i8"]),
                "base": "i32" if x == "i32" else "16",
                "mix": rng.choice(["scattered", "runs"]) if n <= 64 else rng.choice(["scattered", "runs", "runs"]), "pad": pad}
    if op == "heads":
        rows = _log_int(rng, 1, 8192)
        q = rng.choice([1, 4, 8, 12, 16, 32, 40, 64, rng.randint(1, 64)])
        kh = rng.choice([q, max(1, q // 4), max(1, q // 8), 1])
        dim = rng.choice([40, 64, 80, 96, 128, 128, 256])
        step = x == "16" and rng.random() < 0.5
        v = rng.choice([0, kh])
        while rows * (q + kh + v) * dim * (2 if x == "i32" else 1) > 8192 * 48 * 128:
            rows = max(1, rows // 2)
        return {"op": "heads", "rows": rows, "q": q, "kh": kh, "v": v, "dim": dim,
                "rotary": rng.choice([dim, dim, 32, dim // 16 * 8]), "pairs": rng.choice(["halves", "neighbours"]),
                "table": _log_int(rng, 512, 65536), "dtype": dtype, "x": x, "step": step, "pad": pad}
    rows, cols = _log_int(rng, 1, 4096), _log_int(rng, 64, 131072)
    if rng.random() < 0.5:
        cols = max(64, cols // 64 * 64)
    dtype = rng.choice(["f16", "bf16", "f32"]) if x == "16" else "f16"
    step = x == "16" and rng.random() < 0.4
    top = rng.choice([0, 1, 5, 20, 32])
    if cols < 256:
        top = min(top, 8)
    while rows * cols > (1 << 26 if top else 1 << 28):
        rows = max(1, rows // 2)
    return {"op": "logprobs", "rows": rows, "cols": cols, "dtype": dtype, "x": x, "top": top,
            "entropy": rng.random() < 0.6, "temperature": rng.choice([1.0, 0.7, 1.3]),
            "mask": rng.choice(["none", "none", "inf", "lowest"]) if x == "16" else "none", "step": step, "pad": pad}


def _ld(width, pad, step=16):
    """A row stride that keeps rows on 16-byte boundaries for every element type."""
    return (width + step - 1) // step * step + pad


def _strided(t, pad):
    """The same values in rows that are _ld() apart; the tensor itself where it lies so already."""
    if _ld(t.shape[1], pad) == t.shape[1]:
        return t
    out = torch.zeros((t.shape[0], _ld(t.shape[1], pad)), dtype=t.dtype, device=t.device)
    out[:, :t.shape[1]] = t
    return out[:, :t.shape[1]]


def _rotation(rows, rotary):
    """Cosines, then sines, of every position's angles: rows x rotary."""
    at = torch.arange(rotary // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * at / max(1, rotary))
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _inputs(case, seed):
    """The inputs of a case, drawn from its seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    dt, pad = _TORCH[case["dtype"]], case["pad"]
    s = {"row_scale": None, "col_scale": None}

    def rows_of(rows, cols, kind, spread):
        """16-bit (or fp32) rows, or accumulators of an int8 product over a few thousand columns."""
        if kind == "i32":
            s["row_scale"] = 0.02 + 0.02 * uniform(rows)
            s["col_scale"] = spread * (2e-4 + 3e-4 * uniform(cols))
            return (normal(rows, cols) * 1e5).round_().to(torch.int32)
        return (normal(rows, cols) * spread).to(dt)

    if case["op"] == "lora":
        n, k, m, r, count = (case[key] for key in ("n", "k", "m", "rank", "adapters"))
        # activations after a norm: unit variance, a few strong channels
        x = normal(n, k) * (1 + 7 * (uniform(1, k) < 0.01))
        if case["x"] == "i8":
            s["x_scale"] = x.abs().amax(1) / 127
            s["x"] = _strided((x / s["x_scale"][:, None]).round_().to(torch.int8), pad)
        else:
            s["x_scale"], s["x"] = None, _strided(x.to(dt), pad)
        s["a"] = _strided((normal(count * r, k) / math.sqrt(k)).to(dt), 0)
        s["b"] = (normal(count * m, r) * 0.05).to(dt)
        s["scale"] = 0.5 + 1.5 * uniform(count)
        # requests without an adapter among those with one; a prompt's tokens share theirs
        runs = 1 if case["mix"] == "scattered" else min(n, 8)
        named = whole(0, count, -(-n // (n // runs))) if runs > 1 else whole(0, count, n)
        named = torch.where(whole(0, 8, named.numel()) == 0, torch.full_like(named, -1), named)
        if runs > 1:
            named = named.repeat_interleave(n // runs)[:n]
        else:
            named[0] = seed % count
        s["index"] = named.contiguous()
        s["base"] = _strided(rows_of(n, m, case["base"], 1.0), pad)
        return s
    if case["op"] == "heads":
        rows, dim, rotary = case["rows"], case["dim"], case["rotary"]
        cols = (case["q"] + case["kh"] + case["v"]) * dim
        s["x"] = _strided(rows_of(rows, cols, case["x"], 1.0), pad)
        s["gamma_q"], s["gamma_k"] = ((1 + 0.2 * normal(dim)).to(dt) for _ in range(2))
        s["table"] = _rotation(case["table"], rotary)
        # sequences one after the other, each from a place of its own on
        start, length = int(seed) % 97, max(1, rows // 3)
        s["positions"] = (torch.arange(rows, device="cuda") % length + start) % case["table"]
        s["dy"] = _strided(normal(rows, cols).to(dt), pad) if case["step"] else None
        return s
    rows, cols = case["rows"], case["cols"]
    x = rows_of(rows, cols, case["x"], 2.5 if case["x"] == "16" else 1.0)
    if case["x"] == "16":
        x[torch.arange(rows, device="cuda"), whole(0, cols, rows)] = 12.0    # the likeliest token stands out
    s["tokens"] = whole(0, cols, rows)
    if case["mask"] != "none":
        out = uniform(rows, cols) < 0.5
        out[:, ::4] = False
        x.masked_fill_(out, -math.inf if case["mask"] == "inf" else torch.finfo(dt).min)
        s["tokens"] = s["tokens"] // 4 * 4
    s["x"] = _strided(x, pad)
    if case["step"]:
        # a padded batch: the last tokens of some sequences are none
        s["tokens"] = torch.where(whole(0, 10, rows) == 0, torch.full_like(s["tokens"], -100), s["tokens"])
        s["g_logprob"] = -(1 + 0.5 * normal(rows))
        s["g_entropy"] = 0.1 * (1 + normal(rows)) if case["entropy"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import structured_sparse_gemm_nm_amd as nm
    s["nm"], dt, pad = nm, _TORCH[case["dtype"]], case["pad"]

    def rows_like(rows, cols):
        return torch.empty((rows, _ld(cols, pad)), dtype=dt, device="cuda")[:, :cols]

    if case["op"] == "lora":
        n, m = case["n"], case["m"]
        s["y"] = rows_like(n, m)
        s["plan"] = nm.nm_lora_plan_init(m, n, case["k"], case["rank"], case["adapters"], dtype=case["dtype"],
                                         x_dtype="i8" if case["x"] == "i8" else None,
                                         base_dtype="i32" if case["base"] == "i32" else None, lda=s["a"].stride(0),
                                         ldx=s["x"].stride(0), ldc=s["base"].stride(0), ldy=s["y"].stride(0))
        s["workspace"] = s["plan"].empty_workspace()
        return s
    if case["op"] == "heads":
        cols = s["x"].shape[1]
        s["y"] = rows_like(case["rows"], cols)
        s["plan"] = nm.nm_heads_plan_init(case["rows"], case["q"], case["kh"], case["v"], case["dim"], case["rotary"],
                                          pairs=case["pairs"], table_rows=case["table"], dtype=case["dtype"],
                                          x_dtype="i32" if case["x"] == "i32" else None, ldx=s["x"].stride(0),
                                          ldy=s["y"].stride(0), eps=EPS)
        if case["step"]:
            s["dx"] = rows_like(case["rows"], cols)
            s["dgamma_q"], s["dgamma_k"] = torch.empty_like(s["gamma_q"]), torch.empty_like(s["gamma_k"])
            s["workspace"] = s["plan"].empty_workspace()
        return s
    rows, top = case["rows"], case["top"]
    s["plan"] = nm.nm_logprobs_plan_init(rows, case["cols"], dtype="i32" if case["x"] == "i32" else case["dtype"], top=top,
                                         scale=1 / case["temperature"], ldx=s["x"].stride(0), ldg=_ld(case["cols"], pad))
    s["workspace"] = s["plan"].empty_workspace()
    s["logprob"] = torch.empty(rows, device="cuda")
    s["entropy"] = torch.empty(rows, device="cuda") if case["entropy"] else None
    s["top_logprob"] = torch.empty((rows, top), device="cuda") if top else None
    s["top_index"] = torch.empty((rows, top), dtype=torch.int64, device="cuda") if top else None
    s["stats"] = torch.empty((rows, 2), device="cuda") if case["step"] else None
    s["dx"] = rows_like(rows, case["cols"]) if case["step"] else None
    return s


def _values(s, key):
    """Rows in fp32; accumulators times their two scales."""
    x = s[key].float()
    return x * s["row_scale"][:, None] * s["col_scale"] if s["row_scale"] is not None else x


def _plain_lora(s, case, dt):
    n, r, m, count = case["n"], case["rank"], case["m"], case["adapters"]
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"][:, None]
    t = (x @ s["a"].float().t()).reshape(n, count, r)               # every adapter's, then the named one's
    mine = s["index"][:, None] == torch.arange(count, device=x.device)
    t = torch.where(mine[:, :, None], t * s["scale"][None, :, None], torch.zeros((), device=x.device))
    b = s["b"].float().reshape(count, m, r).transpose(0, 1).reshape(m, count * r)
    return {"y": (_values(s, "base") + t.reshape(n, count * r) @ b.t()).to(dt)}


def _turn(v, c, sn, pairs, back=False):
    """The pairs of v's last dimension turned by the angles of (c, sn), or back."""
    if back:
        sn = -sn
    half = v.shape[-1] // 2
    a, b = (v[..., :half], v[..., half:]) if pairs == "halves" else (v[..., 0::2], v[..., 1::2])
    out = (a * c - b * sn, b * c + a * sn)
    return torch.cat(out, -1) if pairs == "halves" else torch.stack(out, -1).flatten(-2)


def _plain_heads(s, case, dt):
    rows, dim, rot = case["rows"], case["dim"], case["rotary"]
    normed = case["q"] + case["kh"]
    u = _values(s, "x").reshape(rows, -1, dim)
    gamma = torch.cat((s["gamma_q"].float().expand(case["q"], dim), s["gamma_k"].float().expand(case["kh"], dim)))
    c, sn = s["table"][s["positions"]][:, None, :].split(rot // 2, 2)
    qk = u[:, :normed]
    f = torch.rsqrt((qk * qk).mean(2, keepdim=True) + EPS)
    v = qk * f * gamma
    v = torch.cat((_turn(v[..., :rot], c, sn, case["pairs"]), v[..., rot:]), 2)
    out = {"y": torch.cat((v, u[:, normed:]), 1).reshape(rows, -1).to(dt)}
    if case["step"]:
        dy = s["dy"].float().reshape(rows, -1, dim)
        g = dy[:, :normed]
        g = torch.cat((_turn(g[..., :rot], c, sn, case["pairs"], back=True), g[..., rot:]), 2)
        dgamma = (g * qk * f).sum(0)
        out["dgamma_q"] = dgamma[:case["q"]].sum(0).to(dt)
        out["dgamma_k"] = dgamma[case["q"]:].sum(0).to(dt)
        w = g * gamma
        dx = f * w - qk * (f * f * f / dim) * (w * qk).sum(2, keepdim=True)
        out["dx"] = torch.cat((dx, dy[:, normed:]), 1).reshape(rows, -1).to(dt)
    return out


def _plain_logprobs(s, case, dt):
    scale = 1 / case["temperature"]
    x = _values(s, "x")
    z = x * scale
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    logp = z - torch.log(total)
    tokens = s["tokens"]
    some = tokens >= 0
    zero = torch.zeros((), device=x.device)
    out = {"logprob": torch.where(some, logp.gather(1, tokens.clamp_min(0)[:, None])[:, 0], zero)}
    p = e / total
    if case["entropy"]:
        out["entropy"] = -torch.where(p > 0, p * logp, zero).sum(1)
    if case["top"]:
        order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :case["top"]]
        out["top_index"], out["top_logprob"] = order, logp.gather(1, order)
    if case["step"]:
        g = torch.where(some, s["g_logprob"], zero)[:, None]
        dx = -g * p
        dx.scatter_add_(1, tokens.clamp_min(0)[:, None], g)
        if case["entropy"]:
            dx -= s["g_entropy"][:, None] * torch.where(p > 0, p * (logp + out["entropy"][:, None]), zero)
        out["dx"] = (dx * scale).to(dt)
    return out


def run(state):
    s, case = state, state["case"]
    if not own:
        plain = {"lora": _plain_lora, "heads": _plain_heads, "logprobs": _plain_logprobs}[case["op"]]
        return plain(s, case, _TORCH[case["dtype"]])
    nm = s["nm"]
    if case["op"] == "lora":
        nm.nm_lora(s["plan"], s["x"], s["a"], s["b"], s["scale"], s["index"], s["base"], s["y"], x_scale=s["x_scale"],
                   row_scale=s["row_scale"], col_scale=s["col_scale"], workspace=s["workspace"])
        return {"y": s["y"]}
    if case["op"] == "heads":
        nm.nm_head_norm_rope(s["plan"], s["x"], s["gamma_q"], s["gamma_k"], s["positions"], s["table"], s["y"],
                             row_scale=s["row_scale"], col_scale=s["col_scale"])
        out = {"y": s["y"]}
        if case["step"]:
            nm.nm_head_norm_rope_backward(s["plan"], s["x"], s["gamma_q"], s["gamma_k"], s["positions"], s["table"],
                                          s["dy"], s["dx"], dgamma_q=s["dgamma_q"], dgamma_k=s["dgamma_k"],
                                          workspace=s["workspace"])
            out.update(dgamma_q=s["dgamma_q"], dgamma_k=s["dgamma_k"], dx=s["dx"])
        return out
    nm.nm_logprobs(s["plan"], s["x"], s["tokens"], s["logprob"], entropy=s["entropy"], stats=s["stats"],
                   top_logprob=s["top_logprob"], top_index=s["top_index"], row_scale=s["row_scale"],
                   col_scale=s["col_scale"], workspace=s["workspace"])
    out = {"logprob": s["logprob"]}
    if case["entropy"]:
        out["entropy"] = s["entropy"]
    if case["top"]:
        out["top_index"], out["top_logprob"] = s["top_index"], s["top_logprob"]
    if case["step"]:
        nm.nm_logprobs_backward(s["plan"], s["x"], s["tokens"], s["stats"], s["dx"], g_logprob=s["g_logprob"],
                                g_entropy=s["g_entropy"], entropy=s["entropy"])
        out["dx"] = s["dx"]
    return out


def _size(kind, dtype="f16"):
    return {"i32": 4, "i8": 1}.get(kind, 4 if dtype == "f32" else 2)


def work(case):
    if case["op"] == "lora":
        n, k, m, r = (case[key] for key in ("n", "k", "m", "rank"))
        runs = min(n, 8) if case["mix"] == "runs" else n
        used = min(case["adapters"], runs)
        rows = n * (k * _size(case["x"]) + m * _size(case["base"]) + 2 * m + 8)
        scales = (4 * n if case["x"] == "i8" else 0) + (4 * (n + m) if case["base"] == "i32" else 0)
        return {"bytes": rows + scales + 2 * used * r * (k + m), "flops": 2 * n * r * (k + m)}
    if case["op"] == "heads":
        rows, cols = case["rows"], (case["q"] + case["kh"] + case["v"]) * case["dim"]
        once = rows * cols * (_size(case["x"]) + 2) + rows * 8 + min(case["table"], rows) * case["rotary"] * 4
        once += 4 * (rows + cols) if case["x"] == "i32" else 0
        return {"bytes": once + (rows * cols * 4 if case["step"] else 0), "flops": rows * cols * (24 if case["step"] else 8)}
    rows, cols = case["rows"], case["cols"]
    size = _size(case["x"], case["dtype"])
    once = rows * cols * size + rows * (12 + 4 * case["entropy"] + 12 * case["top"])
    once += 4 * (rows + cols) if case["x"] == "i32" else 0
    return {"bytes": once + (rows * (cols * size + 8) if case["step"] else 0), "flops": rows * cols * (16 if case["step"] else 6)}


def exact(case, seed):
    s = _inputs(case, seed)
    return {"lora": _exact_lora, "heads": _exact_heads, "logprobs": _exact_logprobs}[case["op"]](s, case)


def _exact_rows(s, x):
    x = x.double()
    if s["row_scale"] is not None:
        x = torch.einsum("rc,r,c->rc", x, s["row_scale"].double(), s["col_scale"].double())
    return x


def _exact_lora(s, case):
    """Adapter by adapter, the tokens that name it."""
    r, m = case["rank"], case["m"]
    y = _exact_rows(s, s["base"])
    for a in sorted(set(s["index"].tolist()) - {-1}):
        mine = (s["index"] == a).nonzero()[:, 0]
        x = s["x"][mine].double()
        if s["x_scale"] is not None:
            x = x * s["x_scale"][mine].double()[:, None]
        inner = x @ s["a"][a * r:(a + 1) * r].double().t().contiguous()
        y[mine] += s["scale"][a].double() * (inner @ s["b"][a * m:(a + 1) * m].double().t().contiguous())
    return {"y": y}


def _exact_heads(s, case):
    """The rotation as a product of complex numbers, the norm's gradient by its projection."""
    rows, dim, rot, q, k = (case[key] for key in ("rows", "dim", "rotary", "q", "kh"))
    x = _exact_rows(s, s["x"]).view(rows, -1, dim)
    half = rot // 2
    table = s["table"].double()[s["positions"]]
    phase = torch.complex(table[:, :half], table[:, half:])[:, None, :]

    def turned(v, by):
        head = v[..., :rot]
        pair = head.unflatten(-1, (2, half)).transpose(-1, -2) if case["pairs"] == "halves" else head.unflatten(-1, (half, 2))
        new = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * by)
        new = new.transpose(-1, -2).flatten(-2) if case["pairs"] == "halves" else new.flatten(-2)
        return torch.cat((new, v[..., rot:]), -1)

    y, dx, dgammas = [], [], []
    for first, last, gamma in ((0, q, "gamma_q"), (q, q + k, "gamma_k")):
        u, gain = x[:, first:last], s[gamma].double()
        size = torch.sqrt(u.square().sum(-1, keepdim=True) / dim + EPS)
        unit = u / size
        y.append(turned(unit * gain, phase))
        if case["step"]:
            g = turned(s["dy"].double().view(rows, -1, dim)[:, first:last], phase.conj())
            dgammas.append((g * unit).sum((0, 1)))
            g = g * gain
            dx.append((g - unit * (g * unit).mean(-1, keepdim=True)) / size)
    y.append(x[:, q + k:])
    out = {"y": torch.cat(y, 1).flatten(1)}
    if case["step"]:
        dx.append(s["dy"].double().view(rows, -1, dim)[:, q + k:])
        out.update(dgamma_q=dgammas[0], dgamma_k=dgammas[1], dx=torch.cat(dx, 1).flatten(1))
    return out


def _exact_logprobs(s, case):
    """A logit is the fp32 value that the row holds (the fp32 product of an accumulator and its scales); the rest in 64 bits."""
    rows, cols, top = case["rows"], case["cols"], case["top"]
    size = max(1, (1 << 26) // cols)
    out = {}

    def put(key, value, r):
        if key not in out:
            out[key] = torch.empty((rows,) + tuple(value.shape[1:]), dtype=value.dtype, device=value.device)
        out[key][r] = value

    for i in range(0, rows, size):
        r = slice(i, min(rows, i + size))
        x = s["x"][r].float()
        if s["row_scale"] is not None:
            x = (x * s["row_scale"][r, None]) * s["col_scale"]
        z = x.double() / case["temperature"]
        logp = z - torch.logsumexp(z, 1, keepdim=True)
        p = logp.exp()
        t = s["tokens"][r]
        given = torch.where(t >= 0, t, 0)[:, None]
        weight = (t >= 0).double()
        put("logprob", torch.where(t >= 0, torch.take_along_dim(logp, given, 1)[:, 0], 0.0), r)
        terms = torch.special.entr(p)
        if case["entropy"]:
            put("entropy", terms.sum(1), r)
        if top:
            # one key a logit: its value, then the lower index
            value, index = torch.topk(x, min(cols, 8 * top + 64), dim=1)
            least = value[:, top - 1:top]
            place = torch.arange(cols, device=x.device)
            order = torch.empty((x.shape[0], top), dtype=torch.int64, device=x.device)
            for j in range(top):
                best = value[:, j:j + 1]
                same = value[:, :j] == best
                rank = same.sum(1, keepdim=True)                      # how many equal ones stand before
                hits = (x == best).to(torch.int8)
                nth = (hits.cumsum(1, dtype=torch.int32) == rank + 1) & (hits == 1)
                order[:, j] = torch.where(nth, place, 0).amax(1)
            assert bool((least <= value[:, :top]).all())
            put("top_index", order, r)
            put("top_logprob", torch.take_along_dim(logp, order, 1), r)
        if case["step"]:
            g = s["g_logprob"][r].double() * weight
            dx = p * -g[:, None]
            dx[torch.arange(dx.shape[0], device=dx.device), given[:, 0]] += g
            if case["entropy"]:
                h = s["g_entropy"][r].double()
                dx += h[:, None] * (terms - p * terms.sum(1, keepdim=True))
            put("dx", dx / case["temperature"], r)
    return out
