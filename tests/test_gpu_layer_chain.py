"""The operators between the products, one behind the other as they are used: a served layer with adapters up to the
answer's log probabilities, and a training step through the 2:4 layer.

Serving: each operator is held against 64 bits of what it was given, by its own tests' bounds; the whole runs captured,
and every replay equals the eager run. Training, f16, against 64 bits of the whole: roundings of 2^-12 at most of a value
in the mean square (half a step is 2^-11) happen to the product, to y, to their two gradients and to dx, and to the
attention's output and its gradient; a score, at most 12 here, of 2 roundings moves its probability by 12 * 2^-11 and the
gradient through it by twice that, 0.012; with the seven plain ones, 0.002, under 2^-6 of a gradient's norm."""
import pytest
import torch

import structured_sparse_gemm_nm_amd as nm
from structured_sparse_gemm_nm_amd.feed_forward import Rows, _Weight
from structured_sparse_gemm_nm_amd.heads import norm_rotate, rotation_table
from structured_sparse_gemm_nm_amd.linear import SemiStructuredSparseLinear
from structured_sparse_gemm_nm_amd.logprobs import token_logprobs
from tests import test_gpu_heads as heads_of, test_gpu_logprobs as logprobs_of, test_gpu_lora as lora_of
from tests.test_gpu_feed_forward import block
from tests.test_gpu_layer_ops import HALF, TINY, close

pytestmark = pytest.mark.gpu
NAMES = {torch.float16: "f16", torch.bfloat16: "bf16"}
HIDDEN, INNER, HEADS, DIM, WORDS, COUNT, RANK = 128, 192, (4, 2, 2), 32, 1008, 5, 16


class Layer:
    def __init__(self, dtype, few):
        g = torch.Generator(device="cuda").manual_seed(5)
        weight = lambda m, k: _Weight((torch.randn(m, k, generator=g, device="cuda") / k ** 0.5).to(dtype))  # noqa: E731
        self.dtype, self.few = dtype, few
        self.qkv, self.out, self.head = weight(sum(HEADS) * DIM, HIDDEN), weight(HIDDEN, HEADS[0] * DIM), weight(WORDS, HIDDEN)
        self.ff, _, _ = block(HIDDEN, INNER, dtype)
        self.gains = [(1 + 0.2 * torch.randn(DIM, generator=g, device="cuda")).to(dtype) for _ in range(2)]
        self.table = rotation_table(64, DIM)
        make = lora_of.adapters
        self.on_qkv = make(COUNT, HIDDEN, sum(HEADS) * DIM, RANK, dtype, 1)
        self.on_ff = make(COUNT, HIDDEN, 2 * INNER, RANK, dtype, 2), make(COUNT, INNER, HIDDEN, RANK, dtype, 3)
        self.seen = {}

    def codes(self, x):
        n, cols = x.shape
        plan = nm.nm_rows_plan_init(n, cols, op="rmsnorm", dtype=NAMES[self.dtype], y_dtype="i8")
        codes, scale = torch.empty((n, cols), dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
        nm.nm_rmsnorm(plan, x, torch.ones(cols, dtype=self.dtype, device="cuda"), codes, y_scale=scale)
        return codes, scale

    def attend(self, y, sequence):
        """Causal attention of one sequence a value of `sequence`, in fp32."""
        q, k, v = y.float().reshape(y.shape[0], -1, DIM).split(HEADS, 1)
        k, v = (t.repeat_interleave(HEADS[0] // HEADS[1], 1) for t in (k, v))
        scores = (q.transpose(0, 1).contiguous() @ k.permute(1, 2, 0).contiguous()) / DIM ** 0.5
        at = torch.arange(y.shape[0], device="cuda")
        sees = (sequence[:, None] == sequence) & (at[:, None] >= at)
        p = torch.where(sees, scores, float("-inf")).softmax(-1)
        return (p @ v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(y.shape[0], -1).to(self.dtype)

    def __call__(self, x, index, positions, sequence, tokens):
        codes, scale = self.codes(x)
        product = self.qkv.product(codes, scale, self.few)
        qkv = self.on_qkv.add(codes, index, product, x_scale=scale)
        y = norm_rotate(qkv, *self.gains, positions, self.table, HEADS)
        plain = norm_rotate(product, *self.gains, positions, self.table, HEADS)       # what a layer without adapters does
        attention = self.attend(y, sequence)
        acc = self.out.product(*self.codes(attention), self.few)
        z, h = self.ff(acc, x, adapters=(index, *self.on_ff), few=self.few)
        logits = self.head.product(*self.codes(h + z.values), self.few)
        answer = token_logprobs(logits, tokens, temperature=0.7, top=5, entropy=True)
        self.seen = dict(codes=codes, scale=scale, product=product, qkv=qkv, y=y, plain=plain, logits=logits)
        return (y, plain, z.values, h, *answer)


def inputs(n, dtype, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, HIDDEN, generator=g, device="cuda").to(dtype)
    index = torch.randint(-1, COUNT, (n,), generator=g, device="cuda")
    sequence = torch.arange(n, device="cuda") // 33
    positions = torch.arange(n, device="cuda") % 33
    positions[-2:] = -1                                        # rows behind the last sequence
    tokens = torch.randint(0, WORDS, (n,), generator=g, device="cuda")
    tokens[-2:] = -1
    return x, index, positions, sequence, tokens


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,few", [(3, True), (40, True), (16, False), (300, False)])
def test_a_served_layer(n, few, dtype):
    layer, args, name = Layer(dtype, few), inputs(n, dtype), NAMES[dtype]
    out = [t.clone() for t in layer(*args)]
    x, index, positions, sequence, tokens = args
    s = {k: (Rows(*(None if t is None else t.cpu() for t in v)) if isinstance(v, Rows) else v.cpu()) for k, v in layer.seen.items()}
    rows = lambda r: {"x": r.values, "row_scale": r.row_scale, "col_scale": r.col_scale, "dtype": name}  # noqa: E731
    given = rows(s["product"])
    ad = layer.on_qkv
    want, tol = lora_of.plain(dict(given, x=s["codes"], base=s["product"].values, x_scale=s["scale"], a=ad.a.cpu(), b=ad.b.cpu(),
                                   scale=ad.scale.cpu(), index=index.cpu()), RANK)
    close(layer.seen["qkv"], want, tol, "adapters")
    for got, source in (("y", Rows(s["qkv"])), ("plain", s["product"])):
        case = dict(rows(source), heads=HEADS, dim=DIM, rotary=DIM, gamma_q=layer.gains[0].cpu(), gamma_k=layer.gains[1].cpu(),
                    positions=positions.cpu(), table=layer.table.cpu())
        want, size = (t.flatten(1)[:-2] for t in heads_of.plain(case, "halves", 1e-6))
        close(layer.seen[got][:-2], want, HALF[name] * want.abs() + heads_of.FWD * size * (1 + HALF[name]) + TINY[name], got)
        assert (layer.seen[got][-2:] == 0).all()
    logits = dict(rows(s["logits"]), dtype="i32" if s["logits"].row_scale is not None else name)
    logp, H, _ = logprobs_of.plain(logits, 1 / 0.7)
    want = logp.gather(1, tokens.cpu().clamp_min(0)[:, None])[:, 0]
    want[-2:] = 0
    logprobs_of.same(out[4], want, logprobs_of.error(None, WORDS, want), "logprob")
    logprobs_of.same(out[5], H, logprobs_of.error(None, WORDS, H), "entropy")
    assert torch.equal(out[7][:, 0].cpu(), logp.argmax(1))
    # captured: other tokens, adapters and positions through the same graph, with eager runs in between
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer(*args)
    for i in range(3):
        for t, other in zip(args, inputs(n, dtype, seed=3 + i)):
            t.copy_(other)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in captured]
        eager = layer(*args)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))
        assert i or all(torch.equal(a, b) for a, b in zip(got, out))


def test_a_training_step():
    n, dtype = 64, torch.float16
    g = torch.Generator(device="cuda").manual_seed(9)
    linear = SemiStructuredSparseLinear(HIDDEN, sum(HEADS) * DIM, dtype=dtype)
    with torch.no_grad():
        linear.weight.copy_(torch.randn(linear.weight.shape, generator=g, device="cuda") / HIDDEN ** 0.5 * 2 ** 0.5)
        # what the layer multiplies by
        dense = linear(torch.eye(HIDDEN, dtype=dtype, device="cuda")).t().double().cpu()
    layer = Layer(dtype, True)
    x = torch.randn(n, HIDDEN, generator=g, device="cuda").to(dtype).requires_grad_()
    gains = [t.clone().requires_grad_() for t in layer.gains]
    words = (torch.randn(WORDS, HEADS[0] * DIM, generator=g, device="cuda") / DIM ** 0.5)
    _, _, positions, sequence, tokens = inputs(n, dtype)
    y = norm_rotate(linear(x), *gains, positions, layer.table, HEADS)
    scored = token_logprobs(layer.attend(y, sequence).float() @ words.t().contiguous(), tokens, entropy=True)
    scale = 256.0                                              # keeps f16 gradients normal
    (scale * (0.01 * scored.entropy.sum() - scored.logprob.sum())).backward()
    # the same in 64 bits
    X, G = x.detach().double().cpu().requires_grad_(), [t.detach().double().cpu().requires_grad_() for t in gains]
    case = {"x": X, "row_scale": None, "heads": HEADS, "dim": DIM, "rotary": DIM, "positions": positions.cpu(), "table": layer.table.cpu()}
    Y = heads_of.plain(case, "halves", 1e-6, gamma_q=G[0], gamma_k=G[1], x=X @ dense.t())[0]
    Y = torch.where((positions.cpu() >= 0)[:, None, None], Y, 0.0)
    q, k, v = Y.split(HEADS, 1)
    k, v = (t.repeat_interleave(HEADS[0] // HEADS[1], 1) for t in (k, v))
    scores = torch.einsum("qhd,khd->hqk", q, k) / DIM ** 0.5
    assert scores.detach().abs().max() < 12
    at, seq = torch.arange(n), sequence.cpu()
    p = torch.where((seq[:, None] == seq) & (at[:, None] >= at), scores, float("-inf")).softmax(-1)
    logp = (torch.einsum("hqk,khd->qhd", p, v).flatten(1) @ words.double().cpu().t()).log_softmax(1)
    T = tokens.cpu()
    lp = torch.where(T >= 0, logp.gather(1, T.clamp_min(0)[:, None])[:, 0], 0.0)
    (scale * (-0.01 * (logp.exp() * logp).sum() - lp.sum())).backward()
    for got, want, what in ((x.grad, X.grad, "x"), (gains[0].grad, G[0].grad, "query gain"), (gains[1].grad, G[1].grad, "key gain")):
        off = (got.double().cpu() - want).norm() / want.norm()
        assert got.isfinite().all() and off < 2.0 ** -6, (what, off)
    assert linear.weight.grad.isfinite().all() and (linear.weight.grad != 0).any()
