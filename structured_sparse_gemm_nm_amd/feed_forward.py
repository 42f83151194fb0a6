"""A gated feed-forward block served with 2:4 weights in 4 bits, over the C ABI.

Per call, for the hidden rows x and the residual r:

- nm_rmsnorm: h = x + r, and its norm in 8 bits with one scale a token;
- the joint gate/up product;
- nm_swiglu: silu(gate) * up, in 8 bits with one scale a token;
- the down product, which the next block's norm takes with the residual h.

The weights are pruned to 2:4 and quantised once, to q - 8 with q in 0..15 and one
scale an output feature, so that the same integers serve both of the library's products:

- few tokens: nm_w4_matvec streams them in 4 bits, and the product is 16-bit;
- a prompt: nm_spmm multiplies them as int8 on the 2:4 instructions, and the product
  is int32 accumulators, which the norm and the activation read with a scale for
  each token and each feature (``Rows``).

The 8-bit activations of the two are the same; they differ in the 16-bit rounding
of the few-token products alone.

Features must be multiples of 16. Weights are prepared with torch; every call runs
in the library's kernels and may be captured into a graph. There is no backward
pass: operands that require a gradient are refused while gradients are recorded.
"""
from typing import NamedTuple, Optional

import torch

from . import nm_compress, nm_plan_init, nm_prune, nm_rmsnorm, nm_rows_plan_init, nm_spmm, nm_swiglu, nm_w4_matvec, \
    nm_w4_pack, nm_w4_plan_init

_DTYPE_NAMES = {torch.float16: "f16", torch.bfloat16: "bf16"}

# The 4-bit product passes over its weights once for every 48 tokens, the int8 2:4
# product works on whole tiles of 128. One block of 4096 and 11008 features, in us:
# 30 and 84 for one token, 50 and 122 for 48, 74 and 122 for 49, 94 and 122 for 96,
# 143 and 75 for 128.
FEW_TOKENS = 96


# Plans that a block keeps, of each of its weights and of its row operators: one for each number of tokens
# and product, the least recently used given up first. They hold host memory only.
MOST_PLANS = 256


class _Plans:
    def __init__(self):
        self._kept = {}

    def __len__(self):
        return len(self._kept)

    def get(self, key, make):
        plan = self._kept.pop(key, None)
        if plan is None:
            plan = make()
        self._kept[key] = plan                     # the last in the dictionary's order
        if len(self._kept) > MOST_PLANS:
            self._kept.pop(next(iter(self._kept)), None)
        return plan


class Rows(NamedTuple):
    """What a product hands on: 16-bit values, or int32 accumulators with a scale a row and a column."""

    values: torch.Tensor
    row_scale: Optional[torch.Tensor] = None
    col_scale: Optional[torch.Tensor] = None

    def dense(self):
        """The values in fp32."""
        v = self.values.float()
        return v if self.row_scale is None else v * self.row_scale[:, None] * self.col_scale


class _Weight:
    """One weight (out x in), 2:4 along in: packed 4-bit codes, and the same integers as int8 with metadata."""

    def __init__(self, w):
        out_f, in_f = w.shape
        self.out_f, self.in_f, self.dtype = out_f, in_f, _DTYPE_NAMES[w.dtype]
        plan = nm_plan_init(out_f, 16, in_f, 2, 4, dtype=self.dtype)
        pruned = torch.empty_like(w)
        nm_prune(plan, w, pruned)
        # Below the smallest normal value scales are whole steps of the type: the next one up, or the largest
        # weight would need more than seven of it. Rows of zeros take one step.
        info = torch.finfo(w.dtype)
        scale, step = (pruned.float().abs().amax(1) / 7).double(), info.tiny * info.eps
        scale = torch.where(scale < info.tiny, (scale / step).ceil().clamp_min(1) * step, scale).to(w.dtype)
        self.scale = scale.float()
        q = (pruned.float() / self.scale[:, None]).round_().clamp_(-8, 7).to(torch.int8)
        plan = nm_plan_init(out_f, 16, in_f, 2, 4, dtype="i8", op_b="T", order_cd="col")
        self.values, self.meta = plan.empty_values(), plan.empty_meta()
        nm_compress(plan, q, self.values, self.meta)
        codes = (self.values[:, :in_f // 2].to(torch.int16) + 8).to(torch.uint8)
        self.few = nm_w4_plan_init(out_f, 1, in_f, group=0, dtype=self.dtype, x_dtype="i8", sparse=True)
        self.packed = self.few.empty_packed(device=w.device)
        nm_w4_pack(self.few, codes[:, 0::2] | codes[:, 1::2] << 4, scale[:, None].contiguous(), self.packed, meta=self.meta)
        self._plans = _Plans()

    def dense(self):
        """The weight that both products multiply by, in fp32."""
        full = torch.zeros((self.out_f, self.in_f), device=self.values.device)
        kept = self.values[:, :self.in_f // 2].float() * self.scale[:, None]
        nib = torch.stack((self.meta & 15, self.meta >> 4), 2).reshape(self.out_f, -1)[:, :self.in_f // 4]
        at = torch.stack((nib & 3, nib >> 2), 2).long() + 4 * torch.arange(self.in_f // 4, device=nib.device)[None, :, None]
        return full.scatter_(1, at.reshape(self.out_f, -1), kept)

    def product(self, x, x_scale, few):
        n, device = x.shape[0], x.device
        if few:
            plan = self._plans.get((n, few), lambda: nm_w4_plan_init(self.out_f, n, self.in_f, group=0, dtype=self.dtype,
                                                                     x_dtype="i8", sparse=True))
            y = torch.empty((n, self.out_f), dtype=plan.y_dtype, device=device)
            nm_w4_matvec(plan, self.packed, x, y, x_scale=x_scale)
            return Rows(y)
        plan = self._plans.get((n, few), lambda: nm_plan_init(self.out_f, n, self.in_f, 2, 4, dtype="i8", op_b="T",
                                                              order_cd="col"))
        y = torch.empty((n, self.out_f), dtype=torch.int32, device=device)
        nm_spmm(plan, 1.0, self.values, self.meta, x, 0.0, None, y)
        return Rows(y, x_scale, self.scale)


class CompressedFeedForward:
    """gamma (hidden), gate_up (2 * inner x hidden: the gate's rows, then the up rows), down (hidden x inner):
    16-bit GPU tensors of one type. The block keeps gamma and the weights' compressed forms as constants: a position
    takes 3/8 byte in 4 bits and 5/8 byte as int8, metadata included, 1 byte together."""

    def __init__(self, gamma, gate_up, down, eps=1e-6):
        for name, w in (("gamma", gamma), ("gate_up", gate_up), ("down", down)):
            if w.dtype not in _DTYPE_NAMES or w.dtype != gamma.dtype:
                raise ValueError("%s must be float16 or bfloat16, like gamma" % name)
            if not w.is_cuda or w.device != gamma.device:
                raise ValueError("%s must be on the GPU, gamma's" % name)
            if w.dim() != (1 if name == "gamma" else 2) or not w.is_contiguous():
                raise ValueError("%s must be a contiguous %s" % (name, "vector" if name == "gamma" else "matrix"))
        self.hidden, self.inner = down.shape
        if gamma.shape != (self.hidden,) or gate_up.shape != (2 * self.inner, self.hidden):
            raise ValueError("expected gamma (hidden), gate_up (2 * inner x hidden) and down (hidden x inner)")
        if self.hidden % 16 or self.inner % 16 or not self.hidden or not self.inner:
            raise ValueError("hidden and inner must be positive multiples of 16")
        self.gamma, self.eps, self.dtype = gamma.detach(), eps, gamma.dtype
        self.gate_up, self.down = _Weight(gate_up), _Weight(down)
        self._plans = _Plans()

    def _rows(self, op, n, cols, x):
        acc = x.values.dtype == torch.int32
        return self._plans.get((op, n, acc), lambda: nm_rows_plan_init(
            n, cols, op=op, dtype=_DTYPE_NAMES[self.dtype], x_dtype="i32" if acc else None, y_dtype="i8", eps=self.eps))

    def _check(self, x, residual):
        """x is what a plan of the block can be made for, and no operand wants a gradient."""
        v, row, col = x
        acc = v.dtype is torch.int32
        if not acc and v.dtype is not self.dtype:
            raise ValueError("x must be %s or int32 accumulators, got %s" % (self.dtype, v.dtype))
        if (row is not None) != acc or (col is not None) != acc:
            raise ValueError("row_scale and col_scale must be given exactly where x is int32")
        if v.dim() != 2 or v.size(1) != self.hidden:
            raise ValueError("x must be (tokens x %d), got %s" % (self.hidden, tuple(v.shape)))
        if torch.is_grad_enabled() and any(getattr(t, "requires_grad", False) for t in (v, row, col, residual)):
            raise RuntimeError("the block has no backward pass: x and residual must not require a gradient "
                               "(detach them, or call it under torch.no_grad())")

    def __call__(self, x, residual=None, few=None):
        """x: Rows or a 16-bit tensor (tokens x hidden); residual: 16-bit (tokens x hidden) or None.
        Returns the down product as Rows and the next residual h = x + residual.
        few: which product to take; by default the 4-bit one up to FEW_TOKENS tokens."""
        x = x if isinstance(x, Rows) else Rows(x)
        self._check(x, residual)
        n, device = x.values.shape[0], x.values.device
        few = n <= FEW_TOKENS if few is None else few
        codes = torch.empty((n, self.hidden), dtype=torch.int8, device=device)
        scale = torch.empty((n,), device=device)
        h = torch.empty((n, self.hidden), dtype=self.dtype, device=device)
        nm_rmsnorm(self._rows("rmsnorm", n, self.hidden, x), x.values, self.gamma, codes, y_scale=scale, residual=residual,
                   h=h, row_scale=x.row_scale, col_scale=x.col_scale)
        y = self.gate_up.product(codes, scale, few)
        inner = torch.empty((n, self.inner), dtype=torch.int8, device=device)
        inner_scale = torch.empty((n,), device=device)
        nm_swiglu(self._rows("swiglu", n, self.inner, y), y.values, inner, y_scale=inner_scale, row_scale=y.row_scale,
                  col_scale=y.col_scale)
        return self.down.product(inner, inner_scale, few), h
