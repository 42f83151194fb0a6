"""Log probabilities of given tokens from the head's product, over the C ABI.

``token_logprobs`` takes rows of logits, 16-bit or fp32, or the ``Rows`` of int32
accumulators that the head's product handed on, and runs nm_logprobs. From 16-bit or
fp32 logits the log probabilities and the entropy are differentiable
(nm_logprobs_backward): minus their mean is the loss that a language model is trained
on, the entropy a term beside it; logits with a forward-mode tangent are refused. A
backward pass may be captured into a graph while no eager graph of the same leaves
lives: torch ties their gradients to the stream of the first.
"""
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import nm_logprobs, nm_logprobs_backward, nm_logprobs_plan_init
from .feed_forward import Rows, _Plans, refuse_tangents
from .heads import _empty_rows, _rows_on_16_bytes

_NAMES = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32", torch.int32: "i32"}
_PLANS = _Plans()


class LogProbs(NamedTuple):
    """One row a token; what was not asked for is None."""

    logprob: torch.Tensor
    entropy: Optional[torch.Tensor] = None
    top_logprob: Optional[torch.Tensor] = None
    top_index: Optional[torch.Tensor] = None


def _plan(x, top, scale):
    key = (tuple(x.shape), x.stride(0), x.dtype, top, scale)
    return _PLANS.get(key, lambda: nm_logprobs_plan_init(
        *x.shape, dtype=_NAMES[x.dtype], top=top, scale=scale, ldx=x.stride(0),
        ldg=_empty_rows(1, x.shape[1], x.dtype, "meta").stride(0)))


def _forward(plan, x, tokens, entropy, stats, row_scale=None, col_scale=None):
    rows, device = x.shape[0], x.device
    out = LogProbs(torch.empty(rows, device=device), torch.empty(rows, device=device) if entropy else None)
    if plan.top:
        out = out._replace(top_logprob=torch.empty((rows, plan.top), device=device),
                           top_index=torch.empty((rows, plan.top), dtype=torch.int64, device=device))
    nm_logprobs(plan, x, tokens, out.logprob, entropy=out.entropy, stats=stats, top_logprob=out.top_logprob,
                top_index=out.top_index, row_scale=row_scale, col_scale=col_scale,
                workspace=plan.empty_workspace(device=device))
    return out


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, tokens, top, scale, entropy):
        x = _rows_on_16_bytes(x)
        plan = _plan(x, top, scale)
        stats = torch.empty((x.shape[0], 2), device=x.device)
        out = _forward(plan, x, tokens, entropy, stats)
        ctx.save_for_backward(x, tokens, stats, out.entropy)
        ctx.plan = plan
        ctx.set_materialize_grads(False)
        if plan.top:
            ctx.mark_non_differentiable(out.top_logprob, out.top_index)
        return tuple(out)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logprob, g_entropy, *_):
        refuse_tangents(g_logprob, g_entropy)
        x, tokens, stats, entropy = ctx.saved_tensors
        if g_logprob is None and g_entropy is None:
            return None, None, None, None, None
        # in rows of its own: logits may be rows far apart in something much larger
        dx = _empty_rows(*x.shape, x.dtype, x.device)
        g_logprob, g_entropy = (None if g is None else g.contiguous() for g in (g_logprob, g_entropy))
        nm_logprobs_backward(ctx.plan, x, tokens, stats, dx, g_logprob=g_logprob, g_entropy=g_entropy, entropy=entropy)
        return dx, None, None, None, None


def token_logprobs(logits, tokens, temperature=1.0, top=0, entropy=False):
    """logits: rows x vocabulary (float16, bfloat16 or float32), or ``Rows``; tokens: int64, one a row, negative for
    none (its log probability is 0 and it has no gradient); top: how many alternatives to return, up to 32. Returns
    LogProbs: fp32 values, and int64 columns of the alternatives, which carry no gradient."""
    logits = logits if isinstance(logits, Rows) else Rows(logits)
    x, acc = logits.values, logits.values.dtype is torch.int32
    if x.dtype not in _NAMES:
        raise ValueError("logits must be float16, bfloat16, float32 or int32 accumulators, got %s" % x.dtype)
    if (logits.row_scale is not None) != acc or (logits.col_scale is not None) != acc:
        raise ValueError("row_scale and col_scale must be given exactly where the logits are int32")
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError("logits must be rows x vocabulary, got %s" % (tuple(x.shape),))
    if not temperature > 0:
        raise ValueError("temperature must be positive, got %r" % (temperature,))
    refuse_tangents(*logits)
    wants = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in logits)
    if acc and wants:
        raise RuntimeError("accumulators have no gradient: call it under torch.no_grad()")
    top, scale = int(top), 1.0 / temperature
    if wants:
        return LogProbs(*_TokenLogprobs.apply(x, tokens, top, scale, bool(entropy)))
    x = _rows_on_16_bytes(x)
    return _forward(_plan(x, top, scale), x, tokens, entropy, None, logits.row_scale, logits.col_scale)
