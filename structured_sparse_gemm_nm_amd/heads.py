"""Norms of query and key heads with the rotation by position, over the C ABI.

``norm_rotate`` takes what the joint query/key/value product handed on, 16-bit rows
or ``Rows`` of int32 accumulators, and runs nm_head_norm_rope in one pass. From
16-bit rows it is differentiable in the rows and in both gains
(nm_head_norm_rope_backward), so it stands between a SemiStructuredSparseLinear and
the attention in training too; operands with a forward-mode tangent are refused. A backward pass may be captured into a graph while no
eager graph of the same leaves lives: torch ties their gradients to the stream of
the first.
"""
import torch
from torch.autograd.function import once_differentiable

from . import nm_head_norm_rope, nm_head_norm_rope_backward, nm_heads_plan_init
from .feed_forward import Rows, _DTYPE_NAMES, _Plans, refuse_tangents

_PLANS = _Plans()


def rotation_table(positions, rotary_dim, base=10000.0, device="cuda"):
    """positions x rotary_dim floats: the cosines of p * base^(-2i / rotary_dim), then the sines. Angles are computed
    in 64 bits: those of far positions lose theirs in 32."""
    if rotary_dim % 8 or rotary_dim < 0:
        raise ValueError("rotary_dim must be a multiple of 8")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * base ** (-2 * i / max(1, rotary_dim))
    return torch.cat((angle.cos(), angle.sin()), 1).float()


def _empty_rows(rows, cols, dtype, device):
    """Rows that the library takes, on 16-byte boundaries, and no further apart."""
    step = 16 // dtype.itemsize
    return torch.empty((rows, (cols + step - 1) // step * step), dtype=dtype, device=device)[:, :cols]


def _rows_on_16_bytes(t):
    """t, or a copy of it in rows that the library takes."""
    step = 16 // t.element_size()
    if t.stride(1) == 1 and t.stride(0) >= t.shape[1] and t.stride(0) % step == 0 and t.data_ptr() % 16 == 0:
        return t
    return _empty_rows(*t.shape, t.dtype, t.device).copy_(t)


def _plan(x, heads, dim, table, gamma, pairs, eps):
    acc = x.dtype == torch.int32
    table_rows, rotary = (0, 0) if table is None else table.shape
    key = (x.shape[0], x.stride(0), heads, dim, rotary, table_rows, gamma.dtype, acc, pairs, eps)
    return _PLANS.get(key, lambda: nm_heads_plan_init(
        x.shape[0], *heads, dim, rotary, pairs=pairs, table_rows=table_rows, dtype=_DTYPE_NAMES[gamma.dtype],
        x_dtype="i32" if acc else None, ldx=x.stride(0), eps=eps, zero_rows=True, ldg=sum(heads) * dim))


class _NormRotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma_q, gamma_k, positions, table, heads, pairs, eps):
        x = _rows_on_16_bytes(x)
        plan = _plan(x, heads, gamma_q.shape[0], table, gamma_q, pairs, eps)
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        nm_head_norm_rope(plan, x, gamma_q, gamma_k, positions, table, y)
        ctx.save_for_backward(x, gamma_q, gamma_k, positions, table)
        ctx.plan = plan
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        refuse_tangents(dy)
        x, gamma_q, gamma_k, positions, table = ctx.saved_tensors
        plan, gains = ctx.plan, ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dy = dy if dy.is_contiguous() and dy.data_ptr() % 16 == 0 else dy.clone(memory_format=torch.contiguous_format)
        # in rows of its own: x may be rows far apart in something much larger
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dq = dk = workspace = None
        if gains:
            dq, dk = torch.empty_like(gamma_q), None if gamma_k is None else torch.empty_like(gamma_k)
            workspace = plan.empty_workspace(device=x.device)
        nm_head_norm_rope_backward(plan, x, gamma_q, gamma_k, positions, table, dy, dx, dgamma_q=dq, dgamma_k=dk,
                                   workspace=workspace)
        return dx, dq, dk, None, None, None, None, None


def norm_rotate(x, gamma_q, gamma_k, positions, table, heads, pairs="halves", eps=1e-6):
    """x: 16-bit rows (tokens x columns) or ``Rows``; heads: (query, key, value) heads in a row; gamma_q, gamma_k: head
    gains (gamma_k None without key heads); positions: int64, one a token, negative where a row holds none (its output
    is zero); table: rotation_table(...), or None for no rotation. Returns 16-bit rows of x's columns."""
    x = x if isinstance(x, Rows) else Rows(x)
    v, heads = x.values, tuple(int(h) for h in heads)
    if len(heads) != 3:
        raise ValueError("heads must be the numbers of query, key and value heads")
    if gamma_q.dtype not in _DTYPE_NAMES or gamma_q.dim() != 1:
        raise ValueError("gamma_q must be a float16 or bfloat16 vector")
    if (gamma_k is not None) != (heads[1] > 0):
        raise ValueError("gamma_k must be given exactly where there are key heads")
    acc = v.dtype is torch.int32
    if not acc and v.dtype is not gamma_q.dtype:
        raise ValueError("x must be %s or int32 accumulators, got %s" % (gamma_q.dtype, v.dtype))
    if (x.row_scale is not None) != acc or (x.col_scale is not None) != acc:
        raise ValueError("row_scale and col_scale must be given exactly where x is int32")
    if v.dim() != 2 or v.shape[1] != sum(heads) * gamma_q.shape[0]:
        raise ValueError("x must be (tokens x %d), got %s" % (sum(heads) * gamma_q.shape[0], tuple(v.shape)))
    if table is not None and table.dim() != 2:
        raise ValueError("table must be positions x rotary_dim")
    refuse_tangents(*x, gamma_q, gamma_k, table)
    wants = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (v, gamma_q, gamma_k, *x[1:]))
    if torch.is_grad_enabled() and table is not None and table.requires_grad:
        raise RuntimeError("the table has no gradient")
    if not acc and wants:
        return _NormRotate.apply(v, gamma_q, gamma_k, positions, table, heads, pairs, eps)
    if wants:
        raise RuntimeError("accumulators have no gradient: detach the gains, or call it under torch.no_grad()")
    v = _rows_on_16_bytes(v)
    plan = _plan(v, heads, gamma_q.shape[0], table, gamma_q, pairs, eps)
    y = torch.empty(v.shape, dtype=gamma_q.dtype, device=v.device)
    nm_head_norm_rope(plan, v, gamma_q, gamma_k, positions, table, y, row_scale=x.row_scale, col_scale=x.col_scale)
    return y
