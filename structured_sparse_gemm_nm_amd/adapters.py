"""Low-rank adapters of many requests beside a shared projection, over the C ABI.

``Adapters`` holds the adapters of one projection and adds to what the shared product
gave, each token by the adapter that its index names: nm_lora. The product may be in 16
bits (nm_w4_matvec, nm_spmm) or the int32 accumulators of an int8 one (``Rows``), the
tokens in 16 bits or in the 8-bit codes that the product took. CompressedFeedForward
takes them for its two projections. They serve: there is no backward pass,
nor a forward-mode derivative.
"""
import torch

from . import nm_lora, nm_lora_plan_init
from .feed_forward import Rows, _DTYPE_NAMES, _Plans, refuse_tangents
from .heads import _rows_on_16_bytes


class Adapters:
    """a: adapters x rank x in, b: adapters x out x rank, 16-bit GPU tensors of one type; scale: one fp32 factor an
    adapter. Ranks up to 128; those that are no multiples of 8 are padded with zeros."""

    def __init__(self, a, b, scale):
        for name, w in (("a", a), ("b", b)):
            if w.dtype not in _DTYPE_NAMES or w.dtype != a.dtype:
                raise ValueError("%s must be float16 or bfloat16, both of one type" % name)
            if not w.is_cuda or w.device != a.device:
                raise ValueError("%s must be on the GPU, both on one" % name)
            if w.dim() != 3:
                raise ValueError("%s must have three dimensions, got %s" % (name, tuple(w.shape)))
        self.count, rank, self.in_f = a.shape
        self.out_f = b.shape[1]
        if b.shape != (self.count, self.out_f, rank) or scale.shape != (self.count,):
            raise ValueError("expected a (adapters x rank x in), b (adapters x out x rank) and scale (adapters)")
        if not 1 <= rank <= 128 or not self.count or self.in_f < 16 or self.out_f < 8:
            raise ValueError("rank must be 1 to 128, in at least 16 and out at least 8, and one adapter be given")
        if scale.dtype != torch.float32 or scale.device != a.device:
            raise ValueError("scale must be float32, with the adapters")
        a, b, pad = a.detach(), b.detach(), -rank % 8
        if pad:
            a, b = torch.nn.functional.pad(a, (0, 0, 0, pad)), torch.nn.functional.pad(b, (0, pad))
        self.rank, self.dtype = rank + pad, a.dtype
        self.a = _rows_on_16_bytes(a.reshape(self.count * self.rank, self.in_f))
        b = b.reshape(self.count * self.out_f, self.rank).contiguous()
        self.b = b if b.data_ptr() % 16 == 0 else b.clone()
        self.scale = scale.detach().contiguous()
        self._plans = _Plans()

    def add(self, x, index, base, x_scale=None, out=None):
        """x: tokens x in, 16-bit, or int8 codes with x_scale; index: int64, one a token, negative for no adapter; base:
        tokens x out of the shared product, a 16-bit tensor or ``Rows``. Returns 16-bit rows: out, which may be base, or
        new ones."""
        base = base if isinstance(base, Rows) else Rows(base)
        refuse_tangents(x, x_scale, *base, out)
        for t in (x, x_scale, *base, out):
            if torch.is_grad_enabled() and t is not None and t.requires_grad:
                raise RuntimeError("adapters that are served have no backward pass: detach the operands, or call it "
                                   "under torch.no_grad()")
        v = base.values
        if x.dim() != 2 or v.dim() != 2:
            raise ValueError("x and base must be matrices")
        if x.dtype not in (self.dtype, torch.int8) or v.dtype not in (self.dtype, torch.int32):
            raise ValueError("x must be %s or int8, base %s or int32" % (self.dtype, self.dtype))
        x = _rows_on_16_bytes(x)
        acc, name = v.dtype is torch.int32, _DTYPE_NAMES[self.dtype]
        given = _rows_on_16_bytes(v)
        if out is None:
            out = _rows_on_16_bytes(torch.empty((x.shape[0], self.out_f), dtype=self.dtype, device=x.device))
        key = (x.shape[0], x.dtype, v.dtype, x.stride(0), given.stride(0), out.stride(0))
        plan = self._plans.get(key, lambda: nm_lora_plan_init(
            self.out_f, x.shape[0], self.in_f, self.rank, self.count, dtype=name, x_dtype="i8" if x.dtype is torch.int8 else None,
            base_dtype="i32" if acc else None, ldx=x.stride(0), lda=self.a.stride(0), ldc=given.stride(0), ldy=out.stride(0)))
        nm_lora(plan, x, self.a, self.b, self.scale, index, given, out, x_scale=x_scale, row_scale=base.row_scale,
                col_scale=base.col_scale, workspace=plan.empty_workspace(device=x.device))
        return out

    def dense(self, index):
        """The projection that the adapters add for each token, in fp32: tokens x out x in (zeros for no adapter)."""
        at = index.clamp_min(0)
        a = self.a.reshape(self.count, self.rank, self.in_f).float()[at]
        b = self.b.reshape(self.count, self.out_f, self.rank).float()[at] * self.scale[at][:, None, None]
        return torch.where((index >= 0)[:, None, None], b @ a, torch.zeros((), device=a.device))
