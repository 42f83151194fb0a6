"""Where an output may lie in an operand's place, their rows must be the same: the rows of one stride would be written while
those of another are still to be read. Refused before any device call."""
import pytest

import structured_sparse_gemm_nm_amd as nm
from tests.test_layer_ops import FAKE

BAD, F, G = nm.NM_ERR_INVALID_ARG, FAKE, FAKE + (1 << 20)


def message():
    return nm.lib().nm_last_error().decode()


@pytest.mark.parametrize("kw", [dict(ldc=64, ldy=72), dict(ldc=72, ldy=64), dict(ldc=64, ldy=64, base_dtype="i32"),
                                dict(ldc=64, ldy=128, base_dtype="i32"), dict(n=1, base_dtype="i32")])
def test_adapters(kw):
    p = nm.nm_lora_plan_init(**dict(dict(m=64, n=4, k=128, rank=16, adapters=3), **kw))
    acc = G if "base_dtype" in kw else None
    assert nm.lib().nm_lora(p.handle, G, None, G, G, G, G, F, acc, acc, F, G, None) == BAD and "d_base" in message()


@pytest.mark.parametrize("kw", [dict(ldx=512, ldy=520), dict(ldx=520, ldy=512), dict(x_dtype="i32"), dict(x_dtype="i32", ldx=512, ldy=1024),
                                dict(rows=1, x_dtype="i32")])
def test_heads(kw):
    p = nm.nm_heads_plan_init(**dict(dict(rows=8, heads_q=4, heads_k=2, heads_v=2, head_dim=64, rotary_dim=0), **kw))
    acc = G if "x_dtype" in kw else None
    assert nm.lib().nm_head_norm_rope(p.handle, F, acc, acc, G, G, G, None, F, None) == BAD and "dX" in message()


@pytest.mark.parametrize("kw", [dict(ldg=520), dict(ldy=520), dict(ldx=520)])
def test_heads_gradient(kw):
    p = nm.nm_heads_plan_init(**dict(dict(rows=8, heads_q=4, heads_k=2, heads_v=2, head_dim=64, rotary_dim=0), **kw))
    back = nm.lib().nm_head_norm_rope_backward
    assert back(p.handle, G, G, G, G, None, F, F, None, None, None, None) == BAD and "d_grad_y" in message()


@pytest.mark.parametrize("kw", [dict(ldg=520), dict(ldy=520, ldg=520), dict(ldx=520, ldg=512)])
def test_heads_gradient_over_x(kw):
    p = nm.nm_heads_plan_init(**dict(dict(rows=8, heads_q=4, heads_k=2, heads_v=2, head_dim=64, rotary_dim=0), **kw))
    assert nm.lib().nm_head_norm_rope_backward(p.handle, F, G, G, G, None, G, F, None, None, None, None) == BAD and "dX" in message()


@pytest.mark.parametrize("kw", [dict(ldg=1008), dict(ldx=1008, ldg=1000)])
def test_logits_gradient(kw):
    p = nm.nm_logprobs_plan_init(**dict(dict(rows=4, cols=1000), **kw))
    assert nm.lib().nm_logprobs_backward(p.handle, F, G, G, None, G, None, F, None) == BAD and "dX" in message()
