"""The operators have no forward-mode derivative: operands that carry a tangent are refused, with and without gradient
mode, before anything is computed from their values alone."""
import pytest
import torch
from torch.autograd import forward_ad

from structured_sparse_gemm_nm_amd.adapters import Adapters
from structured_sparse_gemm_nm_amd.feed_forward import Rows, _Plans
from structured_sparse_gemm_nm_amd.heads import _NormRotate, norm_rotate
from structured_sparse_gemm_nm_amd.logprobs import _TokenLogprobs, token_logprobs
from tests.test_feed_forward_calls import block

HALF, INTS = torch.zeros((4, 32), dtype=torch.float16), torch.zeros((4, 32), dtype=torch.int32)
ROW, COL, GAIN, AT, TABLE = torch.ones(4), torch.ones(32), torch.ones(8, dtype=torch.float16), torch.zeros(4, dtype=torch.int64), \
    torch.zeros((5, 8))


def adapters():
    """Adapters without weights on a GPU: calls reach their checks."""
    ad = Adapters.__new__(Adapters)
    ad.count, ad.rank, ad.in_f, ad.out_f, ad.dtype = 1, 8, 32, 32, torch.float16
    ad.a, ad.b, ad.scale, ad._plans = HALF[:, :32], torch.zeros((32, 8), dtype=torch.float16), torch.ones(1), _Plans()
    return ad


CALLS = [
    # the call, its operands, and which of them are floating point
    (lambda v, gq, gk, t: norm_rotate(v, gq, gk, AT, t, (2, 1, 1)), (HALF, GAIN, GAIN, TABLE)),
    (lambda r, c, gq: norm_rotate(Rows(INTS, r, c), gq, GAIN, AT, TABLE, (2, 1, 1)), (ROW, COL, GAIN)),
    (lambda v: token_logprobs(v, AT), (HALF,)),
    (lambda v: token_logprobs(v, AT, entropy=True, top=3), (HALF.float(),)),
    (lambda r, c: token_logprobs(Rows(INTS, r, c), AT), (ROW, COL)),
    (lambda x, base, out: adapters().add(x, AT, base, out=out), (HALF, HALF, HALF)),
    (lambda s, r, c: adapters().add(INTS.to(torch.int8), AT, Rows(INTS, r, c), x_scale=s), (ROW, ROW, COL)),
    (lambda x, residual: block()(x, residual), (HALF, HALF)),
    (lambda r, c: block()(Rows(INTS, r, c)), (ROW, COL)),
]


@pytest.mark.parametrize("call,which", [(c, i) for c in range(len(CALLS)) for i in range(len(CALLS[c][1]))])
def test_a_tangent_is_refused(call, which):
    run, operands = CALLS[call]
    with forward_ad.dual_level():
        dual = list(operands)
        dual[which] = forward_ad.make_dual(dual[which].clone(), torch.ones_like(dual[which]))
        with pytest.raises(RuntimeError, match="forward"):
            run(*dual)
        with torch.no_grad(), pytest.raises(RuntimeError, match="forward"):
            run(*dual)


@pytest.mark.parametrize("call", range(len(CALLS)))
def test_operands_without_one_pass(call):
    run, operands = CALLS[call]
    with forward_ad.dual_level(), pytest.raises(ValueError, match="GPU"):       # on to the next check: host tensors
        run(*operands)
    with pytest.raises(ValueError, match="GPU"):
        run(*operands)


@pytest.mark.parametrize("function,gradients,which", [(_NormRotate, 1, 0), (_TokenLogprobs, 2, 0), (_TokenLogprobs, 2, 1)])
def test_a_gradient_with_a_tangent_is_refused(function, gradients, which):
    with forward_ad.dual_level():
        given = [None] * gradients
        given[which] = forward_ad.make_dual(ROW.clone(), torch.ones_like(ROW))
        with pytest.raises(RuntimeError, match="forward"):
            function.backward(None, *given)
