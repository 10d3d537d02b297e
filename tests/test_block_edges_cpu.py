"""Edges of the argument checks of the operators around a block's allreduce, without a GPU."""
import pytest

from test_block_ops_cpu import ARG, NULL, OK, combine, combine_bwd, dispatch, gemm, norm, quant


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(dr=None)), (NULL, dict(kept=None)), (ARG, dict(lddr=8)), (ARG, dict(nrows=1 << 31)),
    (OK, dict(nrows=0, dr=None, kept=None, slots=None, g=None, rows=None, weights=None, dw=None)),
    (OK, dict(hidden=0, dr=None, kept=None, slots=None, g=None, rows=None, weights=None, dw=None)),
])
def test_combine_backward_without_tokens(want, kw):
    assert combine_bwd(tokens=0, **kw) == want


# The limits that rx.h states, from both sides. Calls without data are accepted without a launch.
@pytest.mark.parametrize("call,inside,outside", [
    (norm, dict(rows=0, hidden=32768), dict(rows=0, hidden=32769)),
    (gemm, dict(rows=(1 << 22) - 1, n=0), dict(rows=1 << 22, n=0)),
    (gemm, dict(rows=0, n=4194295 * 256), dict(rows=0, n=4194296 * 256)),   # two tiles' rows of 2^22 - 9, 2^22 - 8
    (gemm, dict(rows=0, k=131071, lda=131072, ldb=131072), dict(rows=0, k=131072, lda=131072, ldb=131072)),
    (combine, dict(tokens=0, nrows=(1 << 31) - 1), dict(tokens=0, nrows=1 << 31)),
    (combine, dict(tokens=0, ldr=1 << 36), dict(tokens=0, ldr=(1 << 36) + 1)),
    (combine, dict(tokens=0, hidden=1 << 30, ldr=1 << 30), dict(tokens=0, hidden=(1 << 30) + 1, ldr=1 << 31)),
    (quant, dict(rows=0, k=1 << 30), dict(rows=0, k=(1 << 30) + 1)),
])
def test_limits_of_the_sizes(call, inside, outside):
    assert call(**inside) == OK and call(**outside) == ARG


@pytest.mark.parametrize("tokens,hidden", [((1 << 22) - 1, 4097), (1 << 16, 1 << 18)])
def test_combine_refuses_more_waves_than_a_launch_has(tokens, hidden):
    assert combine(tokens=tokens, hidden=hidden, ldr=1 << 20, ldo=1 << 20) == ARG


def test_dispatch_refuses_more_pairs_than_32_bits_number():
    assert dispatch(tokens=(1 << 22) - 1, topk=64) == NULL   # a plan of this size needs a workspace
    assert dispatch(tokens=1 << 22, topk=64) == ARG
