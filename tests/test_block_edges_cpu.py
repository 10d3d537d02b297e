"""Edges of the argument checks of the operators around a block's allreduce, without a GPU."""
import pytest

from test_block_ops_cpu import ARG, NULL, OK, combine_bwd


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(dr=None)), (NULL, dict(kept=None)), (ARG, dict(lddr=8)), (ARG, dict(nrows=1 << 31)),
    (OK, dict(nrows=0, dr=None, kept=None, slots=None, g=None, rows=None, weights=None, dw=None)),
    (OK, dict(hidden=0, dr=None, kept=None, slots=None, g=None, rows=None, weights=None, dw=None)),
])
def test_combine_backward_without_tokens(want, kw):
    assert combine_bwd(tokens=0, **kw) == want
