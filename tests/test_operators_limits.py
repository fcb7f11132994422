"""Calls at the edge of what the 8-bit forward, the attention and the
attention-block driver take, as far as they are answered without a GPU."""

import pytest

from test_operators_abi import ATTN, INVALID, _block, _call


@pytest.mark.parametrize("n_seq", [(1 << 30) + 1, (1 << 31) - 33, (1 << 31) - 1])
def test_sequences_are_counted_in_strides_of_32(n_seq):
    """Kernels walk the sequences 32 at a time in an int: the number plus a
    stride has to stay inside it, or they read before the offsets."""
    assert _call("sgpt_attention", ATTN, n_seq=n_seq) == INVALID
    assert _block(n_seq=n_seq) == INVALID
