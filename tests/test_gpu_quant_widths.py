"""quant_tokens of rows longer than 16,384 elements: every number of vectors a
thread can hold, at the edges of each."""

import pytest

from test_gpu_linear_i8 import test_quant_tokens as _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vectors", range(9, 17))
def test_long_rows(vectors):
    for d in (2048 * (vectors - 1) + 32, 2048 * vectors - 32, 2048 * vectors):
        _check(67, d)
