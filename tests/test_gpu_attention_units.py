"""pp.attention where CTAs take the units of CTAs that have not started: several
units of several blocks each per CTA, so that operands are refilled, the next
unit's first scores start under the last ones of the unit before, and the ring
of K and V blocks goes on from unit to unit.

The bound is test_gpu_attention's (its lengths and score sizes hold here too).
"""

import pytest
import torch

import post_pruning_b200 as pp
from test_gpu_attention import DEV, _check, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,kv,width", [(16, 4, 128), (8, 8, 64)])
def test_attention_more_ctas_than_units(heads, kv, width):
    """The launch has a CTA for every unit that the lengths could give; here
    most of them find no unit, and one CTA takes many of those one after the
    other. Every repetition gives the same bits."""
    lens = [1] * 150 + [129, 0, 2, 300]
    Q, K, V, off = _inputs(lens, heads, kv, width)
    packed = torch.zeros(2000, dtype=torch.int32, device=DEV)            # the same sequences, then empty ones
    packed[:off.numel()] = off
    packed[off.numel():] = off[-1]
    want = _run(Q, K, V, off)
    _check(want, Q, K, V, off)
    for _ in range(20):
        assert torch.equal(_run(Q, K, V, packed), want)
