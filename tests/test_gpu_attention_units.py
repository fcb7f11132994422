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


@pytest.mark.parametrize("heads,kv,width", [(16, 4, 128), (7, 7, 64)])
def test_attention_bad_offsets_in_a_crowded_launch(heads, kv, width):
    """Bad offsets are reported whichever CTAs of the launch start and whichever
    are taken: the SMs are still full of another stream's launch."""
    lens = [200, 129, 1, 300] * 12
    Q, K, V, off = _inputs(lens, heads, kv, width)
    other = _inputs([2000] * 4, 8, 8, 128, seed=1)
    away = torch.empty_like(other[0])
    streams, infos = [torch.cuda.Stream(), torch.cuda.Stream()], [pp.new_info(), pp.new_info()]
    for i in (0, 20, len(lens) - 1):
        bad = off.clone()
        bad[i + 1] = off[-1] + 1 if i + 1 == len(lens) else off[i] - 1
        torch.cuda.synchronize()
        for _ in range(5):
            pp.info_clear(infos[1], stream=streams[1])
            with torch.cuda.stream(streams[0]):
                pp.attention(*other, away, infos[0])
            with torch.cuda.stream(streams[1]):
                O = torch.empty_like(Q)
                pp.attention(Q, K, V, bad, O, infos[1])
            assert pp.sync_status(infos[1], streams[1]) == 1                  # BAD_LENGTHS
    torch.cuda.synchronize()
    assert pp.sync_status(infos[0]) == 0
