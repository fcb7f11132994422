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


# several hundred CTAs of several blocks each: units of two heads (an even group) and of two row tiles (an odd one),
# one-tile and two-tile units of very different lengths in turn, ends inside a tile
LENS = [900, 129, 700, 1, 640] * 4
SHAPES = [(16, 2, 128), (16, 2, 64), (12, 12, 128), (12, 12, 64), (9, 3, 128), (9, 3, 64)]


@pytest.mark.parametrize("heads,kv,width", SHAPES)
def test_attention_several_units_per_cta(heads, kv, width):
    """Values, and the same bits again after a launch on other inputs in
    between: which CTA takes which unit differs from launch to launch."""
    Q, K, V, off = _inputs(LENS, heads, kv, width)
    want = _run(Q, K, V, off)
    _check(want, Q, K, V, off)
    other = _inputs(LENS[::-1], heads, kv, width, seed=9)
    for _ in range(5):
        _run(*other)
        assert torch.equal(_run(Q, K, V, off), want)


@pytest.mark.parametrize("heads,kv,width", SHAPES)
def test_attention_several_units_of_rising_scores(heads, kv, width):
    """The running maximum moves in most blocks, so results are rescaled while
    the other tile's scores, or the next unit's, are under way; rows of one
    buffer, and rows of NaN behind the last sequence."""
    g = torch.Generator(device=DEV).manual_seed(heads)
    n = sum(LENS)
    buf = torch.randn(n + 40, (heads + 2 * kv) * width, device=DEV, generator=g)
    buf[:n, heads * width:(heads + kv) * width] *= torch.cat([torch.linspace(0.05, 3.0, m) for m in LENS]).to(DEV)[:, None]
    buf[n:] = float("nan")
    Q, K, V = (t.unflatten(1, (-1, width)) for t in
               buf.bfloat16().split([heads * width, kv * width, kv * width], 1))
    off = torch.tensor([0] + LENS, device=DEV).cumsum(0).to(torch.int32)
    O = _run(Q, K, V, off)
    _check(O, Q, K, V, off)
    assert bool((O[n:] == 7).all())


@pytest.mark.parametrize("heads,kv,width", [(16, 2, 128), (9, 3, 64)])
def test_attention_several_units_time_out(heads, kv, width):
    """A wait that runs out in a launch whose CTAs take others' units."""
    Q, K, V, off = _inputs(LENS, heads, kv, width)
    want = _run(Q, K, V, off)
    O = torch.empty_like(want)
    info = pp.new_info()
    pp.set_wait_limit(1)
    try:
        pp.attention(Q, K, V, off, O, info)
        assert pp.sync_status(info) == 4                                  # TIMEOUT
    finally:
        pp.set_wait_limit(0)
    pp.info_clear(info)
    pp.attention(Q, K, V, off, O, info)
    pp.raise_on_info(info)
    assert torch.equal(O, want)


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
