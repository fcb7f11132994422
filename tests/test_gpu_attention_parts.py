"""pp.attention where few heads and long prompts leave SMs idle: clusters of 2, 4
or 8 CTAs take a part of the keys each and join their results.

The bound is test_gpu_attention's. Joining adds to the exponent's argument two
roundings of 2^-24 of the largest score and to the exponential one more 2^-22,
but the fp32 sums then run over at most len / 2 + 8 terms instead of len: at
len <= 3100 they take 2^-23 (1550 + 8) < 1.9e-4 of the 2^-12 that the bound has
for them, and the 5.8e-5 left hold twice the join's error, 2 (2 2^-24 size +
2^-22), for scores up to 200 (here below 40).
"""

import pytest
import torch

import post_pruning_b200 as pp
from test_gpu_attention import DEV, _check, _inputs, _run

pytestmark = pytest.mark.gpu

CASES = [
    ([3000], 8, 2), ([2561], 4, 4),                                  # two parts
    ([513], 4, 4), ([1030], 6, 2), ([2047], 2, 1), ([1153], 3, 1),   # four
    ([1025], 1, 1), ([1407], 2, 1), ([767], 4, 4), ([2176], 1, 1),   # eight
    ([1500, 1, 130, 0], 1, 1), ([1, 1281, 0, 257], 2, 1), ([40, 900, 128], 2, 2),    # parts without keys
]


@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("lens,heads,kv", CASES)
def test_parts(lens, heads, kv, width):
    Q, K, V, off = _inputs(lens, heads, kv, width)
    _check(_run(Q, K, V, off), Q, K, V, off)


@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("spread,scale", [(0.0, None), (2.0, 1e-4), (1.0, 0.5)])
def test_parts_of_rising_and_falling_scores(spread, scale, width):
    """The largest weights in the last part, in the first one, or spread evenly."""
    for rising in (True, False):
        Q, K, V, off = _inputs([1300], 1, 1, width, spread=spread)
        ramp = torch.linspace(0.02, 1.0, 1300, device=DEV)
        K *= (ramp if rising else ramp.flip(0))[:, None, None]
        _check(_run(Q, K, V, off, scale=scale), Q, K, V, off, scale=scale)


@pytest.mark.parametrize("heads,kv,width", [(1, 1, 64), (2, 1, 128)])
def test_parts_strided_rows_and_rows_outside(heads, kv, width):
    n, lens = 1400, [1000, 101]
    g = torch.Generator(device=DEV).manual_seed(5)
    buf = torch.randn(n, (heads + 2 * kv) * width + 16, device=DEV, generator=g).bfloat16()
    Q = buf[:, :heads * width].unflatten(1, (heads, width))
    K = buf[:, heads * width:(heads + kv) * width].unflatten(1, (kv, width))
    V = buf[:, (heads + kv) * width:(heads + 2 * kv) * width].unflatten(1, (kv, width))
    first = 77
    off = torch.tensor([first, first + lens[0], first + sum(lens)], device=DEV, dtype=torch.int32)
    buf[:first] = float("nan")
    buf[first + sum(lens):] = float("nan")
    wide = torch.full((n, heads * width + 8), 7.0, device=DEV).bfloat16()
    O = wide[:, :heads * width].unflatten(1, (heads, width))
    info = pp.new_info()
    pp.attention(Q, K, V, off, O, info)
    pp.raise_on_info(info)
    assert bool((O[:first] == 7).all()) and bool((O[first + sum(lens):] == 7).all())
    assert bool((wide[:, heads * width:] == 7).all())
    _check(O, Q, K, V, off)


@pytest.mark.parametrize("row", [3, 700, 1299])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_parts_report_what_is_not_finite(row, value):
    """A bad value of V reaches its own and later rows, which are reported, and
    no block of 128 rows before its own."""
    Q, K, V, off = _inputs([1300], 1, 1, 64)
    want = _run(Q, K, V, off)
    V[row] = value
    O = torch.empty_like(Q)
    info = pp.new_info()
    pp.attention(Q, K, V, off, O, info)
    assert pp.sync_status(info) == 3                                      # NONFINITE
    first = row // 128 * 128
    assert torch.equal(O[:first], want[:first])
    assert not bool(torch.isfinite(O[row:].float()).any())


@pytest.mark.parametrize("offsets", [[0, 1301], [0, 1200, 1100], [-1, 1300], [0, 2 ** 31 - 1, 1300]])
def test_parts_bad_offsets(offsets):
    Q, K, V, _ = _inputs([1300], 1, 1, 64)
    wide = torch.full((1340, 1, 64), 7.0, device=DEV).bfloat16()
    info = pp.new_info()
    pp.attention(Q, K, V, torch.tensor(offsets, dtype=torch.int32, device=DEV), wide[20:1320], info)
    assert pp.sync_status(info) == 1                                      # BAD_LENGTHS
    assert bool((wide[:20] == 7).all()) and bool((wide[1320:] == 7).all())


def test_parts_repeat_on_streams_and_in_a_graph():
    sets = [_inputs([1500, 20], 2, 1, 128, seed=i) for i in range(3)]
    want = [_run(*s) for s in sets]
    outs = [torch.zeros_like(s[0]) for s in sets]
    info = pp.new_info()
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for st, s, o in zip(streams, sets, outs):                         # two launches at once
        with torch.cuda.stream(st):
            for _ in range(5):
                pp.attention(*s, o, info)
    torch.cuda.synchronize()
    pp.raise_on_info(info)
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for s, o in zip(sets, outs):
            pp.attention(*s, o, info)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    pp.raise_on_info(info)
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    # the same captured launch for other lengths of the same rows
    Q, K, V, off = sets[0]
    for lens in ([1520, 0], [3, 1517], [700, 600]):
        off.copy_(torch.tensor([0] + lens, device=DEV).cumsum(0))
        outs[0].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        pp.raise_on_info(info)
        _check(outs[0], Q, K, V, off)


@pytest.mark.parametrize("heads,kv,width", [(1, 1, 64), (2, 1, 128), (8, 2, 64)])
def test_parts_wait_times_out(heads, kv, width):
    Q, K, V, off = _inputs([1000], heads, kv, width)
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
