"""Causal attention over packed prompts (pp.attention) against its formula in
64 bits.

What a result may be off by, with A_i = sum_j p_ij |v_j| / l_i: the weights
p_ij are rounded to bf16 for the product with V (2^-8 A); a score is a sum of
`width` fp32 products, off by at most (width + 2) 2^-24 sum_k |q_k k_k| scale,
and its exponent's argument by two more roundings of at most 2^-24 of the row's
largest score; an error e in the exponent changes p_ij, and l_i, by a factor
1 + e (2 e A together, with the 2^-22 of the exponential); the sums of the
second product and of l_i run over len terms in fp32 (2 len 2^-24 A, kept
below 2^-12 A here); and the result is rounded to bf16 (2^-8 of its value).
"""

import math

import pytest
import torch

import post_pruning_b200 as pp

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _inputs(lens, heads, kv, width, seed=0, extra=0, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed + sum(lens) + heads)
    n = sum(lens) + extra
    Q = (spread * torch.randn(n, heads, width, device=DEV, generator=g)).bfloat16()
    K = (spread * torch.randn(n, kv, width, device=DEV, generator=g)).bfloat16()
    V = torch.randn(n, kv, width, device=DEV, generator=g).bfloat16()
    off = torch.tensor([0] + list(lens), device=DEV).cumsum(0).to(torch.int32)
    return Q, K, V, off


def _check(O, Q, K, V, off, scale=None, causal_rows=None):
    heads, width = Q.shape[1:]
    share = heads // K.shape[1]
    scale = width ** -0.5 if scale is None else scale
    ends = off.tolist()
    for a, b in zip(ends[:-1], ends[1:]):
        n = b - a
        if not n:
            continue
        later = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
        for h in range(heads):
            q, k, v = Q[a:b, h].double(), K[a:b, h // share].double(), V[a:b, h // share].double()
            x = (q @ k.t() * scale).masked_fill(later, -math.inf)
            p = torch.softmax(x, 1)
            o, A = p @ v, p @ v.abs()
            size = (q.abs() @ k.abs().t() * scale).masked_fill(later, 0).amax(1, keepdim=True)
            e = (width + 2 + 2) * 2.0 ** -24 * size + 2.0 ** -22
            tol = (2.0 ** -8 + 2 * e + 2.0 ** -12) * A + 2.0 ** -8 * o.abs()
            err = (O[a:b, h].double() - o).abs()
            assert bool((err <= tol).all()), (a, b, h, float((err / tol).max()))


def _run(Q, K, V, off, scale=None):
    O = torch.full(Q.shape, 7.0, device=DEV).bfloat16()
    info = pp.new_info()
    pp.attention(Q, K, V, off, O, info, scale=scale)
    pp.raise_on_info(info)
    return O


CASES = [
    ([1], 1, 1), ([2], 2, 1), ([127], 2, 2), ([128], 4, 2), ([129], 1, 1), ([255], 3, 1), ([256], 1, 1), ([257], 3, 3),
    ([1, 1, 1, 1, 1], 2, 1), ([5, 0, 130, 0, 0, 1, 384], 6, 2), ([0, 300], 5, 5), ([640, 3], 8, 1),
    ([1, 127, 128, 129, 200, 256, 257, 511], 4, 4), ([1030], 6, 2),
]


@pytest.mark.parametrize("width", [64, 128])
@pytest.mark.parametrize("lens,heads,kv", CASES)
def test_attention(lens, heads, kv, width):
    Q, K, V, off = _inputs(lens, heads, kv, width)
    _check(_run(Q, K, V, off), Q, K, V, off)


@pytest.mark.parametrize("width,heads,kv", [(128, 4, 2), (64, 3, 1)])
def test_attention_longer_prompts(width, heads, kv):
    Q, K, V, off = _inputs([2047, 3100], heads, kv, width, spread=1.5)
    _check(_run(Q, K, V, off), Q, K, V, off)


@pytest.mark.parametrize("spread,scale", [(0.0, None), (6.0, None), (1.0, 3.0), (2.0, 1e-4)])
def test_attention_flat_and_peaked(spread, scale):
    """Equal scores, and scores whose running maximum grows by hundreds."""
    Q, K, V, off = _inputs([700], 2, 1, 128, spread=spread)
    K *= torch.linspace(0.1, 1.0, 700, device=DEV)[:, None, None]      # later keys score higher
    _check(_run(Q, K, V, off, scale), Q, K, V, off, scale)


def test_attention_many_sequences():
    lens = [(7 * i) % 61 for i in range(300)]                             # more than one scan of 32, with empty ones
    Q, K, V, off = _inputs(lens, 2, 1, 64)
    _check(_run(Q, K, V, off), Q, K, V, off)


@pytest.mark.parametrize("heads,kv", [(2, 1), (1, 1)])
def test_attention_many_sequences_of_several_units(heads, kv):
    """Units are taken by length out of 32 sequences after 32; one with bad
    offsets among them is reported, and no row gets a wrong value."""
    lens = [0, 700, 1, 128, 513, 0, 129, 300] * 9
    Q, K, V, off = _inputs(lens, heads, kv, 64)
    want = _run(Q, K, V, off)
    _check(want, Q, K, V, off)
    at = int(off[34])                                                     # inside the second 32
    off[34] = -1
    O = torch.full(Q.shape, 7.0, device=DEV).bfloat16()
    info = pp.new_info()
    pp.attention(Q, K, V, off, O, info)
    assert pp.sync_status(info) == 1                                      # BAD_LENGTHS
    lost = slice(int(off[33]), int(off[35]))                              # both sequences of that offset
    assert at >= lost.start and bool((O[lost] == 7).all())
    # a CTA that sees the error recorded writes nothing: other rows hold their value or what they held
    assert bool(((O == want) | (O == 7)).flatten(1).all())


@pytest.mark.parametrize("heads,kv", [(4, 2), (3, 3)])
def test_attention_strided_rows_and_rows_outside(heads, kv):
    """Q, K and V parts of one buffer, O a part of a wider one; rows before the
    first and behind the last sequence hold NaN, are not read for a result and
    are left as they were."""
    width, lens = 128, [130, 1, 257]
    n = 3 + sum(lens) + 70
    g = torch.Generator(device=DEV).manual_seed(4)
    both = torch.randn(n, (heads + 2 * kv) * width, device=DEV, generator=g).bfloat16()
    both[:3] = float("nan")
    both[3 + sum(lens):] = float("nan")
    Q, K, V = (p.unflatten(1, (-1, width)) for p in both.split([heads * width, kv * width, kv * width], 1))
    off = (3 + torch.tensor([0] + lens, device=DEV).cumsum(0)).to(torch.int32)
    wide = torch.full((n, (heads + 1) * width), 7.0, device=DEV).bfloat16()
    O = wide[:, :heads * width].unflatten(1, (heads, width))
    info = pp.new_info()
    pp.attention(Q, K, V, off, O, info)
    pp.raise_on_info(info)
    _check(O, Q, K, V, off)
    outside = torch.ones(n, dtype=torch.bool, device=DEV)
    outside[3:3 + sum(lens)] = False
    assert bool((wide[outside] == 7).all()) and bool((wide[:, heads * width:] == 7).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("heads,kv", [(2, 1), (1, 1)])
def test_attention_rows_between_sequences_do_not_reach(value, heads, kv):
    """Sequences on both sides of rows full of NaN or infinities give what they
    give without them; the rows as a sequence of their own are reported."""
    Q, K, V, off = _inputs([100, 60, 200], heads, kv, 64)
    clean = _run(Q, K, V, off)
    for t in (Q, K, V):
        t[100:160] = value
    for a, b in ((0, 100), (160, 360)):
        O = _run(Q, K, V, torch.tensor([a, b], dtype=torch.int32, device=DEV))
        assert torch.equal(O[a:b], clean[a:b]) and bool((O[100:160] == 7).all())
    info = pp.new_info()
    pp.attention(Q, K, V, off, O, info)
    assert pp.sync_status(info) == 3                                      # NONFINITE


@pytest.mark.parametrize("offsets", [[0, 50, 40, 100], [0, 50, 101], [-1, 50, 100], [0, 2 ** 31 - 1, 100]])
def test_attention_bad_offsets(offsets):
    Q, K, V, _ = _inputs([100], 2, 2, 64)
    wide = torch.full((140, 2, 64), 7.0, device=DEV).bfloat16()
    info = pp.new_info()
    pp.attention(Q, K, V, torch.tensor(offsets, dtype=torch.int32, device=DEV), wide[20:120], info)
    assert pp.sync_status(info) == 1                                      # BAD_LENGTHS
    assert bool((wide[:20] == 7).all()) and bool((wide[120:] == 7).all())


def test_attention_nothing_to_do():
    info = pp.new_info()
    e = torch.empty(0, 2, 64, device=DEV, dtype=torch.bfloat16)
    before = pp.kernel_launches()
    pp.attention(e, e, e, torch.zeros(3, dtype=torch.int32, device=DEV), e.clone(), info)
    Q, K, V, _ = _inputs([10], 2, 2, 64)
    pp.attention(Q, K, V, torch.zeros(1, dtype=torch.int32, device=DEV), torch.empty_like(Q), info)
    assert pp.kernel_launches() == before and pp.sync_status(info) == 0


def test_attention_repeats_streams_and_capture():
    lens = [400, 33, 260]
    sets = [_inputs(lens, 8, 2, 128, seed=i) for i in range(3)]
    want = [_run(*s) for s in sets]
    outs, infos = [torch.empty_like(want[0]) for _ in range(2)], [pp.new_info(), pp.new_info()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                pp.attention(*sets[i], outs[i], infos[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    held = [t.clone() for t in sets[0]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pp.attention(*held, outs[0], infos[0])
    for i in (1, 2, 1):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[i])
    # other lengths of the same packed rows, without another capture
    held[3].copy_(torch.tensor([0, 1, 600, 693], dtype=torch.int32, device=DEV))
    g.replay()
    torch.cuda.synchronize()
    _check(outs[0], *held)


def test_attention_wait_times_out():
    Q, K, V, off = _inputs([1000], 4, 2, 128)
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
