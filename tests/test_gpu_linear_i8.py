"""The 8-bit forward (quant_codes, quant_tokens, quant_tokens_silu, linear_i8)
against its definition in 64 bits.

What each check allows: codes, sums and the integer products are exact, so
they are compared as whole numbers; a scale is one IEEE division; a result is
the exact integer rounded to fp32 and two fp32 products, 3 * 2^-24 of its
value, plus 2^-8 of it for a bf16 result. A gated value z = g / (1 + e^-g) * u
carries the two ulp (2^-22) of expf, through 1 + e^-g at most as much again
relative to z, and the roundings of the sum, the quotient and the product
(2^-24 each): 6 * 2^-23 covers it, once for z and once for the row's largest.
"""

import numpy as np
import pytest
import torch

import post_pruning_b200 as pp

pytestmark = pytest.mark.gpu

DEV = "cuda"
Z_REL = 6 * 2.0 ** -23


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _tokens(n, d, guard=0):
    """Output buffers, `guard` rows longer than they need to be."""
    return (torch.full((n + guard, d), 99, dtype=torch.int8, device=DEV)[:n],
            torch.full((n + guard,), -1.0, device=DEV)[:n],
            torch.full((n + guard,), -7, dtype=torch.int32, device=DEV)[:n])


def _codes64(z, top):
    top = torch.where(top == 0, torch.ones_like(top), top)
    return torch.round(127 * z / top[:, None])


def _check_tokens(X, q, s, t):
    x = X.double()
    top = x.abs().amax(1)
    ref = _codes64(x, top)
    assert torch.equal(q.double(), ref)
    assert torch.equal(s, (top / 127).float())           # bf16 / 127 in 64 bits, then 32: no tie is near
    assert torch.equal(t.long(), q.long().sum(1))


# both sides of every width at which more threads share a row, few rows (a cluster each above 4096) and many
@pytest.mark.parametrize("n,d", [(1, 32), (9, 96), (1, 1024), (3, 1056), (200, 4096), (1, 4128), (17, 5120), (2, 8192),
                                 (5, 8224), (1, 25600), (64, 32768), (65, 5120), (70, 8224), (66, 16416), (65, 26624),
                                 (66, 26656), (65, 32768), (2000, 768)])
def test_quant_tokens(n, d):
    g = _gen(n + d)
    X = (torch.randn(n, d, device=DEV, generator=g) * torch.exp(2 * torch.randn(d, device=DEV, generator=g))).bfloat16()
    X[n // 2] = 0 if n > 4 else X[n // 2]
    q, s, t = _tokens(n, d)
    info = pp.new_info()
    pp.quant_tokens(X, q, s, t, info)
    pp.raise_on_info(info)
    _check_tokens(X, q, s, t)


# every number of vectors per thread, a row per warp (many rows) and per CTA
@pytest.mark.parametrize("n,d", [(21, 256), (21, 288), (20, 544), (19, 800), (130, 1056), (130, 2080), (66, 3104), (66, 6176),
                                 (66, 8224), (66, 10272), (66, 12320), (66, 14368), (66, 16384)] +
                         [(n, d) for n in (4095, 4096, 4101) for d in (1056, 1280, 1312, 1568, 1824, 2048, 2080)])
def test_quant_tokens_vectors(n, d):
    test_quant_tokens(n, d)
    test_quant_tokens_silu(n, d, True)


@pytest.mark.parametrize("n,d", [(65, 20480), (65, 20512), (300, 24576), (300, 24608), (65, 28672), (65, 28704)])
def test_quant_tokens_silu_long_rows(n, d):
    test_quant_tokens_silu(n, d, False)


def test_quant_tokens_ties_and_extremes():
    """Every bf16 magnitude against largest values that make exact ties
    (254 x an odd multiple of the largest), and rows of huge, tiny and
    subnormal values."""
    d = 32768 // 2
    every = torch.arange(0, 0x7f80, device=DEV, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)   # all >= 0
    rows = []
    for top in (1.0, 127.0, 254.0, 2.0 ** 100, 3.0e38, 2.0 ** 119, 2.0 ** 120, 1.0e-30, 2.0 ** -126):
        v = every[every.float() <= torch.tensor(top, device=DEV).bfloat16().float()]
        v = v[-(d - 1):]
        row = torch.zeros(d, device=DEV, dtype=torch.bfloat16)
        row[:v.numel()] = v
        row[1::2] = -row[1::2]
        row[-1] = top
        rows.append(row)
    halves = torch.arange(0, 254, device=DEV).float().mul(0.5)           # k + 1/2 of a largest 127
    row = torch.zeros(d, device=DEV)
    row[:254] = halves
    row[254:508] = -halves
    row[-1] = 127.0
    rows.append(row.bfloat16())
    X = torch.stack(rows)
    n = X.shape[0]
    q, s, t = _tokens(n, d)
    info = pp.new_info()
    pp.quant_tokens(X, q, s, t, info)
    pp.raise_on_info(info)
    _check_tokens(X, q, s, t)


def test_quant_tokens_strided_rows_and_guards():
    g = _gen(5)
    wide = torch.randn(37, 3 * 640, device=DEV, generator=g).bfloat16()
    X = wide[:, 640:1280]
    q, s, t = _tokens(37, 640, guard=3)
    info = pp.new_info()
    pp.quant_tokens(X, q, s, t, info)
    pp.raise_on_info(info)
    _check_tokens(X, q, s, t)
    assert bool((q._base[37:] == 99).all()) and bool((s._base[37:] == -1).all()) and bool((t._base[37:] == -7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("gated", [False, True])
def test_non_finite_tokens_are_reported(bad, gated):
    X = torch.ones(12, 1536, device=DEV).bfloat16()
    X[7, 1531] = bad
    q, s, t = _tokens(12, 1536)
    info = pp.new_info()
    if gated:
        pp.quant_tokens_silu(X, torch.ones_like(X), q, s, t, info)
    else:
        pp.quant_tokens(X, q, s, t, info)
    assert pp.sync_status(info) == 3                      # NONFINITE
    assert bool(torch.isnan(s[7])) and not bool(q[7].any())
    # a later call sees the recorded error and leaves its outputs alone
    y = torch.full((12, 64), 5.0, device=DEV)
    pp.linear_i8(q, s, t, torch.zeros(64, 1536, dtype=torch.int8, device=DEV), torch.ones(64, 2, device=DEV), y, info)
    assert pp.sync_status(info) == 3 and bool((y == 5).all())


@pytest.mark.parametrize("n,d,strided", [(1, 64, False), (11, 768, True), (3, 5120, False), (2, 25600, True), (1, 32768, False),
                                         (65, 4128, True), (66, 8224, False), (65, 16416, True), (65, 32768, False)])
def test_quant_tokens_silu(n, d, strided):
    g = _gen(3 * n + d)
    if strided:
        both = (3 * torch.randn(n, 2 * d, device=DEV, generator=g)).bfloat16()
        G, U = both[:, :d], both[:, d:]
    else:
        G = (3 * torch.randn(n, d, device=DEV, generator=g)).bfloat16()
        U = (3 * torch.randn(n, d, device=DEV, generator=g)).bfloat16()
    G[0, :8] = torch.tensor([-200.0, -90.0, 90.0, 0.0, -0.0, 1e-30, -1e30, 88.0], device=DEV).bfloat16()
    U[0, :8] = 1.0
    q, s, t = _tokens(n, d)
    info = pp.new_info()
    pp.quant_tokens_silu(G, U, q, s, t, info)
    pp.raise_on_info(info)
    g64 = G.double()
    z = g64 * torch.sigmoid(g64) * U.double()
    top = z.abs().amax(1)
    assert bool(((s.double() - top / 127).abs() <= (Z_REL + 2.0 ** -24) * top / 127).all())
    off = (q.double() - 127 * z / top[:, None]).abs()
    assert float(off.max()) <= 0.5 + 127 * (2 * Z_REL + 2 * 2.0 ** -24)
    assert torch.equal(t.long(), q.long().sum(1))


@pytest.mark.parametrize("d", [96, 512 * 56])                # a row per warp; rows in shared memory
@pytest.mark.parametrize("size", [1e-37, 3e-38, 1e-30, 1e-25, 1e30, 3e38])
def test_quant_tokens_silu_extremes(d, size):
    """Rows whose gated values are all tiny or huge: 127 / max and 127 z stay
    inside fp32. (Values this small are short of bits in fp32: the codes are
    checked against the fp32 values u, where silu(g) is 1 to the last bit.)"""
    g = _gen(d)
    n = 70
    G = torch.full((n, d), 64.0, device=DEV).bfloat16()               # silu(64) = 64
    U = ((torch.rand(n, d, device=DEV, generator=g) * 2 - 1) * (size / 64)).bfloat16()
    q, s, t = _tokens(n, d)
    info = pp.new_info()
    pp.quant_tokens_silu(G, U, q, s, t, info)
    pp.raise_on_info(info)
    z = U.double() * 64
    top = z.abs().amax(1)
    off = (q.double() - 127 * z / top[:, None]).abs()
    assert float(off.max()) <= 0.5 + 127 * (2 * Z_REL + 2 * 2.0 ** -24)
    assert bool(((s.double() - top / 127).abs() <= Z_REL * top / 127 + 2.0 ** -149).all())
    assert torch.equal(t.long(), q.long().sum(1))


@pytest.mark.parametrize("qbits", [2, 4, 8])
def test_quant_codes_stand_for_the_grid(qbits):
    """Codes of arbitrary weights are the nearest levels, and codes of weights
    that lie on the grid stand for them exactly."""
    g = _gen(qbits)
    r, d = 77, 160
    W = torch.randn(r, d + 32, device=DEV, generator=g)[:, :d]
    W[3] = 0
    grid = torch.empty(r, 2, device=DEV)
    pp.quant_grid(W, qbits, grid)
    codes = torch.full((r, d), 100, dtype=torch.int8, device=DEV)
    info = pp.new_info()
    pp.quant_codes(W, grid, codes, info, qbits=qbits)
    pp.raise_on_info(info)
    half = 2 ** (qbits - 1)
    w32 = W.cpu().numpy()
    scale, zero = grid.cpu().numpy()[:, :1], grid.cpu().numpy()[:, 1:]
    ref = np.clip(np.rint(w32 / scale) + zero, 0, 2 ** qbits - 1) - half            # IEEE fp32, ties to even
    assert np.array_equal(codes.cpu().numpy().astype(np.float32), ref)
    level = grid[:, :1] * (codes.float() + half - grid[:, 1:])                       # fp32, as the sweep forms it
    again = torch.empty_like(codes)
    pp.quant_codes(level.contiguous(), grid, again, info, qbits=qbits)
    pp.raise_on_info(info)
    assert torch.equal(codes, again)


def test_quant_codes_non_finite():
    W = torch.randn(8, 64, device=DEV)
    grid = torch.empty(8, 2, device=DEV)
    pp.quant_grid(W, 8, grid)
    W[5, 60] = float("nan")
    codes = torch.empty(8, 64, dtype=torch.int8, device=DEV)
    info = pp.new_info()
    pp.quant_codes(W, grid, codes, info)
    assert pp.sync_status(info) == 3


def _problem(n, d_in, d_out, qbits=8, seed=0, full=False):
    g = _gen(seed + n + d_in + d_out)
    lo, hi = -2 ** (qbits - 1), 2 ** (qbits - 1)
    if full:                                              # the largest magnitudes an int32 has to hold
        codes = torch.full((d_out, d_in), lo, dtype=torch.int8, device=DEV)
        q = torch.full((n, d_in), 127, dtype=torch.int8, device=DEV)
        zero = torch.full((d_out,), float(2 ** qbits - 1), device=DEV)
    else:
        codes = torch.randint(lo, hi, (d_out, d_in), device=DEV, generator=g).to(torch.int8)
        q = torch.randint(-127, 128, (n, d_in), device=DEV, generator=g).to(torch.int8)
        zero = torch.randint(0, 2 ** qbits, (d_out,), device=DEV, generator=g).float()
    grid = torch.stack([torch.rand(d_out, device=DEV, generator=g) + 0.01, zero], 1).contiguous()
    s = torch.rand(n, device=DEV, generator=g) + 0.01
    t = q.long().sum(1).to(torch.int32)
    w = codes.double() - (zero.double()[:, None] - 2 ** (qbits - 1))
    whole = q.double() @ w.t()                            # exact: below 2^53
    return q, s, t, codes, grid, whole


def _check_linear(Y, whole, s, grid):
    ref = whole * s.double()[:, None] * grid[:, 0].double()
    tol = 3.1 * 2.0 ** -24 + (2.0 ** -8 if Y.dtype == torch.bfloat16 else 0.0)
    err = (Y.double() - ref).abs()
    assert bool((err <= tol * ref.abs()).all()), float((err / ref.abs().clamp(min=1e-30)).max())


SHAPES = [(1, 32, 1), (1, 5120, 1024), (2, 96, 130), (16, 4096, 257), (17, 160, 128), (32, 1024, 384), (33, 320, 1000),
          (64, 768, 768), (65, 2048, 100), (128, 640, 513), (129, 256, 129), (300, 11008, 256), (513, 128, 2000),
          (1000, 768, 8), (2049, 544, 777)]


@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_i8(n, d_in, d_out, dtype):
    q, s, t, codes, grid, whole = _problem(n, d_in, d_out)
    buf = torch.full((n + 2, d_out), -3.0, device=DEV, dtype=dtype)
    Y = buf[:n]
    info = pp.new_info()
    pp.linear_i8(q, s, t, codes, grid, Y, info)
    pp.raise_on_info(info)
    _check_linear(Y, whole, s, grid)
    assert bool((buf[n:] == -3).all())


# one shape for every tile and number of parts of K that the plan can choose
VARIANTS = [(3, 160, 177), (7, 3232, 110), (2, 4416, 115), (1, 16736, 103), (506, 160, 521), (608, 3552, 130),
            (321, 5440, 171), (146, 28832, 130), (429, 128, 2740), (599, 4672, 386), (602, 7904, 129), (330, 24544, 130),
            (460, 128, 11952), (65, 4704, 6305), (216, 128, 10599), (134, 16640, 4707)]


@pytest.mark.parametrize("n,d_in,d_out", VARIANTS)
def test_linear_i8_every_variant(n, d_in, d_out):
    q, s, t, codes, grid, whole = _problem(n, d_in, d_out, seed=3)
    info = pp.new_info()
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((n + 2, d_out), -3.0, device=DEV, dtype=dtype)
        pp.linear_i8(q, s, t, codes, grid, buf[:n], info)
        pp.raise_on_info(info)
        _check_linear(buf[:n], whole, s, grid)
        assert bool((buf[n:] == -3).all())


@pytest.mark.parametrize("n,d_in,d_out", [(384, 1024, 3101), (300, 2048, 4001), (384, 8224, 1542), (383, 8224, 1541)])
def test_linear_i8_pairs_on_128_tokens(n, d_in, d_out):
    """Pairs on tiles of 128 tokens, K in one part and in two, and their timeouts."""
    test_linear_i8_every_variant(n, d_in, d_out)
    test_linear_i8_wait_times_out(n, d_in, d_out)


@pytest.mark.parametrize("n,d_in,d_out", [(475, 5280, 523), (290, 9120, 387), (194, 29440, 290), (845, 1056, 1285),
                                          (789, 5280, 645), (200, 25600, 5001), (17, 20608, 2050), (50, 14336, 1000)])
def test_linear_i8_wide_tiles_with_k_split(n, d_in, d_out):
    """Tiles of 64 tokens with K in two, four and eight, pairs on 128 and 256
    tokens with K in one and two, a few tokens of long rows."""
    test_linear_i8_every_variant(n, d_in, d_out)
    test_linear_i8_wait_times_out(n, d_in, d_out)


@pytest.mark.parametrize("n", [1, 24, 200])
def test_linear_i8_many_tiles_per_cta(n):
    q, s, t, codes, grid, whole = _problem(n, 256, 60000)
    Y = torch.empty(n, 60000, device=DEV)
    info = pp.new_info()
    pp.linear_i8(q, s, t, codes, grid, Y, info)
    pp.raise_on_info(info)
    _check_linear(Y, whole, s, grid)


@pytest.mark.parametrize("qbits", [2, 4, 8])
def test_linear_i8_largest_sums(qbits):
    q, s, t, codes, grid, whole = _problem(3, 32768, 160, qbits=qbits, full=True)
    Y = torch.empty(3, 160, device=DEV)
    info = pp.new_info()
    pp.linear_i8(q, s, t, codes, grid, Y, info, qbits=qbits)
    pp.raise_on_info(info)
    _check_linear(Y, whole, s, grid)


def test_no_tokens():
    info = pp.new_info()
    q, s, t = _tokens(0, 64)
    before = pp.kernel_launches()
    pp.quant_tokens(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), q, s, t, info)
    pp.linear_i8(q, s, t, torch.zeros(8, 64, dtype=torch.int8, device=DEV), torch.ones(8, 2, device=DEV),
                 torch.empty(0, 8, device=DEV), info)
    assert pp.kernel_launches() == before and pp.sync_status(info) == 0


def test_results_repeat_and_capture():
    """Two calls at once on two streams with their own buffers, and a captured
    and replayed call on new inputs, give the bits of a plain call."""
    def call(X, bufs, w, info):
        q, s, t, Y = bufs
        pp.quant_tokens(X, q, s, t, info)
        pp.linear_i8(q, s, t, *w, Y, info)

    n, d_in, d_out = 40, 4096, 1100
    _, _, _, codes, grid, _ = _problem(1, d_in, d_out)
    Xs = [torch.randn(n, d_in, device=DEV, generator=_gen(i)).bfloat16() for i in range(3)]
    bufs = [(*_tokens(n, d_in), torch.empty(n, d_out, device=DEV)) for _ in range(2)]
    info = [pp.new_info(), pp.new_info()]
    want = []
    for X in Xs:
        call(X, bufs[0], (codes, grid), info[0])
        want.append(bufs[0][3].clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(Xs[i], bufs[i], (codes, grid), info[i])
    torch.cuda.synchronize()
    assert torch.equal(bufs[0][3], want[0]) and torch.equal(bufs[1][3], want[1])
    X = Xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(X, bufs[0], (codes, grid), info[0])
    for i in (1, 2, 1):
        X.copy_(Xs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[0][3], want[i])


@pytest.mark.parametrize("n,d_in,d_out", [(600, 2048, 640), (2, 4416, 115), (65, 4704, 6305), (216, 512, 10599)])
def test_linear_i8_wait_times_out(n, d_in, d_out):
    """A wait that runs out is reported, leaves the GPU usable, and the same
    call succeeds again: single CTAs, a cluster, pairs, pairs with K in two."""
    q, s, t, codes, grid, whole = _problem(n, d_in, d_out)
    Y = torch.empty(n, d_out, device=DEV)
    info = pp.new_info()
    pp.set_wait_limit(1)
    try:
        pp.linear_i8(q, s, t, codes, grid, Y, info)
        assert pp.sync_status(info) == 4                  # TIMEOUT
    finally:
        pp.set_wait_limit(0)
    pp.info_clear(info)
    pp.linear_i8(q, s, t, codes, grid, Y, info)
    pp.raise_on_info(info)
    _check_linear(Y, whole, s, grid)


def test_gated_rows_wait_times_out():
    """The copies of long gated rows, as above."""
    G = torch.randn(200, 25600, device=DEV, generator=_gen(6)).bfloat16()
    q, s, t = _tokens(200, 25600)
    info = pp.new_info()
    pp.quant_tokens_silu(G, G, q, s, t, info)
    pp.raise_on_info(info)
    want = q.clone()
    pp.set_wait_limit(1)
    try:
        pp.quant_tokens_silu(G, G, q, s, t, info)
        assert pp.sync_status(info) == 4                  # TIMEOUT
    finally:
        pp.set_wait_limit(0)
    pp.info_clear(info)
    q.zero_()
    pp.quant_tokens_silu(G, G, q, s, t, info)
    pp.raise_on_info(info)
    assert torch.equal(q, want)


def test_pruned_and_quantized_layer_runs_as_integers():
    """The sweep's joint result through the integer forward: its codes stand
    for the pruned weights exactly, so Y is X's 8-bit form times them."""
    g = _gen(1)
    d_out, d_in, n = 96, 256, 700
    W = torch.randn(d_out, d_in, device=DEV, generator=g) / 16
    X = torch.randn(2048, d_in, device=DEV, generator=g).bfloat16()
    grid = torch.empty(d_out, 2, device=DEV)
    pp.quant_grid(W, 8, grid)
    bufs = pp.LayerBuffers.allocate(d_out, d_in, X.shape[0])
    bufs.run(W, X, pp.Params("2:4", qbits=8, qgrid=grid))
    pp.raise_on_info(bufs.info)
    codes = torch.empty(d_out, d_in, dtype=torch.int8, device=DEV)
    pp.quant_codes(W, grid, codes, bufs.info)
    q, s, t = _tokens(n, d_in)
    Y = torch.empty(n, d_out, device=DEV)
    pp.quant_tokens(X[:n], q, s, t, bufs.info)
    pp.linear_i8(q, s, t, codes, grid, Y, bufs.info)
    pp.raise_on_info(bufs.info)
    ints = codes.double() + 128 - grid[:, 1:].double()
    assert torch.equal((grid[:, :1] * ints.float()), W)                  # the fp32 levels themselves
    assert int((ints == 0).sum()) >= d_out * d_in // 2                   # pruned weights are exact zeros
    _check_linear(Y, q.double() @ ints.t(), s, grid)


def test_marshalled_calls_are_the_checked_ones(monkeypatch):
    """The extension module makes the plain calls itself, with the same result
    as the Python path, and leaves the others to it."""
    from post_pruning_b200 import sgpt as S
    pp.lib()
    m = S._marshal
    X = torch.randn(5, 2 * 512, device=DEV, generator=_gen(2)).bfloat16()[:, 512:]
    codes = torch.randint(-128, 128, (70, 512), device=DEV, generator=_gen(3)).to(torch.int8)
    grid = torch.rand(70, 2, device=DEV, generator=_gen(4))
    H = torch.randn(9, 6, 64, device=DEV, generator=_gen(5)).bfloat16()
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device=DEV)
    info = pp.new_info()

    def calls():
        q, s, t = _tokens(5, 512)
        Y, O = torch.empty(5, 70, device=DEV), torch.empty(9, 2, 64, device=DEV, dtype=torch.bfloat16)
        pp.quant_tokens(X, q, s, t, info)
        pp.linear_i8(q, s, t, codes, grid, Y, info)
        pp.attention(H[:, :2], H[:, 2:4], H[:, 4:], off, O, info)
        q2, s2, t2 = _tokens(5, 512)
        pp.quant_tokens_silu(X, X, q2, s2, t2, info)
        return q, s, t, Y, O, q2, s2, t2

    fast = calls()
    monkeypatch.setattr(S, "_marshal", None)
    for a, b in zip(fast, calls()):
        assert torch.equal(a, b)
    monkeypatch.undo()
    q, s, t = _tokens(5, 512)
    Y = torch.empty(5, 70, device=DEV)
    assert m.quant_tokens(X, q, s, t, info) == 0 and m.linear_i8(q, s, t, codes, grid, Y, info, 8) == 0
    for bad in ((X.float(), q, s, t, info), (X.t(), q, s, t, info), (X, q[:4], s, t, info), (X, q, s.double(), t, info),
                (X, q, s, t.cpu(), info), (X, q.t().contiguous().t(), s, t, info), (X[:, :500], q, s, t, info)):
        assert m.quant_tokens(*bad) == -1
    for bad in (dict(qbits=9), dict(Y=Y.half()), dict(Y=Y[:, :69]), dict(codes=codes[:, :500]), dict(grid=grid[:, 0])):
        a = dict(codes=codes, grid=grid, Y=Y, qbits=8) | bad
        assert m.linear_i8(q, s, t, a["codes"], a["grid"], a["Y"], info, a["qbits"]) == -1
        with pytest.raises((ValueError, TypeError, pp.SgptError)):
            pp.linear_i8(q, s, t, a["codes"], a["grid"], a["Y"], info, qbits=a["qbits"])
    # a call that the library refuses comes back with its status
    with pytest.raises(pp.SgptError):
        pp.quant_tokens(X[:, :40], *_tokens(5, 40), info)
    with pytest.raises(pp.SgptError):
        pp.quant_tokens(X[:1].expand(5, 512), q, s, t, info)
    side = torch.cuda.Stream()
    pp.linear_i8(q, s, t, codes, grid, Y, info, stream=side)             # an explicit stream
    side.synchronize()
    assert torch.equal(Y, fast[3])
    pp.raise_on_info(info)
