"""The attention-block driver (pp.prune_attn_block), and the forward of a
pruned and quantized decoder block in 8-bit integers.

The driver launches the library's own kernels in a fixed order and every one
of them is deterministic, so its weights, masks, attention output and result
equal, bit for bit, those of the same steps called one by one; the result is
also checked against the block's formula in 64 bits.
"""

import pytest
import torch

import post_pruning_b200 as pp

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _make(hidden, heads, kv, width, n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dq, dk = heads * width, kv * width
    W = [torch.randn(r, c, device=DEV, generator=g) / c ** 0.5 for r, c in ((dq, hidden), (dk, hidden), (dk, hidden),
                                                                           (hidden, dq))]
    X = (torch.randn(n, hidden, device=DEV, generator=g) * torch.exp(torch.randn(hidden, device=DEV, generator=g)))
    return W, X.bfloat16()


def _masks(W):
    return [torch.zeros(w.shape[0], w.shape[1] // 32, dtype=torch.int32, device=DEV) for w in W]


def _mix(W, X, off, heads, kv, width, info):
    """q, k, v, attention as the driver forms them."""
    n = X.shape[0]
    parts = []
    for w in W[:3]:
        wb, y = torch.empty(w.shape, dtype=torch.bfloat16, device=DEV), torch.empty(n, w.shape[0], device=DEV)
        pp.to_bf16(w, wb, info)
        pp.linear_bf16(X, wb, y, info)
        yb = torch.empty(y.shape, dtype=torch.bfloat16, device=DEV)
        pp.to_bf16(y, yb, info)
        parts.append(yb.unflatten(1, (-1, width)))
    A = torch.zeros(n, heads, width, dtype=torch.bfloat16, device=DEV)
    pp.attention(*parts, off, A, info)
    return A.flatten(1)


def _out(W_o, A, X, info):
    wb, y = torch.empty(W_o.shape, dtype=torch.bfloat16, device=DEV), torch.empty(X.shape, device=DEV)
    pp.to_bf16(W_o, wb, info)
    pp.linear_bf16(A, wb, y, info)
    return (X.float() + y).bfloat16()


def _prune(W, masks, X, params, info):
    d = X.shape[1]
    ws = pp.workspace(max(w.shape[0] for w in W), d, X.shape[0])
    H, U = torch.empty(d, d, device=DEV), torch.empty(d, d, device=DEV)
    pp.hessian_compute(H, X, ws, info)
    pp.factor(H, X.shape[0], params.damp, U, ws, info)
    for w, m in zip(W, masks):
        pp.prune(w, U, params, m, ws, info)


CASES = [(256, 4, 2, 64, [300, 1, 0, 211], 20, "2:4", 0), (320, 3, 1, 128, [700], 0, "unstructured:0.5", 0),
         (256, 2, 2, 128, [129, 400, 77], 0, "4:8", 8)]


@pytest.mark.parametrize("mode", [pp.DRIVER_SEQUENTIAL, pp.DRIVER_PARALLEL])
@pytest.mark.parametrize("hidden,heads,kv,width,lens,outside,pattern,qbits", CASES)
def test_attn_block_is_its_steps(hidden, heads, kv, width, lens, outside, pattern, qbits, mode):
    n = sum(lens) + outside
    W0, X = _make(hidden, heads, kv, width, n, hidden + n)
    off = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    params = pp.Params(pattern, qbits=qbits)
    info = pp.new_info()

    W, masks = [w.clone() for w in W0], _masks(W0)
    X_next, A = torch.empty_like(X), torch.empty(n, heads * width, dtype=torch.bfloat16, device=DEV)
    ws = pp.attn_block_workspace(hidden, heads, kv, width, n)
    pp.prune_attn_block(*W, masks, X, off, width, params, X_next, ws, info, mode=mode, A=A)
    pp.raise_on_info(info)

    V, vm = [w.clone() for w in W0], _masks(W0)
    if mode == pp.DRIVER_SEQUENTIAL:
        _prune(V[:3], vm[:3], X, params, info)
        a = _mix(V, X, off, heads, kv, width, info)
        _prune(V[3:], vm[3:], a, params, info)
        x = _out(V[3], a, X, info)
    else:
        a = _mix(V, X, off, heads, kv, width, info)
        x = _out(V[3], a, X, info)
        _prune(V[:3], vm[:3], X, params, info)
        _prune(V[3:], vm[3:], a, params, info)
    pp.raise_on_info(info)
    for p, q in zip(W + masks + [A, X_next], V + vm + [a, x]):
        assert torch.equal(p, q)
    assert not torch.equal(W[0], W0[0])
    if outside:
        assert not bool(A[n - outside:].any()) and torch.equal(X_next[n - outside:], X[n - outside:])

    # the result against the formula, from the driver's own a and the weights it used for the output
    Wo = (W if mode == pp.DRIVER_SEQUENTIAL else W0)[3].bfloat16().double()
    ref = X.double() + A.double() @ Wo.t()
    size = X.double().abs() + A.double().abs() @ Wo.abs().t()
    # the product's fp32 sums (1e-5 of the sum of magnitudes), one fp32 addition and one rounding to bf16
    err = (X_next.double() - ref).abs()
    assert bool((err <= 2.0 ** -8 * ref.abs() + (1e-5 + 2.0 ** -24) * 1.01 * size).all())


def test_attn_block_without_a_buffer_and_captured():
    """A kept in the workspace gives the same result; a captured call replays
    on new contents of the same buffers."""
    hidden, heads, kv, width, lens = 256, 4, 2, 64, [200, 333]
    n = sum(lens)
    off = torch.tensor([0, 200, 533], dtype=torch.int32, device=DEV)
    ws = pp.attn_block_workspace(hidden, heads, kv, width, n)
    info = pp.new_info()
    want = []
    for seed in (1, 2):
        W, X = _make(hidden, heads, kv, width, n, seed)
        masks, X_next, A = _masks(W), torch.empty_like(X), torch.empty(n, heads * width, dtype=torch.bfloat16, device=DEV)
        pp.prune_attn_block(*W, masks, X, off, width, pp.Params("2:4"), X_next, ws, info, A=A)
        pp.raise_on_info(info)
        want.append([*W, *masks, X_next])
    W, X = _make(hidden, heads, kv, width, n, 1)
    masks, X_next = _masks(W), torch.empty_like(X)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pp.prune_attn_block(*W, masks, X, off, width, pp.Params("2:4"), X_next, ws, info)
    for i, seed in enumerate((1, 2)):
        W1, X1 = _make(hidden, heads, kv, width, n, seed)
        for a, b in zip([*W, X], [*W1, X1]):
            a.copy_(b)
        g.replay()
        pp.raise_on_info(info)
        for a, b in zip([*W, *masks, X_next], want[i]):
            assert torch.equal(a, b)


def test_attn_block_reports_bad_offsets():
    W, X = _make(256, 2, 2, 64, 100, 3)
    info = pp.new_info()
    pp.prune_attn_block(*W, _masks(W), X, torch.tensor([0, 80, 70], dtype=torch.int32, device=DEV), 64,
                        pp.Params("2:4"), torch.empty_like(X), pp.attn_block_workspace(256, 2, 2, 64, 100), info)
    assert pp.sync_status(info) == 1


def test_quantized_decoder_block_in_integers():
    """A pruned and 8-bit quantized block run as it would be served: tokens to
    8 bits, integer q/k/v, attention, tokens to 8 bits, integer o; then gate
    and up, the gated quantization and down. Each stage is checked against
    its definition in 64 bits on the inputs that it had."""
    hidden, heads, kv, width, inter, lens = 512, 4, 2, 128, 1408, [333, 1, 190]
    n = sum(lens)
    W, X = _make(hidden, heads, kv, width, n, 9)
    g = torch.Generator(device=DEV).manual_seed(10)
    W += [torch.randn(inter, hidden, device=DEV, generator=g) / hidden ** 0.5 for _ in range(2)]
    W += [torch.randn(hidden, inter, device=DEV, generator=g) / inter ** 0.5]
    off = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    info = pp.new_info()
    X = (X.float() / X.float().std()).bfloat16()
    grids = []
    for w in W:                                            # the joint sweep, with the grid of each dense matrix
        grid = torch.empty(w.shape[0], 2, device=DEV)
        pp.quant_grid(w, 8, grid)
        grids.append(grid)
        _prune([w], _masks([w]), X if w.shape[1] == hidden else torch.randn(2 * w.shape[1], w.shape[1], device=DEV,
                                                                            generator=g).bfloat16(),
               pp.Params("2:4", qbits=8, qgrid=grid), info)
    codes = []
    for w, grid in zip(W, grids):
        c = torch.empty(w.shape, dtype=torch.int8, device=DEV)
        pp.quant_codes(w, grid, c, info)
        codes.append(c)
    pp.raise_on_info(info)

    def tokens(d):
        return (torch.empty(n, d, dtype=torch.int8, device=DEV), torch.empty(n, device=DEV),
                torch.empty(n, dtype=torch.int32, device=DEV))

    def product(tok, i, dtype=torch.bfloat16):
        y = torch.empty(n, W[i].shape[0], dtype=dtype, device=DEV)
        pp.linear_i8(*tok, codes[i], grids[i], y, info)
        # the codes stand for the pruned weights: y = dequantized tokens times W
        ref = (tok[0].double() * tok[1].double()[:, None]) @ W[i].double().t()
        size = (tok[0].double() * tok[1].double()[:, None]).abs() @ W[i].double().abs().t()
        half = 2.0 ** -8 if dtype is torch.bfloat16 else 0.0
        # W on its fp32 grid is scale * integer rounded once (2^-24 of each term); the result's own three roundings
        assert bool(((y.double() - ref).abs() <= half * ref.abs() + 2.0 ** -24 * (4 * ref.abs() + 1.01 * size)).all())
        return y

    tok = tokens(hidden)
    pp.quant_tokens(X, *tok, info)
    q, k, v = (product(tok, i).unflatten(1, (-1, width)) for i in range(3))
    a = torch.empty(n, heads, width, dtype=torch.bfloat16, device=DEV)
    pp.attention(q, k, v, off, a, info)
    first = 0
    for m in lens:
        later = torch.ones(m, m, dtype=torch.bool, device=DEV).triu(1)
        for h in range(heads):
            s = slice(first, first + m)
            p = torch.softmax((q[s, h].double() @ k[s, h // 2].double().t() * width ** -0.5).masked_fill(later, -torch.inf), 1)
            o, size = p @ v[s, h // 2].double(), p @ v[s, h // 2].double().abs()
            # weights and result rounded to bf16, scores and sums in fp32
            assert bool(((a[s, h].double() - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -10) * size).all())
        first += m
    tok = tokens(heads * width)
    pp.quant_tokens(a.flatten(1), *tok, info)
    x = (X.float() + product(tok, 3, torch.float32)).bfloat16()
    tok = tokens(hidden)
    pp.quant_tokens(x, *tok, info)
    gate, up = product(tok, 4), product(tok, 5)
    tok = tokens(inter)
    pp.quant_tokens_silu(gate, up, *tok, info)
    y = product(tok, 6, torch.float32)
    pp.raise_on_info(info)
    # the whole MLP against the unquantized formula: 8-bit tokens of z are off by at most half a step each
    z = torch.nn.functional.silu(gate.double()) * up.double()
    ref = z @ W[6].double().t()
    step = z.abs().amax(1, keepdim=True) / 127
    assert bool(((y.double() - ref).abs() <= 0.51 * step * W[6].double().abs().sum(1)[None] + 1e-6).all())
