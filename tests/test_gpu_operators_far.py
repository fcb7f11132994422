"""The operators where offsets into their arrays pass 32 bits: the last rows are
checked as the small tests check all of them."""

import pytest
import torch

import post_pruning_b200 as pp
from test_gpu_attention import _check
from test_gpu_linear_i8 import _check_linear, _check_tokens, _tokens

pytestmark = pytest.mark.gpu

DEV = "cuda"
TAIL = 70


def _rows(n, d, scale=1.0):
    """bf16 [n, d], a block of rows repeated (made in place: no larger temporary)."""
    g = torch.Generator(device=DEV).manual_seed(n)
    X = torch.empty(n, d, dtype=torch.bfloat16, device=DEV)
    some = (scale * torch.randn(4099, d, device=DEV, generator=g)).bfloat16()
    for a in range(0, n, 4099):
        X[a:a + 4099] = some[:min(4099, n - a)]
    return X


@pytest.mark.parametrize("gated", [False, True])
def test_far_tokens(gated):
    n, d = 2 ** 31 // 25600 + 500, 25600
    X = _rows(n, d)
    q, s, t = _tokens(n, d)
    info = pp.new_info()
    if gated:
        pp.quant_tokens_silu(X, X, q, s, t, info)
    else:
        pp.quant_tokens(X, q, s, t, info)
    pp.raise_on_info(info)
    for rows in (slice(0, TAIL), slice(n - TAIL, n)):
        if not gated:
            _check_tokens(X[rows], q[rows], s[rows], t[rows])
            continue
        x = X[rows].double()
        z = x * torch.sigmoid(x) * x
        off = q[rows].double() - 127 * z / z.abs().amax(1, keepdim=True)
        assert float(off.abs().max()) <= 0.5 + 127 * 13 * 2.0 ** -23      # as test_quant_tokens_silu
        assert torch.equal(t[rows].long(), q[rows].long().sum(1))


def test_far_codes():
    r, d = 2 ** 31 // 32768 + 40, 32768
    g = torch.Generator(device=DEV).manual_seed(1)
    W = torch.empty(r, d, device=DEV)
    W[:] = torch.randn(d, device=DEV, generator=g)
    W *= torch.linspace(0.5, 2.0, r, device=DEV)[:, None]
    grid = torch.stack([torch.full((r,), 0.03, device=DEV), torch.full((r,), 128.0, device=DEV)], 1).contiguous()
    codes = torch.full((r, d), 100, dtype=torch.int8, device=DEV)
    info = pp.new_info()
    pp.quant_codes(W, grid, codes, info)
    pp.raise_on_info(info)
    for rows in (slice(0, TAIL), slice(r - TAIL, r)):
        ref = (torch.round(W[rows] / grid[rows, :1]) + 128).clamp(0, 255) - 128
        assert torch.equal(codes[rows].float(), ref)


@pytest.mark.parametrize("n,d_out", [(200, 2 ** 24), (2 ** 24 + 3, 131), (40, 2 ** 24), (2 ** 25 + 1, 80)])
def test_far_products(n, d_out):
    """Y [n, d_out] of more than 2^31 values (40 tokens: more than 2^31 bytes)."""
    d = 32
    g = torch.Generator(device=DEV).manual_seed(n + d_out)
    q = torch.randint(-127, 128, (n, d), device=DEV, generator=g, dtype=torch.int8)
    codes = torch.randint(-128, 128, (d_out, d), device=DEV, generator=g, dtype=torch.int8)
    s = torch.rand(n, device=DEV, generator=g) + 0.01
    t = q.sum(1, dtype=torch.int32)
    grid = torch.stack([torch.rand(d_out, device=DEV, generator=g) + 0.01,
                        torch.randint(0, 256, (d_out,), device=DEV, generator=g).float()], 1).contiguous()
    Y = torch.full((n, d_out), -3.0, dtype=torch.bfloat16, device=DEV)
    info = pp.new_info()
    pp.linear_i8(q, s, t, codes, grid, Y, info)
    pp.raise_on_info(info)
    for a in (slice(0, TAIL), slice(max(0, n // 2 - TAIL), n // 2), slice(max(0, n - TAIL), n)):
        for b in (slice(0, 300), slice(max(0, d_out // 2), d_out // 2 + 300), slice(max(0, d_out - 300), d_out)):
            whole = q[a].double() @ (codes[b].double() - (grid[b, 1:].double() - 128)).t()
            _check_linear(Y[a, b], whole, s[a], grid[b])


@pytest.mark.parametrize("width,heads,kv", [(128, 32, 4), (64, 33, 11)])
def test_far_rows(width, heads, kv):
    """Q and O of more than 2^31 values, packed from many prompts."""
    lens = [1200, 1, 300, 0, 777] * 2
    n = 2 ** 31 // (heads * width) + 3000
    lens = lens + [2000] * ((n - 2 * sum(lens)) // 2000) + lens
    n = sum(lens) + 9
    Q, K, V = _rows(n, heads * width).unflatten(1, (heads, width)), *(_rows(n, kv * width, s).unflatten(1, (kv, width))
                                                                      for s in (1.0, 0.7))
    off = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
    O = torch.full(Q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    info = pp.new_info()
    pp.attention(Q, K, V, off, O, info)
    pp.raise_on_info(info)
    assert bool((O[n - 9:] == 7).all())
    _check(O, Q, K, V, off[:4])
    _check(O, Q, K, V, off[-11:])
