"""The binding's two ways to a call that is made per token and layer: through
the extension module and through the Python functions alone."""

import pytest
import torch

import post_pruning_b200 as pp
from post_pruning_b200 import sgpt as S

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _operands():
    g = torch.Generator(device=DEV).manual_seed(2)
    n, d, rows, heads, width = 37, 512, 96, 4, 64
    wide = torch.randn(n, 2 * d, device=DEV, generator=g).bfloat16()
    codes = torch.randint(-128, 128, (rows, d), device=DEV, generator=g).to(torch.int8)
    grid = torch.stack([torch.rand(rows, device=DEV, generator=g) + 0.01, torch.full((rows,), 100.0, device=DEV)], 1).contiguous()
    qkv = torch.randn(n, 3 * heads * width, device=DEV, generator=g).bfloat16()
    off = torch.tensor([0, 11, 11, n], dtype=torch.int32, device=DEV)
    return n, d, wide, codes, grid, qkv, heads, width, off


def _pass(info):
    """Every call once; all outputs."""
    n, d, wide, codes, grid, qkv, heads, width, off = _operands()
    out = []
    for gated in (False, True):
        q, s, t = (torch.empty(n, d, dtype=torch.int8, device=DEV), torch.empty(n, device=DEV),
                   torch.empty(n, dtype=torch.int32, device=DEV))
        if gated:
            pp.quant_tokens_silu(wide[:, :d], wide[:, d:], q, s, t, info)
        else:
            pp.quant_tokens(wide[:, d:], q, s, t, info)
        out += [q, s, t]
        for dtype in (torch.float32, torch.bfloat16):
            out.append(torch.empty(n, codes.shape[0], dtype=dtype, device=DEV))
            pp.linear_i8(q, s, t, codes, grid, out[-1], info)
    q, k, v = (x.unflatten(1, (heads, width)) for x in qkv.chunk(3, 1))
    for scale in (None, 0.25):
        out.append(torch.empty(n, heads, width, dtype=torch.bfloat16, device=DEV))
        pp.attention(q, k, v, off, out[-1], info, scale=scale)
    return out


def test_python_functions_alone_give_the_same_bits(monkeypatch):
    info = pp.new_info()
    pp.lib()
    assert S._marshal is not None
    want = _pass(info)
    monkeypatch.setattr(S, "_marshal", None)
    before = pp.kernel_launches()
    for got, ref in zip(_pass(info), want):
        assert torch.equal(got, ref)
    assert pp.kernel_launches() == before + 8
    pp.raise_on_info(info)


@pytest.mark.parametrize("alone", [False, True])
@pytest.mark.parametrize("bad,error", [(dict(dtype=torch.int64), TypeError), (dict(dtype=torch.uint8), TypeError),
                                       (dict(dtype=torch.float32), TypeError), (dict(size=0), ValueError)])
def test_the_error_word_is_an_int32(bad, error, alone, monkeypatch):
    """A kernel writes four bytes there: a shorter or emptier tensor is refused,
    a longer type would not read as the code."""
    info = torch.zeros(bad.get("size", 1), dtype=bad.get("dtype", torch.int32), device=DEV)
    n, d, wide, codes, grid, qkv, heads, width, off = _operands()
    q, s, t = (torch.empty(n, d, dtype=torch.int8, device=DEV), torch.empty(n, device=DEV),
               torch.empty(n, dtype=torch.int32, device=DEV))
    qh = qkv[:, :heads * width].unflatten(1, (heads, width))
    W = [torch.zeros(256, 256, device=DEV) for _ in range(4)]
    masks = [torch.zeros(256, 8, dtype=torch.int32, device=DEV) for _ in range(4)]
    X = torch.zeros(n, 256, dtype=torch.bfloat16, device=DEV)
    ws = pp.attn_block_workspace(256, 4, 4, 64, n)
    pp.lib()
    if alone:
        monkeypatch.setattr(S, "_marshal", None)
    before = pp.kernel_launches()
    for call in (lambda: pp.quant_codes(torch.zeros(96, d, device=DEV), grid, codes, info),
                 lambda: pp.quant_tokens(wide[:, d:], q, s, t, info),
                 lambda: pp.quant_tokens_silu(wide[:, :d], wide[:, d:], q, s, t, info),
                 lambda: pp.linear_i8(q, s, t, codes, grid, torch.empty(n, 96, device=DEV), info),
                 lambda: pp.attention(qh, qh, qh, off, torch.empty_like(qh), info),
                 lambda: pp.prune_attn_block(*W, masks, X, off, 64, pp.Params("2:4"), torch.empty_like(X), ws, info)):
        with pytest.raises(error):
            call()
    assert pp.kernel_launches() == before
