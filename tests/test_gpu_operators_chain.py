"""The operators after one another on one stream, as a decoder block calls them:
each may start before the one before it has ended, and reads what that one (or
anything else before it) wrote."""

import pytest
import torch

import post_pruning_b200 as pp

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("n,width", [(40, 64), (700, 128)])
def test_operators_read_what_the_ones_before_them_wrote(n, width):
    """Offsets and rows that are written right before the call, outputs that
    the next call reads, in buffers that the last pass has used: the bits of
    passes that wait after every step."""
    heads, kv = 8, 2
    d, inter = heads * width, 1408
    g = torch.Generator(device=DEV).manual_seed(n)
    wo = torch.randint(-128, 128, (2 * inter, d), device=DEV, generator=g).to(torch.int8)
    wd = torch.randint(-128, 128, (d, inter), device=DEV, generator=g).to(torch.int8)
    grids = [torch.stack([torch.rand(w.shape[0], device=DEV, generator=g) * 1e-3 + 1e-4,
                          torch.full((w.shape[0],), 128.0, device=DEV)], 1).contiguous() for w in (wo, wd)]
    sets = []
    for i in range(3):
        cut = sorted(torch.randint(0, n + 1, (3,), generator=torch.Generator().manual_seed(i)).tolist())
        off = torch.tensor([0, *cut, n], dtype=torch.int32, device=DEV)
        sets.append((torch.randn(n, (heads + 2 * kv) * width, device=DEV, generator=g).bfloat16(), off))
    qkv, off = torch.empty_like(sets[0][0]), torch.empty_like(sets[0][1])
    q, k, v = (t.unflatten(1, (-1, width)) for t in qkv.split([d, kv * width, kv * width], 1))
    a = torch.empty(n, heads, width, dtype=torch.bfloat16, device=DEV)
    gu = torch.empty(n, 2 * inter, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(n, d, device=DEV)
    info = pp.new_info()

    def tokens(c):
        return (torch.empty(n, c, dtype=torch.int8, device=DEV), torch.empty(n, device=DEV),
                torch.empty(n, dtype=torch.int32, device=DEV))
    ta, tz = tokens(d), tokens(inter)
    steps = [lambda: pp.attention(q, k, v, off, a, info), lambda: pp.quant_tokens(a.flatten(1), *ta, info),
             lambda: pp.linear_i8(*ta, wo, grids[0], gu, info),
             lambda: pp.quant_tokens_silu(gu[:, :inter], gu[:, inter:], *tz, info),
             lambda: pp.linear_i8(*tz, wd, grids[1], y, info)]

    def one(s, wait):
        qkv.copy_(s[0])
        off.copy_(s[1])
        for f in steps:
            f()
            if wait:
                torch.cuda.synchronize()
        return [t.clone() for t in (a, *ta, gu, *tz, y)]

    want = [one(s, True) for s in sets]
    pp.raise_on_info(info)
    for i in range(30):
        for got, ref in zip(one(sets[i % 3], False), want[i % 3]):
            assert torch.equal(got, ref)
    pp.raise_on_info(info)
