"""Buffers of the block drivers (pp.prune_attn_block, pp.prune_mlp_block) that a program
passes when blocks are pruned one after another: x' written over x."""

import pytest
import torch

import post_pruning_b200 as pp
from test_gpu_attn_driver import DEV, _make, _masks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [pp.DRIVER_SEQUENTIAL, pp.DRIVER_PARALLEL])
def test_attn_block_in_place(mode):
    hidden, heads, kv, width, n = 256, 4, 2, 64, 700
    W0, X = _make(hidden, heads, kv, width, n, 7)
    off = torch.tensor([0, 100, 650], dtype=torch.int32, device=DEV)
    ws = pp.attn_block_workspace(hidden, heads, kv, width, n)
    info = pp.new_info()
    results = []
    for inplace in (False, True):
        W, masks, x = [w.clone() for w in W0], _masks(W0), X.clone()
        X_next = x if inplace else torch.empty_like(X)
        A = torch.empty(n, heads * width, dtype=torch.bfloat16, device=DEV)
        pp.prune_attn_block(*W, masks, x, off, width, pp.Params("2:4"), X_next, ws, info, mode=mode, A=A)
        pp.raise_on_info(info)
        results.append([*W, *masks, A, X_next])
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("mode", [pp.DRIVER_SEQUENTIAL, pp.DRIVER_PARALLEL])
def test_mlp_block_in_place(mode):
    hidden, inter, n = 256, 448, 900
    g = torch.Generator(device=DEV).manual_seed(11)
    W0 = [torch.randn(r, c, device=DEV, generator=g) / c ** 0.5 for r, c in ((inter, hidden), (inter, hidden), (hidden, inter))]
    X = torch.randn(n, hidden, device=DEV, generator=g).bfloat16()
    ws = pp.mlp_block_workspace(hidden, inter, n)
    info = pp.new_info()
    results = []
    for inplace in (False, True):
        W, masks, x = [w.clone() for w in W0], _masks(W0), X.clone()
        X_next = x if inplace else torch.empty_like(X)
        Z = torch.empty(n, inter, dtype=torch.bfloat16, device=DEV)
        pp.prune_mlp_block(*W, masks, x, pp.Params("2:4"), X_next, ws, info, mode=mode, Z=Z)
        pp.raise_on_info(info)
        results.append([*W, *masks, Z, X_next])
    for a, b in zip(*results):
        assert torch.equal(a, b)
