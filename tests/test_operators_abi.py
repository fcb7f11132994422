"""Refusals of the 8-bit forward, the attention and the attention-block driver,
before anything touches a GPU."""

import ctypes

import pytest
import torch

import post_pruning_b200 as pp
from post_pruning_b200 import sgpt as S

FAKE = 1 << 20          # an aligned non-null address; never dereferenced
ODD = FAKE + 4
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 6, 8


def _call(entry, good, **change):
    args = dict(good, **change)
    return getattr(pp.lib(), entry)(*args.values())


CODES = dict(W=FAKE, d_out=64, d_in=256, ldw=256, grid=FAKE, qbits=8, codes=FAKE, info=FAKE, stream=None)
TOKENS = dict(X=FAKE, n=5, d=256, ldx=256, Xq=FAKE, scale=FAKE, sums=FAKE, info=FAKE, stream=None)
SILU = dict(G=FAKE, U=FAKE, n=5, d=256, ldg=256, ldu=512, Xq=FAKE, scale=FAKE, sums=FAKE, info=FAKE, stream=None)
LINEAR = dict(Xq=FAKE, scale=FAKE, sums=FAKE, n=5, codes=FAKE, grid=FAKE, qbits=8, d_in=256, d_out=64, Y=FAKE,
              bf16=0, info=FAKE, stream=None)
ATTN = dict(Q=FAKE, ldq=512, K=FAKE, ldk=256, V=FAKE, ldv=256, offsets=FAKE, n_seq=2, n_tok=100, heads=4, kv_heads=2,
            width=128, scale=ctypes.c_float(0.1), O=FAKE, ldo=512, info=FAKE, stream=None)


@pytest.mark.parametrize("change", [
    dict(W=None), dict(W=ODD), dict(grid=None), dict(codes=ODD), dict(info=None), dict(qbits=1), dict(qbits=9),
    dict(d_in=250), dict(d_in=32800, ldw=32800), dict(d_out=0), dict(ldw=255), dict(ldw=258)])
def test_quant_codes_refuses(change):
    assert _call("sgpt_quant_codes", CODES, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(X=None), dict(X=FAKE + 2), dict(Xq=None), dict(Xq=ODD), dict(scale=None), dict(sums=None), dict(info=None),
    dict(n=-1), dict(n=(1 << 30) + 1), dict(d=0), dict(d=264), dict(d=40), dict(d=32800, ldx=32800), dict(ldx=255),
    dict(ldx=0), dict(ldx=257), dict(ldx=260), dict(ldx=-256)])
def test_quant_tokens_refuses(change):
    if change == dict(d=264):
        change = dict(d=264, ldx=264)             # not a multiple of 32
    assert _call("sgpt_quant_tokens", TOKENS, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(G=None), dict(U=None), dict(U=ODD), dict(Xq=ODD), dict(scale=ODD), dict(sums=ODD), dict(info=None), dict(n=-1),
    dict(d=250), dict(ldg=248), dict(ldu=248), dict(ldu=514)])
def test_quant_tokens_silu_refuses(change):
    assert _call("sgpt_quant_tokens_silu", SILU, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(Xq=None), dict(Xq=ODD), dict(scale=None), dict(sums=None), dict(codes=None), dict(codes=ODD), dict(grid=ODD),
    dict(Y=None), dict(Y=ODD), dict(info=None), dict(n=-1), dict(n=(1 << 30) + 1), dict(qbits=1), dict(qbits=9),
    dict(d_in=8), dict(d_in=48), dict(d_in=32800), dict(d_out=0), dict(d_out=(1 << 24) + 1)])
def test_linear_i8_refuses(change):
    assert _call("sgpt_linear_i8", LINEAR, **change) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(Q=None), INVALID), (dict(K=ODD), INVALID), (dict(V=None), INVALID), (dict(O=ODD), INVALID),
    (dict(offsets=None), INVALID), (dict(offsets=FAKE + 2), INVALID), (dict(info=None), INVALID),
    (dict(n_seq=-1), INVALID), (dict(n_tok=-1), INVALID), (dict(n_tok=(1 << 30) + 1), INVALID),
    (dict(heads=0), INVALID), (dict(heads=5), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID),
    (dict(width=0), INVALID), (dict(width=96, ldq=512), UNSUPPORTED), (dict(width=256), UNSUPPORTED),
    (dict(ldq=504), INVALID), (dict(ldq=516), INVALID), (dict(ldk=128), INVALID), (dict(ldv=252), INVALID),
    (dict(ldo=511), INVALID), (dict(scale=ctypes.c_float(0.0)), INVALID), (dict(scale=ctypes.c_float(-1.0)), INVALID),
    (dict(scale=ctypes.c_float(float("nan"))), INVALID), (dict(scale=ctypes.c_float(float("inf"))), INVALID),
    (dict(n_tok=1 << 30, heads=4096, kv_heads=1, ldq=1 << 20, ldo=1 << 20), UNSUPPORTED)])
def test_attention_refuses(change, status):
    assert _call("sgpt_attention", ATTN, **change) == status


def test_nothing_to_do_is_ok_without_a_gpu():
    assert _call("sgpt_quant_tokens", TOKENS, n=0, X=None, Xq=None, scale=None, sums=None) == OK
    assert _call("sgpt_quant_tokens_silu", SILU, n=0, G=None, U=None) == OK
    assert _call("sgpt_linear_i8", LINEAR, n=0, Xq=None, Y=None) == OK
    assert _call("sgpt_attention", ATTN, n_tok=0, Q=None, O=None) == OK
    assert _call("sgpt_attention", ATTN, n_seq=0) == OK


def _block(**change):
    names = [f[0] for f in S._AttnBlock._fields_]
    blk = S._AttnBlock(*(change.pop(n, FAKE) for n in names))
    args = dict(blk=ctypes.byref(blk), hidden=256, heads=4, kv_heads=2, width=64, scale=ctypes.c_float(0.125), X=FAKE,
                n_tok=100, offsets=FAKE, n_seq=2, mode=0, p=ctypes.byref(S.Params("2:4").to_c()), X_next=FAKE, A=None,
                ws=FAKE, ws_bytes=1 << 40, info=FAKE, stream=None)
    args.update(change)
    return pp.lib().sgpt_prune_attn_block(*args.values())


def test_attn_block_refuses():
    for name in ("W_q", "W_k", "W_v", "W_o", "mask_q", "mask_o"):
        assert _block(**{name: None}) == INVALID and _block(**{name: ODD}) == INVALID
    for change in (dict(X=None), dict(X_next=ODD), dict(A=ODD), dict(offsets=None), dict(offsets=FAKE + 1),
                   dict(info=None), dict(n_seq=-1), dict(n_tok=0), dict(n_tok=(1 << 30) + 1), dict(hidden=100),
                   dict(heads=5), dict(heads=0), dict(heads=514, kv_heads=2), dict(width=0), dict(mode=2), dict(p=None),
                   dict(scale=ctypes.c_float(0.0)), dict(scale=ctypes.c_float(float("nan")))):
        assert _block(**change) == INVALID, change
    assert _block(width=80) == UNSUPPORTED
    assert _block(ws_bytes=1000) == WORKSPACE and _block(ws=FAKE + 16) == WORKSPACE and _block(ws=None) == WORKSPACE
    forced = S.Params("2:4", forced=True).to_c()
    assert _block(p=ctypes.byref(forced)) == INVALID
    wide = S.Params("16:128").to_c()
    assert _block(p=ctypes.byref(wide), hidden=320) == INVALID
    assert _block(p=ctypes.byref(S.Params("3:6").to_c())) == UNSUPPORTED


def test_attn_block_workspace_sizes():
    need = pp.lib().sgpt_attn_block_workspace_bytes
    base = need(256, 4, 2, 64, 1000)
    # at least H and its factor for both inputs, and the fp32 product
    assert base >= 4 * (2 * 256 * 256 * 2 + 1000 * 256)
    assert need(256, 4, 2, 64, 5000) > base
    for bad in ((250, 4, 2, 64, 1000), (256, 4, 3, 64, 1000), (256, 4, 2, 96, 1000), (256, 4, 2, 64, 0),
                (256, 0, 1, 64, 10), (256, 512, 8, 128, 10)):
        assert need(*bad) == 0, bad


def test_binding_refuses_before_the_library():
    """Types, shapes and devices that the binding answers for itself."""
    f = dict(dtype=torch.bfloat16)
    X, q = torch.zeros(4, 64, **f), torch.zeros(4, 64, dtype=torch.int8)
    s, t, info = torch.zeros(4), torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    codes, grid = torch.zeros(8, 64, dtype=torch.int8), torch.ones(8, 2)
    h = torch.zeros(4, 2, 64, **f)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: pp.quant_tokens(X, q, s, t, info), lambda: pp.quant_tokens_silu(X, X, q, s, t, info),
                 lambda: pp.linear_i8(q, s, t, codes, grid, torch.zeros(4, 8), info),
                 lambda: pp.attention(h, h, h, off, h.clone(), info),
                 lambda: pp.quant_codes(torch.zeros(8, 64), grid, codes, info),
                 lambda: pp.quant_tokens(None, q, s, t, info)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        pp.attn_block_workspace(250, 4, 2, 64, 100)
    with pytest.raises(ValueError):
        S._heads_stride(torch.zeros(4, 64, **f), "Q")
    with pytest.raises(ValueError):
        S._heads_stride(torch.zeros(4, 64, 2, **f).transpose(1, 2), "Q")
    with pytest.raises(ValueError):
        S._row_stride(torch.zeros(4, 64, **f).t(), "X")
    # a broadcast row has no stride the library takes; a single row has no stride at all
    assert S._row_stride(torch.zeros(1, 64, **f).expand(4, 64), "X") == 0
    assert S._row_stride(torch.zeros(4, 64, **f)[::4], "X") == 64
    assert S._heads_stride(torch.zeros(4, 6, 64, **f)[:, 2:4], "Q") == 6 * 64


def test_marshalling_answers_only_what_is_plainly_valid():
    """The extension module takes no CPU tensor, wrong type or wrong count;
    the Python functions then raise."""
    pp.lib()
    m = S._marshal
    X, q = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8)
    s, t, info = torch.zeros(4), torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    if torch.cuda.is_available():
        pytest.skip("the refusals below are those of a machine without a GPU")
    assert m.quant_tokens(X, q, s, t, info) == -1
    assert m.quant_tokens(X, q, s, t) == -1
    assert m.quant_tokens(None, q, s, t, info) == -1
    assert m.quant_tokens_silu(X, X, q, s, t, info) == -1
    assert m.linear_i8(q, s, t, q, s, s, info, "8") == -1
    assert m.attention(X, X, X, t, X, info, None) == -1
    with pytest.raises(TypeError):
        m.bind(1, 2, 3)
