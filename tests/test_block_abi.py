"""Refusals of the operators around the expert MLP, none of which needs a GPU: the
C entry points report a bad argument before any device call, and the Python
functions before they touch the library."""

import ctypes
import math

import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
from bit_quantized_mixture_nf4_amd import _lib

FAKE = 0x10000  # 16-byte aligned, never dereferenced on these paths
L = _lib


def _stack(E=1, out=64, inn=64, cb=0, packed=FAKE, absmax=FAKE, bs=64, scales=None):
    return _lib.E4bStack(packed, absmax, E, out, inn, bs, cb, scales)


def _route(T=4, E=8, k=2, logits=FAKE, idx=FAKE, w=FAKE):
    return e4b.load().e4b_route(logits, T, E, k, idx, w, None)


def _route_bwd(T=4, E=8, k=2, idx=FAKE, w=FAKE, gw=FAKE, gl=FAKE):
    return e4b.load().e4b_route_backward(idx, w, gw, T, E, k, gl, None)


@pytest.mark.parametrize("kw", [dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(k=33, E=64), dict(T=-1),
                                dict(T=1 << 24)])
def test_route_shapes(kw):
    assert _route(**kw) == L.E4B_ERR_SHAPE
    assert _route_bwd(**kw) == L.E4B_ERR_SHAPE


def test_route_pointers():
    for name in ("logits", "idx", "w"):
        assert _route(**{name: None}) == L.E4B_ERR_NULL
        assert _route(**{name: FAKE + 4}) == L.E4B_ERR_ALIGN
    for name in ("idx", "w", "gw", "gl"):
        assert _route_bwd(**{name: None}) == L.E4B_ERR_NULL
        assert _route_bwd(**{name: FAKE + 8}) == L.E4B_ERR_ALIGN
    assert _route(T=0, logits=None, idx=None, w=None) == L.E4B_OK
    assert _route_bwd(T=0, idx=None, w=None, gw=None, gl=None) == L.E4B_OK


def _permute(T=4, k=2, E=8, H=64, dt=1, idx=FAKE, x=FAKE, rows=FAKE, off=FAKE, order=FAKE, pos=FAKE):
    return e4b.load().e4b_permute(T, k, E, H, dt, idx, x, rows, off, order, pos, None)


def _unpermute(T=4, k=2, E=8, H=64, dt=1, off=FAKE, pos=FAKE, w=FAKE, rows=FAKE, y=FAKE):
    return e4b.load().e4b_unpermute(T, k, E, H, dt, off, pos, w, rows, y, None)


def _unpermute_bwd(T=4, k=2, E=8, H=64, dt=1, off=FAKE, pos=FAKE, w=FAKE, rows=FAKE, gy=FAKE, gr=FAKE, gw=FAKE):
    return e4b.load().e4b_unpermute_backward(T, k, E, H, dt, off, pos, w, rows, gy, gr, gw, None)


@pytest.mark.parametrize("call", [_permute, _unpermute, _unpermute_bwd])
def test_order_shapes_and_types(call):
    for kw in (dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(H=0), dict(H=1 << 24), dict(T=-1),
               dict(T=1 << 24)):
        assert call(**kw) == L.E4B_ERR_SHAPE, kw
    assert call(dt=2) == L.E4B_ERR_DTYPE
    assert call(dt=-1) == L.E4B_ERR_DTYPE


def test_order_pointers():
    for name in ("idx", "off", "order", "pos", "x", "rows"):
        assert _permute(**{name: None}) == L.E4B_ERR_NULL, name
        assert _permute(**{name: FAKE + 4}) == L.E4B_ERR_ALIGN, name
    assert _permute(T=0, off=None) == L.E4B_ERR_NULL  # the offsets are written for an empty batch too
    for name in ("off", "pos", "rows", "y"):
        assert _unpermute(**{name: None}) == L.E4B_ERR_NULL, name
    for name in ("off", "pos", "rows", "y", "w"):
        assert _unpermute(**{name: FAKE + 4}) == L.E4B_ERR_ALIGN, name
    for name in ("off", "pos", "rows", "gy", "gr"):
        assert _unpermute_bwd(**{name: None}) == L.E4B_ERR_NULL, name
    for name in ("off", "pos", "rows", "gy", "gr", "gw", "w"):
        assert _unpermute_bwd(**{name: FAKE + 2}) == L.E4B_ERR_ALIGN, name
    assert _unpermute(T=0, off=None, pos=None, rows=None, y=None) == L.E4B_OK
    assert _unpermute_bwd(T=0, off=None, pos=None, rows=None, gy=None, gr=None) == L.E4B_OK


def _linear(st=None, rows=4, off=None, x=FAKE, bias=FAKE, act=0, res=FAKE, dt=1, y=FAKE, pre=FAKE, ws=FAKE,
            ws_bytes=1 << 40):
    st = st or _stack()
    return e4b.load().e4b_expert_linear(ctypes.byref(st), rows, off, x, bias, act, res, dt, y, pre, ws, ws_bytes, None)


def _linear_bwd(st=None, rows=4, off=None, gy=FAKE, dt=1, pre=FAKE, x=FAKE, bias=FAKE, act=0, gx=FAKE, gb=FAKE, ws=FAKE,
                ws_bytes=1 << 40):
    st = st or _stack()
    return e4b.load().e4b_expert_linear_dgrad(ctypes.byref(st), rows, off, gy, dt, pre, x, bias, act, gx, gb, ws,
                                              ws_bytes, None)


@pytest.mark.parametrize("call", [_linear, _linear_bwd])
def test_linear_arguments(call):
    assert call(st=_stack(inn=96)) == L.E4B_ERR_SHAPE
    assert call(st=_stack(out=0)) == L.E4B_ERR_SHAPE
    assert call(st=_stack(E=1025), off=FAKE) == L.E4B_ERR_SHAPE
    assert call(st=_stack(bs=32)) == L.E4B_ERR_BLOCKSIZE
    assert call(st=_stack(cb=9)) == L.E4B_ERR_CODEBOOK
    assert call(st=_stack(packed=None)) == L.E4B_ERR_NULL
    assert call(st=_stack(cb=3, bs=32)) == L.E4B_ERR_NULL  # MXFP4 needs its scales
    assert call(rows=-1) == L.E4B_ERR_SHAPE
    assert call(rows=(1 << 30) + 1) == L.E4B_ERR_SHAPE
    assert call(st=_stack(out=1 << 21)) == L.E4B_ERR_SHAPE
    assert call(st=_stack(inn=1 << 21)) == L.E4B_ERR_SHAPE
    assert call(st=_stack(out=1 << 16), rows=1 << 22) == L.E4B_ERR_SHAPE  # more tiles than a launch has
    assert call(act=5) == L.E4B_ERR_ACT and call(act=-1) == L.E4B_ERR_ACT
    assert call(dt=2) == L.E4B_ERR_DTYPE
    assert call(st=_stack(E=4)) == L.E4B_ERR_NULL  # several experts need offsets
    # (rows and columns enough for tiles)
    assert call(st=_stack(out=4096), rows=16384, ws=None) == L.E4B_ERR_NULL
    assert call(st=_stack(out=4096), rows=16384, ws_bytes=16) == L.E4B_ERR_WORKSPACE


def test_linear_pointers():
    for name in ("x", "y"):
        assert _linear(**{name: None}) == L.E4B_ERR_NULL
    for name in ("off", "x", "bias", "res", "y", "pre", "ws"):
        assert _linear(**{name: FAKE + 4}) == L.E4B_ERR_ALIGN, name
    assert _linear(rows=0, x=None, y=None, ws=None) == L.E4B_OK
    for name in ("gy", "gx"):
        assert _linear_bwd(**{name: None}) == L.E4B_ERR_NULL
    for name in ("off", "gy", "pre", "x", "bias", "gx", "gb", "ws"):
        assert _linear_bwd(**{name: FAKE + 4}) == L.E4B_ERR_ALIGN, name
    # an activation needs z, or x to make it from
    assert _linear_bwd(act=2, pre=None, x=None) == L.E4B_ERR_NULL
    assert _linear_bwd(rows=0, gy=None, gx=None, gb=None, ws=None) == L.E4B_OK


def test_linear_workspace_sizes():
    lib = e4b.load()
    st, rows = _stack(E=4, out=4096, inn=64), 16384
    fwd = lib.e4b_expert_linear_workspace_bytes(ctypes.byref(st), rows)
    bwd = lib.e4b_expert_linear_dgrad_workspace_bytes(ctypes.byref(st), rows, 0)
    rec = lib.e4b_expert_linear_dgrad_workspace_bytes(ctypes.byref(st), rows, 1)
    assert 0 < fwd < bwd < rec
    assert rec >= bwd + rows * 4096 * 4
    assert _linear(st=st, rows=rows, off=FAKE, ws_bytes=fwd - 1) == L.E4B_ERR_WORKSPACE
    assert _linear(st=st, rows=rows, off=FAKE, ws=None) == L.E4B_ERR_NULL
    assert _linear_bwd(st=st, rows=rows, off=FAKE, ws_bytes=bwd - 1) == L.E4B_ERR_WORKSPACE
    assert _linear_bwd(st=st, rows=rows, off=FAKE, act=2, pre=None, ws_bytes=rec - 1) == L.E4B_ERR_WORKSPACE
    # few rows read the offsets themselves
    assert lib.e4b_expert_linear_workspace_bytes(ctypes.byref(st), 8) == 0
    assert lib.e4b_expert_linear_workspace_bytes(ctypes.byref(st), 0) == 0
    bad = _stack(inn=100)
    assert lib.e4b_expert_linear_workspace_bytes(ctypes.byref(bad), 300) == 0
    assert lib.e4b_expert_linear_dgrad_workspace_bytes(ctypes.byref(bad), 300, 1) == 0


def _norm_desc(T=4, H=64, dt=1, kind=0, eps=1e-6, scale=1.0, post=FAKE, pre=FAKE, gate=None):
    return _lib.E4bNorm(T, H, dt, kind, eps, scale, post, pre, gate)


def _norm(n=None, x=FAKE, y=FAKE, r=FAKE, h=FAKE, ry=FAKE, rr=FAKE, **kw):
    n = n or _norm_desc(**kw)
    return e4b.load().e4b_block_norm(ctypes.byref(n), x, y, r, h, ry, rr, None)


def _norm_bwd(n=None, x=FAKE, y=FAKE, ry=FAKE, rr=FAKE, gr=FAKE, gh=FAKE, gx=FAKE, gy=FAKE, gg=None, gpost=FAKE,
              gpre=FAKE, ws=FAKE, ws_bytes=1 << 40, **kw):
    n = n or _norm_desc(**kw)
    return e4b.load().e4b_block_norm_backward(ctypes.byref(n), x, y, ry, rr, gr, gh, gx, gy, gg, gpost, gpre, ws,
                                              ws_bytes, None)


@pytest.mark.parametrize("call", [_norm, _norm_bwd])
def test_norm_descriptor(call):
    for kw in (dict(T=-1), dict(T=1 << 23), dict(H=0), dict(H=16385), dict(eps=0.0), dict(eps=-1e-6), dict(eps=math.nan),
               dict(kind=3, gate=FAKE), dict(kind=-1, gate=FAKE)):
        assert call(**kw) == L.E4B_ERR_SHAPE, kw
    assert call(dt=2) == L.E4B_ERR_DTYPE
    assert call(kind=1) == L.E4B_ERR_NULL  # a gate kind without a gate
    assert call(kind=0, gate=FAKE) == L.E4B_ERR_NULL  # and the reverse
    assert call(y=None) == L.E4B_ERR_NULL  # w_post acts on y
    assert call(y=None, post=None, kind=2, gate=FAKE) == L.E4B_ERR_NULL
    assert call(y=None, post=None, pre=None) == L.E4B_ERR_NULL
    for kw in (dict(post=FAKE + 4), dict(pre=FAKE + 4), dict(kind=1, gate=FAKE + 4)):
        assert call(**kw) == L.E4B_ERR_ALIGN, kw


def test_norm_pointers():
    for name in ("x", "r", "h", "ry", "rr"):
        assert _norm(**{name: None}) == L.E4B_ERR_NULL, name
    for name in ("x", "y", "r", "h", "ry", "rr"):
        assert _norm(**{name: FAKE + 4}) == L.E4B_ERR_ALIGN, name
    for name in ("x", "ry", "rr", "gh", "gx", "gy"):
        assert _norm_bwd(**{name: None}) == L.E4B_ERR_NULL, name
    # column gradients over more than a few rows take the workspace
    assert _norm_bwd(T=100, ws=None) == L.E4B_ERR_NULL
    n = _norm_desc(T=100)
    need = e4b.load().e4b_block_norm_workspace_bytes(ctypes.byref(n))
    assert need > 0 and _norm_bwd(n=n, ws_bytes=need - 1) == L.E4B_ERR_WORKSPACE
    n = _norm_desc(T=4)
    assert e4b.load().e4b_block_norm_workspace_bytes(ctypes.byref(n)) == 0
    assert _norm_bwd(gr=None, pre=None, gpre=None) == L.E4B_ERR_NULL  # then nothing reaches r
    assert _norm_bwd(gg=FAKE) == L.E4B_ERR_NULL  # the gradient of a gate that is not there
    assert _norm_bwd(pre=None, gpre=FAKE) == L.E4B_ERR_NULL
    assert _norm_bwd(post=None, gpost=FAKE) == L.E4B_ERR_NULL
    assert _norm_bwd(T=100, gpost=None, ws=None) == L.E4B_ERR_NULL  # one column gradient is enough to need it
    for name in ("x", "y", "ry", "rr", "gr", "gh", "gx", "gy", "gpost", "gpre", "ws"):
        assert _norm_bwd(**{name: FAKE + 4}) == L.E4B_ERR_ALIGN, name
    assert _norm(T=0, x=None, r=None, h=None, ry=None, rr=None) == L.E4B_OK
    assert _norm(T=0, x=None, y=None, r=None, h=None, ry=None, rr=None, kind=1, gate=FAKE) == L.E4B_OK


def test_status_text_of_an_activation():
    assert _lib.status_string(L.E4B_ERR_ACT) == "unknown activation"


def test_python_checks():
    """Host tensors, wrong types and shapes are refused before any device call."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    st = e4b.QuantStack(torch.zeros(1, 64 * 32, dtype=torch.uint8), torch.zeros(1, 64), 1, 64, 64)
    perm = e4b.Permutation(torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), ids)
    with pytest.raises(ValueError, match="device tensor"):
        e4b.moe_route(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError, match="float32"):
        e4b.moe_route(x, 2)
    with pytest.raises(TypeError, match="int32"):
        e4b.moe_permute(ids.long(), 8, x)
    with pytest.raises(ValueError, match="device tensor"):
        e4b.moe_permute(ids, 8, x)
    with pytest.raises(ValueError, match="device tensor"):
        e4b.moe_unpermute(perm, x)
    with pytest.raises(ValueError, match="device tensor"):
        e4b.moe_unpermute_backward(perm, x, x)
    with pytest.raises(TypeError, match="bfloat16"):
        e4b.expert_linear(st, x.float())
    with pytest.raises(ValueError, match="device tensor"):
        e4b.expert_linear(st, x)
    with pytest.raises(ValueError, match="device tensor"):
        e4b.expert_linear_dgrad(st, x)
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        e4b.block_norm(x.half(), w_pre=torch.ones(64))
    with pytest.raises(ValueError, match="device tensor"):
        e4b.block_norm(x, w_pre=torch.ones(64))
