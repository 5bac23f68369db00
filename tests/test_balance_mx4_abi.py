"""Refusals of the router's balance, the microscaled rows and their product, none of which
needs a GPU: the C entry points report a bad argument before any device call, and the
Python functions before they touch the library."""

import ctypes

import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
from bit_quantized_mixture_nf4_amd import _lib

FAKE = 0x10000  # 16-byte aligned, never dereferenced on these paths
L = _lib


def _b(T=4, E=8, S=1, k=2, cu=None, mask=None):
    return _lib.E4bBalance(T, E, S, k, cu, mask)


def _fwd(b=None, logits=FAKE, idx=FAKE, counts=FAKE, tokens=FAKE, prob=FAKE, loss=FAKE, z=FAKE, lse=FAKE, ws=FAKE,
         ws_bytes=1 << 40, **kw):
    return e4b.load().e4b_moe_balance(ctypes.byref(b or _b(**kw)), logits, idx, counts, tokens, prob, loss, z, lse, ws,
                                      ws_bytes, None)


def _bwd(b=None, logits=FAKE, counts=FAKE, tokens=FAKE, lse=FAKE, gl=FAKE, gz=FAKE, add=FAKE, out=FAKE, **kw):
    return e4b.load().e4b_moe_balance_backward(ctypes.byref(b or _b(**kw)), logits, counts, tokens, lse, gl, gz, add, out,
                                               None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_balance_shapes(call):
    for kw in (dict(T=-1), dict(T=1 << 24), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, k=33), dict(S=0),
               dict(S=65537, cu=FAKE)):
        assert call(**kw) == L.E4B_ERR_SHAPE, kw
    assert call(S=2) == L.E4B_ERR_NULL  # several sequences need their bounds
    assert call(cu=FAKE + 4) == L.E4B_ERR_ALIGN
    assert call(mask=FAKE + 1) == L.E4B_ERR_ALIGN


def test_balance_pointers():
    for name in ("logits", "idx", "counts", "tokens", "prob", "loss", "z", "lse"):
        assert _fwd(T=100, **{name: None}) == L.E4B_ERR_NULL, name
        assert _fwd(T=100, **{name: FAKE + 4}) == L.E4B_ERR_ALIGN, name
    for name in ("logits", "counts", "tokens", "lse", "out"):
        assert _bwd(**{name: None}) == L.E4B_ERR_NULL, name
    for name in ("logits", "counts", "tokens", "lse", "gl", "gz", "add", "out"):
        assert _bwd(**{name: FAKE + 8}) == L.E4B_ERR_ALIGN, name
    assert e4b.load().e4b_moe_balance(None, *[FAKE] * 9, 1 << 40, None) == L.E4B_ERR_NULL
    assert _bwd(T=0, logits=None, counts=None, tokens=None, lse=None, out=None) == L.E4B_OK


def test_balance_workspace():
    need = lambda **kw: e4b.load().e4b_moe_balance_workspace_bytes(ctypes.byref(_b(**kw)))  # noqa: E731
    assert need(T=64) == 0 and need(T=0, S=3, cu=FAKE) == 0 and need(T=-1) == 0
    for kw in (dict(T=65), dict(T=8, S=3, cu=FAKE), dict(T=70000, E=257, S=9, cu=FAKE)):
        n = need(**kw)
        assert n > 0
        assert _fwd(ws_bytes=n - 1, **kw) == L.E4B_ERR_WORKSPACE
        assert _fwd(ws=None, **kw) == L.E4B_ERR_NULL
        assert _fwd(ws=FAKE + 8, **kw) == L.E4B_ERR_ALIGN


def _rows(x=FAKE, dt=1, n=4, K=64, gated=0, codes=FAKE, scales=FAKE):
    return e4b.load().e4b_mx4_rows(x, dt, n, K, gated, codes, scales, None)


def _rows_bwd(x=FAKE, dt=1, g=FAKE, gdt=1, n=4, K=64, gx=FAKE):
    return e4b.load().e4b_mx4_rows_backward(x, dt, g, gdt, n, K, gx, None)


def test_rows_refusals():
    for kw in (dict(n=-1), dict(K=0), dict(K=32), dict(K=96), dict(K=(1 << 20) + 64), dict(n=(1 << 30) + 1),
               dict(n=1 << 30, K=64), dict(n=1 << 15, K=1 << 20)):
        assert _rows(**kw) == L.E4B_ERR_SHAPE, kw
        assert _rows_bwd(**kw) == L.E4B_ERR_SHAPE, kw
    assert _rows(dt=2) == _rows_bwd(dt=-1) == _rows_bwd(gdt=7) == L.E4B_ERR_DTYPE
    for name in ("x", "codes", "scales"):
        assert _rows(**{name: None}) == L.E4B_ERR_NULL
        assert _rows(**{name: FAKE + 8}) == L.E4B_ERR_ALIGN
    for name in ("x", "g", "gx"):
        assert _rows_bwd(**{name: None}) == L.E4B_ERR_NULL
        assert _rows_bwd(**{name: FAKE + 8}) == L.E4B_ERR_ALIGN
    assert _rows(n=0, x=None, codes=None, scales=None) == L.E4B_OK
    assert _rows_bwd(n=0, x=None, g=None, gx=None) == L.E4B_OK


def _stack(E=1, out=64, inn=64, cb=3, packed=FAKE, bs=32, scales=FAKE):
    return _lib.E4bStack(packed, FAKE, E, out, inn, bs, cb, scales)


def _linear(st=None, rows=4, off=None, order=None, k=1, x=FAKE, xs=FAKE, bias=FAKE, act=0, res=FAKE, dt=1, y=FAKE, pre=FAKE,
            ws=FAKE, ws_bytes=1 << 40):
    st = st or _stack()
    return e4b.load().e4b_mx_linear(ctypes.byref(st), rows, off, order, k, x, xs, bias, act, res, dt, y, pre, ws, ws_bytes,
                                    None)


def test_product_refusals():
    assert _linear(st=_stack(cb=0, bs=64)) == L.E4B_ERR_CODEBOOK  # NF4
    assert _linear(st=_stack(cb=2, bs=64)) == L.E4B_ERR_CODEBOOK  # bf16
    assert _linear(st=_stack(bs=64)) == L.E4B_ERR_BLOCKSIZE
    assert _linear(st=_stack(inn=96)) == L.E4B_ERR_SHAPE
    assert _linear(st=_stack(E=1025), off=FAKE) == L.E4B_ERR_SHAPE
    assert _linear(rows=-1) == _linear(rows=(1 << 30) + 1) == L.E4B_ERR_SHAPE
    assert _linear(st=_stack(out=(1 << 20) + 1)) == L.E4B_ERR_SHAPE
    assert _linear(act=5) == _linear(act=-1) == L.E4B_ERR_ACT
    assert _linear(dt=2) == L.E4B_ERR_DTYPE
    assert _linear(st=_stack(E=2)) == L.E4B_ERR_NULL  # several experts without offsets
    for k in (0, 33, 3):  # rows = 4
        assert _linear(order=FAKE, k=k) == L.E4B_ERR_SHAPE
    for name in ("x", "xs", "y"):
        assert _linear(**{name: None}) == L.E4B_ERR_NULL
    for name in ("x", "xs", "y", "bias", "res", "pre", "off", "order", "ws"):
        assert _linear(**{name: FAKE + 4}) == L.E4B_ERR_ALIGN, name
    assert _linear(st=_stack(packed=None)) == _linear(st=_stack(scales=None)) == L.E4B_ERR_NULL
    assert _linear(st=_stack(scales=FAKE + 4)) == L.E4B_ERR_ALIGN
    assert _linear(rows=0, x=None, xs=None, y=None) == L.E4B_OK


def test_product_workspace():
    need = lambda st, rows: e4b.load().e4b_mx_linear_workspace_bytes(ctypes.byref(st), rows)  # noqa: E731
    assert need(_stack(cb=0, bs=64), 4) == 0 and need(_stack(), -1) == 0 and need(_stack(), 0) == 0
    for st, rows in ((_stack(E=8, out=4096, inn=4096), 8192), (_stack(out=4096, inn=2048), 2048), (_stack(E=64, out=256), 6000)):
        n = need(st, rows)
        if n:
            assert _linear(st=st, rows=rows, off=FAKE, ws_bytes=n - 1) == L.E4B_ERR_WORKSPACE
            assert _linear(st=st, rows=rows, off=FAKE, ws=None) == L.E4B_ERR_NULL


def test_python_refusals_without_a_device():
    t = torch.zeros
    with pytest.raises(ValueError, match="device tensor"):
        e4b.moe_balance(t(4, 8), t(4, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="logits"):
        e4b.moe_balance(t(4, 8, dtype=torch.bfloat16), t(4, 2, dtype=torch.int32))
    with pytest.raises(TypeError):
        e4b.moe_balance([1.0], t(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        e4b.mx4_rows(t(4, 64))
    with pytest.raises(TypeError):
        e4b.mx4_rows(t(4, 64, dtype=torch.float16))
    with pytest.raises(TypeError):
        e4b.mx4_rows_backward(t(4, 128, dtype=torch.float64), t(4, 64))
    with pytest.raises(TypeError):
        e4b.mx4_values(e4b.MxRows(t(4, 32), t(4, 2)))
    with pytest.raises(ValueError, match="device tensor"):
        e4b.mx4_values(e4b.MxRows(t(4, 32, dtype=torch.uint8), t(4, 2, dtype=torch.uint8)))
