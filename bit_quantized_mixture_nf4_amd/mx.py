"""Microscaled 4-bit floating point: rows of activations in E2M1 codes with an E8M0
scale for every 32 elements, and their product with a stored MXFP4 stack.

The product multiplies both operands as they are stored, on gfx950's block-scaled
matrix instructions. Trained through, the rounding of the rows is passed straight
through: the gradient of a product is ``expert_linear_dgrad``'s over the same stack,
that of gated rows ``mx4_rows_backward``'s. Each function runs on the current stream of its
tensors' device.
"""

import ctypes
from dataclasses import dataclass

import torch

from . import CODEBOOKS, _need, _vp
from ._lib import E4bStack, load
from .block import ACTS, _DTYPES, _aligned, _linear_args, _overlap, _rows, _run, _workspace


@dataclass
class MxRows:
    """n rows of K values in microscaled 4-bit floats, in the layout of a stored MXFP4
    stack: ``codes`` uint8 [n, K/2] (even element in the high nibble), ``scales`` uint8
    [n, K/32] (E8M0). Parts of longer rows, codes[a:b] and scales[a:b], are rows too (scales
    that begin off 16 bytes are copied by each call)."""

    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def rows(self):
        return self.codes.shape[0]

    @property
    def K(self):
        return self.codes.shape[1] * 2

    @property
    def device(self):
        return self.codes.device

    def check(self):
        codes = self.codes
        _need(codes, "codes", torch.uint8)
        shape = codes.shape
        if len(shape) != 2 or shape[1] % 32 or shape[1] == 0:
            raise ValueError(f"codes must be [n, K/2] with K % 64 == 0, got {tuple(shape)}")
        dev = codes.device
        _need(self.scales, "scales", torch.uint8, dev, (shape[0], shape[1] // 16))
        return dev


def mx4_rows(x, gated=False):
    """``x`` [n, K] in bfloat16 or float32 as ``MxRows``, by the rule of ``quantize(..., "mxfp4")``.

    With ``gated``, ``x`` is [n, 2K] = [g | u] and silu(g) u is converted, without a
    rounding in between. A block of 32 that holds an infinity or a NaN reads as NaN. K % 64 == 0.
    """
    code = _rows(x, "x")
    n, K = x.shape
    if gated:
        if K % 2:
            raise ValueError(f"gated rows are [n, 2K], got {tuple(x.shape)}")
        K //= 2
    codes = torch.empty(n, K // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(n, K // 32, dtype=torch.uint8, device=x.device)
    _run("e4b_mx4_rows", x.device, x.data_ptr(), code, n, K, int(bool(gated)), codes.data_ptr(), scales.data_ptr())
    return MxRows(codes, scales)


def mx4_rows_backward(x, grad):
    """Gradient [n, 2K] (as ``x``) of ``mx4_rows(x, gated=True)``, straight through the rounding,
    from ``grad`` [n, K] in bfloat16 or float32. Rows that are not gated pass their gradient on."""
    code = _rows(x, "x")
    n, K2 = x.shape
    if K2 % 2:
        raise ValueError(f"gated rows are [n, 2K], got {tuple(x.shape)}")
    gcode = _rows(grad, "grad", x.device, (n, K2 // 2))
    out = torch.empty_like(x)
    _run("e4b_mx4_rows_backward", x.device, x.data_ptr(), code, grad.data_ptr(), gcode, n, K2 // 2, out.data_ptr())
    return out


def mx4_values(q, dtype=torch.bfloat16):
    """The values [n, K] that ``MxRows`` stand for, exact in float32 and bfloat16."""
    dev = q.check()
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    out = torch.empty(q.rows, q.K, dtype=dtype, device=dev)
    if q.rows:  # (as a stack of so many experts of one row, of which there may be as many as rows)
        _held, scales = _aligned(q.scales)
        c = E4bStack(q.codes.data_ptr(), None, q.rows, 1, q.K, 32, CODEBOOKS["mxfp4"], scales)
        _run("e4b_dequantize_nf4", dev, ctypes.byref(c), _DTYPES[dtype], out.data_ptr())
    return out


def mx_linear_workspace_bytes(stack, rows):
    c = stack.as_c()
    return int(load().e4b_mx_linear_workspace_bytes(ctypes.byref(c), rows))


def mx_linear(stack, q, offsets=None, perm=None, bias=None, act="none", residual=None, out_dtype=torch.bfloat16,
              save=False, workspace=None, out=None):
    """y = act(W[e] x + bias[e]) + residual for microscaled rows and an MXFP4 stack.

    ``q`` are the ``MxRows`` of expert-sorted rows, with ``offsets`` int32 [E + 1] (None for
    a stack of one expert); or, with ``perm`` (``moe_permute``'s ``Permutation``), of the
    T tokens: row r of the product is then pair perm.sorted_pair[r], and its token's row is
    read where it lies. ``bias``, ``act``, ``residual``, ``out`` and the rows of no expert
    are as in ``expert_linear``; ``save`` keeps the fp32 pre-activation, which
    ``expert_linear_dgrad`` takes as ``pre``.
    Returns ``(y [rows, out] in out_dtype, pre float32 [rows, out] or None)``.
    """
    dev = q.check()
    if q.device != stack.device:
        raise ValueError(f"the rows are on {q.device}, expected {stack.device}")
    if stack.codebook != "mxfp4":
        raise ValueError(f"the stack must be mxfp4, got {stack.codebook}")
    if q.K != stack.inn:
        raise ValueError(f"the rows must have {stack.inn} values, got {q.K}")
    rows, order, top_k = q.rows, None, 1
    if perm is not None:
        if offsets is not None:
            raise ValueError("give offsets or perm, not both")
        perm.check()
        T, top_k = perm.pos.shape
        if q.rows != T:
            raise ValueError(f"perm orders {T} tokens, got {q.rows} rows")
        rows, offsets, order = T * top_k, perm.offsets, perm.sorted_pair
        _need(order, "sorted_pair", torch.int32, dev, (rows,))
    _linear_args(stack, rows, offsets, bias, act)
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, dev, (rows, stack.out))
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be float32 or bfloat16")
    if out is None:
        y = torch.empty(rows, stack.out, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev, (rows, stack.out))
        if _overlap(out, q.codes) or _overlap(out, q.scales) or (
                residual is not None and _overlap(out, residual)
                and (out.data_ptr() != residual.data_ptr() or out_dtype != residual.dtype)):
            raise ValueError("out must not overlap the rows, nor the residual unless it is the residual")
        y = out
    pre = torch.empty(rows, stack.out, dtype=torch.float32, device=dev) if save else None
    _held, scales = _aligned(q.scales)
    c = stack.as_c()
    st = ctypes.byref(c)
    ws, at, nbytes = _workspace(workspace, int(load().e4b_mx_linear_workspace_bytes(st, rows)), dev)
    _run("e4b_mx_linear", dev, st, rows, _vp(offsets), _vp(order), top_k, q.codes.data_ptr(), scales,
         _vp(bias), ACTS[act], _vp(residual), _DTYPES[out_dtype], y.data_ptr(), _vp(pre), at, nbytes)
    return y, pre
