"""What a MoE block needs around its expert MLP: the router with the gradient of
its logits and the losses that keep its experts evenly used, tokens into expert
order and back, the product of expert rows with a stored stack and an epilogue,
the norms before and after a block.

Like the rest of the package these functions check torch tensors and marshal
them into ``libe4b.so``; forwards and gradients are explicit calls. Each runs on
the current stream of its tensors' device.
"""

import ctypes
from dataclasses import dataclass

import torch

from . import _lib, _need, _need_buffer, _vp
from ._lib import E4bBalance, E4bNorm, check, load

ACTS = {"none": _lib.E4B_ACT_NONE, "relu": _lib.E4B_ACT_RELU, "silu": _lib.E4B_ACT_SILU,
        "gelu": _lib.E4B_ACT_GELU, "gelu_tanh": _lib.E4B_ACT_GELU_TANH}
_DTYPES = {torch.float32: _lib.E4B_F32, torch.bfloat16: _lib.E4B_BF16}


# the current stream's handle without the Stream object that torch.cuda.current_stream makes
# (1.9 us of a call whose launch takes 3.3); torch.cuda.current_stream where torch has no such function
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(name, device, *args):
    """Call entry point ``name`` on the current stream of ``device``."""
    fn = getattr(load(), name)
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            code = fn(*args, _raw_stream(index))
    else:
        code = fn(*args, _raw_stream(index))
    if code:
        check(name, code)


def _dtype(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return code


def _rows(t, name, device=None, shape=None):
    """A contiguous [n, H] device tensor in bf16 or fp32; its dtype code."""
    code = _dtype(t, name)
    _need(t, name, t.dtype, device, shape)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(t.shape)}")
    return code


def _workspace(ws, need, device):
    """(the buffer to keep alive, its address, its bytes); a call that needs none gets none"""
    if ws is None:
        if not need:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _need_buffer(ws, "workspace", need, device)
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _overlap(a, b):
    lo = max(a.data_ptr(), b.data_ptr())
    return lo < min(a.data_ptr() + a.numel() * a.element_size(), b.data_ptr() + b.numel() * b.element_size())


# ---- the router ----


def moe_route(logits, top_k):
    """Top-k of router logits and the softmax over the selected ones.

    ``logits`` float32 [T, E], finite or -inf (an expert out of service: weight 0).
    Returns ``(topk_idx int32 [T, k], topk_w float32 [T, k])``, the routing that
    ``moe_forward`` makes from the same logits; a row that is -inf throughout
    gets weights 0.
    """
    _need(logits, "logits", torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    dev = logits.device
    k = max(int(top_k), 0)
    idx = torch.empty(T, k, dtype=torch.int32, device=dev)
    w = torch.empty(T, k, dtype=torch.float32, device=dev)
    _run("e4b_route", dev, logits.data_ptr(), T, E, int(top_k), idx.data_ptr(), w.data_ptr())
    return idx, w


def moe_route_backward(topk_idx, topk_w, grad_topk_w, E):
    """Gradient of the logits [T, E] from that of the routing weights (the
    ``grad_topk_w`` of ``moe_dgrad`` or ``moe_unpermute_backward``), the selection
    held fixed."""
    _need(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, k]")
    dev = topk_idx.device
    _need(topk_w, "topk_w", torch.float32, dev, topk_idx.shape)
    _need(grad_topk_w, "grad_topk_w", torch.float32, dev, topk_idx.shape)
    T, k = topk_idx.shape
    out = torch.empty(T, max(int(E), 0), dtype=torch.float32, device=dev)
    _run("e4b_route_backward", dev, topk_idx.data_ptr(), topk_w.data_ptr(), grad_topk_w.data_ptr(), T, int(E), k,
         out.data_ptr())
    return out


@dataclass
class Balance:
    """``moe_balance``'s results for S sequences: ``counts`` int32 [S, E] (pairs of each
    expert), ``tokens`` int32 [S] (counted tokens), ``prob`` float32 [S, E] (sums of the
    router's probabilities), ``loss`` and ``z_loss`` float32 [S], ``lse`` float32 [T]
    (-inf for a token that is not counted), and the ``top_k`` they were made with."""

    counts: torch.Tensor
    tokens: torch.Tensor
    prob: torch.Tensor
    loss: torch.Tensor
    z_loss: torch.Tensor
    lse: torch.Tensor
    top_k: int


def _aligned(t):
    """(``t``, its address), or a copy's where a view begins off the library's 16 bytes"""
    if t is None:
        return None, None
    at = t.data_ptr()
    if at % 16:
        t = t.clone()
        at = t.data_ptr()
    return t, at


def _balance_args(logits, top_k, cu_tokens, token_mask):
    """(the C descriptor, sequences, the tensors that it points to)"""
    _need(logits, "logits", torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    dev = logits.device
    S = 1
    if cu_tokens is not None:
        _need(cu_tokens, "cu_tokens", torch.int32, dev)
        if cu_tokens.dim() != 1 or cu_tokens.shape[0] < 2:
            raise ValueError("cu_tokens must be [sequences + 1]")
        S = cu_tokens.shape[0] - 1
    if token_mask is not None:
        _need(token_mask, "token_mask", torch.bool, dev, (T,))
    # a batch's part of longer bounds or of a longer mask, mask[a:b], begins anywhere
    cu_tokens, cu = _aligned(cu_tokens)
    token_mask, mask = _aligned(token_mask)
    return E4bBalance(T, E, S, int(top_k), cu, mask), S, (cu_tokens, token_mask)


def moe_balance(logits, topk_idx, cu_tokens=None, token_mask=None, workspace=None):
    """How evenly a router uses its experts, and the losses that keep it even: a ``Balance``.

    ``logits`` float32 [T, E] (entries may be -inf), ``topk_idx`` int32 [T, k] as
    ``moe_route`` gives them (an id outside [0, E) is no expert's). ``cu_tokens`` int32
    [S + 1]: sequence s has tokens cu_tokens[s] .. cu_tokens[s + 1] - 1 and losses of its
    own (None: one sequence of all tokens). ``token_mask`` bool [T], False for tokens that
    are not counted, as padding; nor are those of no sequence and those with logits of -inf throughout.
    Both, and ``topk_idx``, may be parts of longer tensors (one that begins off 16 bytes is copied first).
    With N counted tokens and p the softmax of all logits,
    loss = E / (k N^2) sum_e counts_e prob_e (1 for an even use) and
    z_loss = 1 / N sum_t (log sum_e exp l_te)^2; both are 0 for a sequence without a token.
    """
    _need(logits, "logits", torch.float32)
    dev = logits.device
    _need(topk_idx, "topk_idx", torch.int32, dev)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, k]")
    k = topk_idx.shape[1]
    b, S, _held = _balance_args(logits, k, cu_tokens, token_mask)
    topk_idx, idx = _aligned(topk_idx)
    T, E = logits.shape
    if topk_idx.shape[0] != T:
        raise ValueError(f"topk_idx must have {T} rows, got {topk_idx.shape[0]}")
    counts = torch.empty(S, E, dtype=torch.int32, device=dev)
    tokens = torch.empty(S, dtype=torch.int32, device=dev)
    prob = torch.empty(S, E, dtype=torch.float32, device=dev)
    loss = torch.empty(S, dtype=torch.float32, device=dev)
    z = torch.empty(S, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    ws, at, nbytes = _workspace(workspace, int(load().e4b_moe_balance_workspace_bytes(ctypes.byref(b))), dev)
    _run("e4b_moe_balance", dev, ctypes.byref(b), logits.data_ptr(), idx, counts.data_ptr(),
         tokens.data_ptr(), prob.data_ptr(), loss.data_ptr(), z.data_ptr(), lse.data_ptr(), at, nbytes)
    return Balance(counts, tokens, prob, loss, z, lse, k)


def moe_balance_workspace_bytes(logits, top_k, cu_tokens=None):
    """Bytes of ``moe_balance``'s workspace for these arguments."""
    b, _, _held = _balance_args(logits, top_k, cu_tokens, None)
    return int(load().e4b_moe_balance_workspace_bytes(ctypes.byref(b)))


def moe_balance_backward(fwd, logits, grad_loss=None, grad_z=None, cu_tokens=None, add=None, out=None):
    """Gradient [T, E] of the logits of sum(grad_loss loss) + sum(grad_z z_loss), the
    selection held fixed, plus ``add``.

    ``fwd`` is ``moe_balance``'s result and ``cu_tokens`` its argument; ``grad_loss`` and
    ``grad_z`` float32 [S], which may be parts of longer tensors (None: zeros); ``add``
    float32 [T, E], as ``moe_route_backward`` gives it; ``out`` the result's place, which may
    be ``add``. Tokens that are not counted get ``add`` alone. With ``fwd.counts`` and ``fwd.tokens`` summed over ranks first, the
    gradient is that of the loss over all ranks' tokens.
    """
    b, S, _held = _balance_args(logits, fwd.top_k, cu_tokens, None)
    T, E = logits.shape
    dev = logits.device
    _need(fwd.counts, "counts", torch.int32, dev, (S, E))
    _need(fwd.tokens, "tokens", torch.int32, dev, (S,))
    _need(fwd.lse, "lse", torch.float32, dev, (T,))
    for t, name, shape in ((grad_loss, "grad_loss", (S,)), (grad_z, "grad_z", (S,)), (add, "add", (T, E)),
                           (out, "out", (T, E))):
        if t is not None:
            _need(t, name, torch.float32, dev, shape)
    if out is None:
        out = torch.empty(T, E, dtype=torch.float32, device=dev)
    elif any(t is not None and _overlap(out, t)
             for t in (logits, fwd.counts, fwd.tokens, fwd.lse, grad_loss, grad_z, cu_tokens)) or (
            add is not None and _overlap(out, add) and out.data_ptr() != add.data_ptr()):
        raise ValueError("out must not overlap what the call reads, but that it may be add")
    grad_loss, gl = _aligned(grad_loss)
    grad_z, gz = _aligned(grad_z)
    _run("e4b_moe_balance_backward", dev, ctypes.byref(b), logits.data_ptr(), fwd.counts.data_ptr(),
         fwd.tokens.data_ptr(), fwd.lse.data_ptr(), gl, gz, None if add is None else add.data_ptr(), out.data_ptr())
    return out


# ---- tokens into expert order and back ----


@dataclass
class Permutation:
    """The expert order of T tokens' k routed pairs: ``offsets`` int32 [E + 1]
    (first row of each expert; offsets[E] = pairs that have one), ``sorted_pair``
    int32 [T k] (pair t k + j at each row), ``pos`` int32 [T, k] (row of each pair)."""

    offsets: torch.Tensor
    sorted_pair: torch.Tensor
    pos: torch.Tensor

    @property
    def T(self):
        return self.pos.shape[0]

    @property
    def top_k(self):
        return self.pos.shape[1]

    @property
    def E(self):
        return self.offsets.shape[0] - 1

    def check(self):
        _need(self.offsets, "offsets", torch.int32)
        if self.offsets.dim() != 1:
            raise ValueError("offsets must be [E + 1]")
        dev = self.offsets.device
        _need(self.pos, "pos", torch.int32, dev)
        if self.pos.dim() != 2:
            raise ValueError("pos must be [T, k]")
        return dev


def moe_permute(topk_idx, E, x=None):
    """Tokens into expert order: ``(rows [T k, H] or None, Permutation)``.

    ``topk_idx`` int32 [T, k]; a pair whose id lies outside [0, E) goes to no expert
    (a padding token, an expert of another rank): it comes last and its row is
    zeros. ``x`` [T, H] in bfloat16 or float32; without it only the order is made.
    """
    _need(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, k]")
    T, k = topk_idx.shape
    dev = topk_idx.device
    E = int(E)
    code, H, rows = _lib.E4B_BF16, 1, None
    if x is not None:
        code = _rows(x, "x", dev)
        if x.shape[0] != T:
            raise ValueError(f"x must have {T} rows, got {x.shape[0]}")
        H = x.shape[1]
        rows = torch.empty(T * k, H, dtype=x.dtype, device=dev)
    offsets = torch.empty(max(E, 0) + 1, dtype=torch.int32, device=dev)
    order = torch.empty(T * k, dtype=torch.int32, device=dev)
    pos = torch.empty(T, k, dtype=torch.int32, device=dev)
    _run("e4b_permute", dev, T, k, E, H, code, topk_idx.data_ptr(), None if x is None else x.data_ptr(),
         None if x is None else rows.data_ptr(), offsets.data_ptr(), order.data_ptr(), pos.data_ptr())
    return rows, Permutation(offsets, order, pos)


def _unpermute(perm, rows, name, topk_w):
    dev = perm.check()
    T, k = perm.pos.shape
    code = _rows(rows, name, dev)
    if rows.shape[0] != T * k:
        raise ValueError(f"{name} must have {T * k} rows, got {rows.shape[0]}")
    if topk_w is not None:
        _need(topk_w, "topk_w", torch.float32, dev, (T, k))
    H = rows.shape[1]
    y = torch.empty(T, H, dtype=rows.dtype, device=dev)
    _run("e4b_unpermute", dev, T, k, perm.E, H, code, perm.offsets.data_ptr(), perm.pos.data_ptr(),
         None if topk_w is None else topk_w.data_ptr(), rows.data_ptr(), y.data_ptr())
    return y


def moe_permute_backward(perm, grad_rows):
    """Gradient of ``moe_permute``'s x: the sum of each token's rows of ``grad_rows``."""
    return _unpermute(perm, grad_rows, "grad_rows", None)


def moe_unpermute(perm, rows, topk_w=None):
    """Back into token order: y[t] = sum_j topk_w[t, j] rows[pos(t, j)] (weights of 1
    without ``topk_w``); pairs without an expert add nothing."""
    return _unpermute(perm, rows, "rows", topk_w)


def moe_unpermute_backward(perm, rows, grad_y, topk_w=None, grad_w=True):
    """Gradients of ``moe_unpermute``: ``(grad_rows, grad_topk_w float32 [T, k] or None)``.
    ``rows`` is needed for ``grad_w`` only."""
    dev = perm.check()
    T, k = perm.pos.shape
    code = _rows(grad_y, "grad_y", dev)
    if grad_y.shape[0] != T:
        raise ValueError(f"grad_y must have {T} rows, got {grad_y.shape[0]}")
    H = grad_y.shape[1]
    if topk_w is not None:
        _need(topk_w, "topk_w", torch.float32, dev, (T, k))
    if grad_w:
        if rows is None:
            raise ValueError("grad_w needs rows")
        _need(rows, "rows", grad_y.dtype, dev, (T * k, H))
    grad_rows = torch.empty(T * k, H, dtype=grad_y.dtype, device=dev)
    gw = torch.empty(T, k, dtype=torch.float32, device=dev) if grad_w else None
    _run("e4b_unpermute_backward", dev, T, k, perm.E, H, code, perm.offsets.data_ptr(), perm.pos.data_ptr(),
         None if topk_w is None else topk_w.data_ptr(), rows.data_ptr() if grad_w else None, grad_y.data_ptr(),
         grad_rows.data_ptr(), gw.data_ptr() if grad_w else None)
    return grad_rows, gw


# ---- products with a stored stack ----


def _linear_args(stack, rows, offsets, bias, act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    dev = stack.device
    if offsets is None:
        if stack.E != 1:
            raise ValueError("a stack of several experts needs offsets")
    else:
        _need(offsets, "offsets", torch.int32, dev, (stack.E + 1,))
    if bias is not None:
        _need(bias, "bias", torch.float32, dev, (stack.E, stack.out))
    return dev


def expert_linear_workspace_bytes(stack, rows):
    c = stack.as_c()
    return int(load().e4b_expert_linear_workspace_bytes(ctypes.byref(c), rows))


def expert_linear_dgrad_workspace_bytes(stack, rows, recompute=False):
    c = stack.as_c()
    return int(load().e4b_expert_linear_dgrad_workspace_bytes(ctypes.byref(c), rows, int(recompute)))


def expert_linear(stack, x, offsets=None, bias=None, act="none", residual=None, out_dtype=torch.bfloat16, save=False,
                  workspace=None, out=None):
    """y = act(W[e] x + bias[e]) + residual for expert-sorted rows.

    ``stack`` any QuantStack; ``x`` bfloat16 [rows, in]; ``offsets`` int32 [E + 1]
    (``Permutation.offsets``; None for a stack of one expert, which then takes every
    row); ``bias`` float32 [E, out]; ``act`` one of none, relu, silu, gelu, gelu_tanh;
    ``residual`` bfloat16 [rows, out]. Rows from offsets[E] on come out as zeros.
    ``save`` keeps the fp32 pre-activation for the gradient. ``out`` may be the
    residual itself (added in place); it must not overlap x.
    Returns ``(y [rows, out] in out_dtype, pre float32 [rows, out] or None)``.
    """
    _need(x, "x", torch.bfloat16, stack.device)
    if x.dim() != 2 or x.shape[1] != stack.inn:
        raise ValueError(f"x must be [rows, {stack.inn}], got {tuple(x.shape)}")
    rows = x.shape[0]
    dev = _linear_args(stack, rows, offsets, bias, act)
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, dev, (rows, stack.out))
    if out_dtype not in _DTYPES:
        raise ValueError("out_dtype must be float32 or bfloat16")
    if out is None:
        y = torch.empty(rows, stack.out, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", out_dtype, dev, (rows, stack.out))
        if _overlap(out, x) or (residual is not None and _overlap(out, residual)
                                and (out.data_ptr() != residual.data_ptr() or out_dtype != residual.dtype)):
            raise ValueError("out must not overlap x, nor the residual unless it is the residual")
        y = out
    pre = torch.empty(rows, stack.out, dtype=torch.float32, device=dev) if save else None
    c = stack.as_c()
    st = ctypes.byref(c)
    ws, at, nbytes = _workspace(workspace, int(load().e4b_expert_linear_workspace_bytes(st, rows)), dev)
    _run("e4b_expert_linear", dev, st, rows, _vp(offsets), x.data_ptr(), _vp(bias), ACTS[act], _vp(residual),
         _DTYPES[out_dtype], y.data_ptr(), _vp(pre), at, nbytes)
    return y, pre


def expert_linear_dgrad(stack, grad_y, x=None, offsets=None, bias=None, act="none", pre=None, grad_bias=False,
                        workspace=None):
    """Gradients of ``expert_linear`` over a frozen stack:
    ``(grad_x bfloat16 [rows, in], grad_bias float32 [E, out] or None)``.

    An activation needs the forward's ``pre``, or ``x`` and ``bias`` to compute it
    again (bit for bit). The residual's gradient is ``grad_y`` itself.
    """
    code = _rows(grad_y, "grad_y", stack.device)
    rows = grad_y.shape[0]
    if grad_y.shape[1] != stack.out:
        raise ValueError(f"grad_y must be [rows, {stack.out}], got {tuple(grad_y.shape)}")
    dev = _linear_args(stack, rows, offsets, bias, act)
    recompute = False
    if act != "none":
        if pre is not None:
            _need(pre, "pre", torch.float32, dev, (rows, stack.out))
        elif x is None:
            raise ValueError("give pre, or x (and bias) to recompute it")
        else:
            _need(x, "x", torch.bfloat16, dev, (rows, stack.inn))
            recompute = True
    gx = torch.empty(rows, stack.inn, dtype=torch.bfloat16, device=dev)
    gb = torch.empty(stack.E, stack.out, dtype=torch.float32, device=dev) if grad_bias else None
    c = stack.as_c()
    st = ctypes.byref(c)
    need = int(load().e4b_expert_linear_dgrad_workspace_bytes(st, rows, int(recompute)))
    ws, at, nbytes = _workspace(workspace, need, dev)
    _run("e4b_expert_linear_dgrad", dev, st, rows, _vp(offsets), grad_y.data_ptr(), code,
         None if act == "none" else _vp(pre), x.data_ptr() if recompute else None,
         _vp(bias) if recompute else None, ACTS[act], gx.data_ptr(), _vp(gb), at, nbytes)
    return gx, gb


# ---- the norms around a block ----


@dataclass
class BlockNorm:
    """``block_norm``'s results: the residual stream ``r`` (x itself without y), the
    next block's input ``h``, and the row statistics its gradient needs (``rstd``
    float32 [2, T rounded up to 4]: 1 / rms of y's rows, then of r's; a row that its
    norm does not have is not written)."""

    r: torch.Tensor
    h: torch.Tensor
    rstd: torch.Tensor


@dataclass
class BlockNormGrads:
    """``block_norm_backward``'s results; None for what was not there."""

    grad_x: torch.Tensor
    grad_y: torch.Tensor
    grad_gate: torch.Tensor
    grad_w_post: torch.Tensor
    grad_w_pre: torch.Tensor


def _norm_args(x, y, w_post, gate_token, gate_channel, scale, w_pre, eps):
    code = _rows(x, "x")
    T, H = x.shape
    dev = x.device
    if y is not None:
        _need(y, "y", torch.bfloat16, dev, (T, H))
    elif w_post is not None or gate_token is not None or gate_channel is not None:
        raise ValueError("w_post and the gates act on y: give y")
    elif w_pre is None:
        raise ValueError("give y, w_pre or both")
    if gate_token is not None and gate_channel is not None:
        raise ValueError("give gate_token or gate_channel, not both")
    for t, name, shape in ((w_post, "w_post", (H,)), (w_pre, "w_pre", (H,)), (gate_token, "gate_token", (T,)),
                           (gate_channel, "gate_channel", (H,))):
        if t is not None:
            _need(t, name, torch.float32, dev, shape)
    gate = gate_channel if gate_token is None else gate_token
    kind = (_lib.E4B_GATE_NONE if gate is None else
            _lib.E4B_GATE_CHANNEL if gate_token is None else _lib.E4B_GATE_TOKEN)
    return dev, T, H, gate, E4bNorm(T, H, code, kind, eps, scale, None if w_post is None else w_post.data_ptr(),
                                    None if w_pre is None else w_pre.data_ptr(),
                                    # an empty batch's gate has no address
                                    None if gate is None else gate.data_ptr() or 16)


def block_norm(x, y=None, w_post=None, gate_token=None, gate_channel=None, scale=1.0, w_pre=None, eps=1e-6):
    """r = x + scale g N(y) w_post and h = N(r) w_pre, N the RMS norm of a row.

    ``x`` [T, H] in bfloat16 or float32 is the residual stream, ``y`` bfloat16 [T, H]
    a block's output; ``w_post`` / ``w_pre`` float32 [H] (no post-norm / no h without
    them); the gate g is ``gate_token`` float32 [T] or ``gate_channel`` float32 [H].
    Without y only h = N(x) w_pre is made. Returns a ``BlockNorm``.
    """
    dev, T, H, _, n = _norm_args(x, y, w_post, gate_token, gate_channel, scale, w_pre, eps)
    r = torch.empty_like(x) if y is not None else None
    h = torch.empty(T, H, dtype=torch.bfloat16, device=dev) if w_pre is not None else None
    rstd = torch.empty(2, -(-T // 4) * 4, dtype=torch.float32, device=dev)
    rstd_y, rstd_r = _rstd(rstd)
    _run("e4b_block_norm", dev, ctypes.byref(n), x.data_ptr(), _vp(y), _vp(r), _vp(h), rstd_y, rstd_r)
    return BlockNorm(x if r is None else r, h, rstd)


def _rstd(rstd):
    """The addresses of its two rows."""
    p = rstd.data_ptr()
    return p, p + rstd.shape[1] * 4


def block_norm_backward(fwd, x, grad_r=None, grad_h=None, y=None, w_post=None, gate_token=None, gate_channel=None,
                        scale=1.0, w_pre=None, eps=1e-6, weight_grads=True, workspace=None):
    """Gradients of sum(grad_r r) + sum(grad_h h): a ``BlockNormGrads``.

    ``fwd`` is ``block_norm``'s result and the other arguments its arguments;
    ``grad_r`` [T, H] as x (None: zeros, with w_pre), ``grad_h`` bfloat16 [T, H] (with
    w_pre). ``weight_grads=False`` leaves out those of w_post, w_pre and
    gate_channel.
    """
    dev, T, H, gate, n = _norm_args(x, y, w_post, gate_token, gate_channel, scale, w_pre, eps)
    if w_pre is not None:
        if grad_h is None:
            raise ValueError("w_pre needs grad_h")
        _need(grad_h, "grad_h", torch.bfloat16, dev, (T, H))
    elif grad_r is None:
        raise ValueError("give grad_r")
    if grad_r is not None:
        _need(grad_r, "grad_r", x.dtype, dev, (T, H))
    _need(fwd.rstd, "rstd", torch.float32, dev, (2, -(-T // 4) * 4))
    rstd_y, rstd_r = _rstd(fwd.rstd)
    gx = torch.empty_like(x)
    gy = torch.empty_like(y) if y is not None else None
    gg = torch.empty_like(gate) if gate is not None and (weight_grads or gate_token is not None) else None
    gpost = torch.empty_like(w_post) if w_post is not None and weight_grads else None
    gpre = torch.empty_like(w_pre) if w_pre is not None and weight_grads else None
    # the column gradients' partial sums
    need = 0
    if gpost is not None or gpre is not None or (gg is not None and gate_channel is not None):
        need = int(load().e4b_block_norm_workspace_bytes(ctypes.byref(n)))
    ws, at, nbytes = _workspace(workspace, need, dev)
    _run("e4b_block_norm_backward", dev, ctypes.byref(n), x.data_ptr(), _vp(y), rstd_y, rstd_r,
         _vp(grad_r), _vp(grad_h) if w_pre is not None else None, gx.data_ptr(), _vp(gy), _vp(gg), _vp(gpost),
         _vp(gpre), at, nbytes)
    return BlockNormGrads(gx, gy, gg, gpost, gpre)


def block_norm_workspace_bytes(x, y=None, w_post=None, gate_token=None, gate_channel=None, scale=1.0, w_pre=None,
                               eps=1e-6):
    """Bytes of ``block_norm_backward``'s workspace for these arguments."""
    n = _norm_args(x, y, w_post, gate_token, gate_channel, scale, w_pre, eps)[-1]
    return int(load().e4b_block_norm_workspace_bytes(ctypes.byref(n)))
