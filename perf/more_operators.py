"""Balancing a router and the experts' products in microscaled 4-bit floats, as measured cases.

Three operators, with their gradients:

* ``balance``: how evenly a router uses its experts: pairs and probability of each
  expert, the balance loss and the z loss of every sequence, and the gradient of the
  logits, added to the one that the routing weights gave;
* ``rows``:    rows of activations in E2M1 codes with an E8M0 scale for every 32 (the
  OCP MX v1.0 conversion), plain or of silu(g) u with its gradient;
* ``product``: such rows, by place or gathered by token, times a stored stack of the
  same format, with bias, activation and residual in the epilogue.

``run`` computes them in elementary torch operations, or, where ``own`` is set,
through the library's entry points. ``exact`` computes them in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_T = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases ----

def _balance(T, E, k, way, seqs=1, masked=False, **kw):
    return dict(op="balance", T=T, E=E, k=k, way=way, seqs=seqs, masked=masked, **kw)


def _rows(n, K, way, dtype="bf16", gated=False, **kw):
    return dict(op="rows", n=n, K=K, way=way, dtype=dtype, gated=gated, **kw)


def _product(rows, E, inn, out, act="none", k=0, touched=0, bias=False, residual=False, y="bf16", save=False, tail=0,
             skew=0.0, drop=0.0, **kw):
    return dict(op="product", rows=rows, E=E, inn=inn, out=out, act=act, k=k, touched=touched, bias=bias,
                residual=residual, y=y, save=save, tail=tail, skew=skew, drop=drop, **kw)


def listed():
    return [
        # the load of a 128-expert layer while eight sequences each decode a token
        _balance(8, 128, 8, "forward", name="balance, 8 tokens"),
        # the losses of a prefill-sized training batch through the same router, and their gradient
        _balance(16384, 128, 8, "step", name="balance, 16384 tokens, step"),
        # the losses sequence by sequence over a ragged, padded batch of a 64-expert layer
        _balance(32749, 64, 8, "step", seqs=37, masked=True, name="balance, 37 sequences, step"),
        # the hidden states of one decode step
        _rows(8, 2048, "forward", name="rows, 8 x 2048"),
        # a ragged batch of hidden states that were kept in fp32
        _rows(8191, 4096, "forward", dtype="fp32", name="rows, 8191 x 4096 fp32"),
        # what a 64-expert layer's second product takes in a training microbatch, and the gradient
        _rows(32768, 1024, "step", gated=True, name="gated rows, 32768 x 1024, step"),
        # a dense projection of a decode step, with fp32 output
        _product(8, 1, 2048, 4096, y="fp32", bias=True, name="product, 8 rows"),
        # the first expert product of that decode step: 64 pairs on 40 of 128 experts
        _product(64, 128, 2048, 1536, touched=40, skew=1.0, name="product, 64 rows"),
        # a dense projection of a prefill chunk, added to the residual stream
        _product(2048, 1, 2048, 4096, act="gelu", residual=True, name="product, 2048 rows"),
        # the first product of a 64-expert layer's training microbatch: 4096 tokens gathered 8 times each
        _product(32768, 64, 2048, 2048, k=8, name="product, 4096 x 8 rows"),
        # an ungated expert product of that layer that keeps its pre-activation for the gradient
        _product(16381, 64, 1024, 2048, act="silu", touched=64, bias=True, save=True, tail=19, skew=0.5,
                 name="product, 16381 rows, kept"),
        # the first product of a wide 8-expert layer, 8192 tokens gathered twice each
        _product(16384, 8, 4096, 28672, k=2, name="product, 8192 x 2 rows"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("balance", "rows", "product"))
    way = rng.choice(("forward", "step"))
    if op == "balance":
        E, T = _log(rng, 4, 512), _log(rng, 1, 65536)
        return _balance(T, E, rng.randint(1, min(E, 16)), way, rng.choice((1, _log(rng, 1, 64))), rng.random() < 0.4)
    if op == "rows":
        return _rows(_log(rng, 1, 32768), 64 * _log(rng, 1, 64), way, rng.choice(("bf16", "fp32")), rng.random() < 0.5)
    inn, out = 64 * _log(rng, 1, 64), rng.choice((64 * _log(rng, 1, 64), rng.randint(17, 4097)))
    E = rng.choice((1, _log(rng, 2, 128)))
    rows = _log(rng, 1, 32768)
    common = dict(act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")), bias=rng.random() < 0.5,
                  residual=rng.random() < 0.3, y=rng.choice(("bf16", "bf16", "fp32")), save=rng.random() < 0.3,
                  skew=rng.choice((0.0, 1.0)))
    if E > 1 and rng.random() < 0.5:
        k = rng.randint(1, min(E, 8))
        return _product(-(-rows // k) * k, E, inn, out, k=k, drop=rng.choice((0.0, 0.0, 0.3)), **common)
    return _product(rows, E, inn, out, touched=rng.randint(1, min(E, rows)), tail=rng.choice((0, rng.randint(1, 40))),
                    **common)


# ---- inputs ----

def _expert_scores(E, skew, g):
    p = 1.0 / torch.arange(1, E + 1, device=DEV, dtype=torch.float32) ** skew
    return p[torch.randperm(E, generator=g, device=DEV)].log()


def _lengths(n, parts, g):
    """Uneven lengths of `parts` sequences that fill n tokens, as their first tokens and the end."""
    cuts = torch.randint(0, n + 1, (parts - 1,), generator=g, device=DEV).sort().values
    ends = torch.tensor([0, n], device=DEV)
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def _to_mx(v):
    """(codes [n, K/2], scales [n, K/32]) of rows v, the even element of a byte in its high half."""
    n, K = v.shape
    b = v.double().view(n, K // 32, 32)
    sh = _shared(b.abs().amax(2))
    y = torch.ldexp(b.abs(), -sh[..., None])
    code = _nearest(y) + 8 * torch.signbit(b)
    code = code.view(n, K // 2, 2).to(torch.uint8)
    return code[..., 0] * 16 + code[..., 1], (sh + 127).to(torch.uint8)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV).mul_(scale).to(dtype)

    s = dict(c)
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        # some experts are liked more than others
        s["logits"] = randn(T, E).mul_(1.5).add_(randn(E, scale=0.5))
        s["mask"] = None
        if c["masked"]:
            # padding tokens, and experts out of service for a token (for some tokens all of them)
            s["mask"] = torch.rand(T, generator=g, device=DEV) > 0.15
            off = torch.rand(T, E, generator=g, device=DEV) < 0.1
            off[torch.rand(T, generator=g, device=DEV) < 0.02] = True
            s["logits"].masked_fill_(off, -math.inf)
        s["idx"] = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
        s["cu"] = _lengths(T, c["seqs"], g) if c["seqs"] > 1 else None
        s["grad_loss"], s["grad_z"] = randn(c["seqs"]), randn(c["seqs"], scale=0.1)
        s["grad_route"] = randn(T, E, scale=0.01)
    elif c["op"] == "rows":
        n, K, dt = c["n"], c["K"], _T[c["dtype"]]
        # rows of hidden states differ in size, and a few channels stand out
        channel = torch.exp(randn(2 * K if c["gated"] else K, scale=0.7))
        s["x"] = (randn(n, channel.numel()) * channel * torch.exp(randn(n, 1))).to(dt)
        s["grad"] = randn(n, K, dtype=torch.bfloat16)
    else:
        E, inn, out, rows, k = c["E"], c["inn"], c["out"], c["rows"], c["k"]
        s["packed"] = torch.randint(0, 256, (E, out * inn // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["wscales"] = torch.randint(118, 123, (E, out * inn // 32), generator=g, device=DEV, dtype=torch.uint8)
        s["order"] = s["pos"] = None
        if k:
            # distinct experts a token; a dropped pair has id -1, as one whose expert lives on another rank has
            T = rows // k
            u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-7)
            ids = (_expert_scores(E, c["skew"], g) - torch.log(-torch.log(u))).topk(k, dim=1).indices
            ids = torch.where(torch.rand(ids.shape, generator=g, device=DEV) < c["drop"], torch.full_like(ids, E), ids)
            flat = ids.reshape(-1)
            order = torch.argsort(flat, stable=True)
            pos = torch.empty_like(order)
            pos[order] = torch.arange(rows, device=DEV)
            counts = torch.bincount(flat, minlength=E + 1)[:E]
            s["order"], s["pos"] = order.to(torch.int32), pos.to(torch.int32).view(T, k)
        else:
            # every touched expert has a row, the others follow the skew
            T = rows + c["tail"]
            p = _expert_scores(c["touched"] or 1, c["skew"], g).exp()
            more = torch.multinomial(p, max(rows - p.numel(), 1), replacement=True, generator=g)[:rows - p.numel()]
            counts = torch.zeros(E, dtype=torch.int64, device=DEV)
            counts[torch.randperm(E, generator=g, device=DEV)[:p.numel()]] = torch.bincount(more, minlength=p.numel()) + 1
        s["live"], s["cap"] = counts.nonzero()[:, 0], max(int(counts.max()), 1)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32) if E > 1 or c["tail"] else None
        s["codes"], s["scales"] = _to_mx(randn(T, inn) * torch.exp(randn(inn, scale=0.5)))
        R = rows + c["tail"]
        s["bias_v"] = randn(E, out, scale=0.1) if c["bias"] else None
        s["residual_v"] = randn(R, out, dtype=torch.bfloat16) if c["residual"] else None
    return s


# ---- the plain forms ----

def _plain_balance(s):
    lg, k = s["logits"], s["k"]
    T, E = lg.shape
    S, cu = s["seqs"], s["cu"]
    top = lg.amax(1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    z = torch.exp(lg - top)
    tot = z.sum(1, keepdim=True)
    used = tot[:, 0] > 0
    if s["mask"] is not None:
        used = used & s["mask"]
    p = torch.where(used[:, None], z / tot, torch.zeros_like(z))
    lse = torch.where(used, top[:, 0] + torch.log(tot[:, 0]), torch.full_like(tot[:, 0], -math.inf))
    lse0 = torch.where(used, lse, torch.zeros_like(lse))
    if cu is None:
        seg = torch.zeros(T, dtype=torch.int64, device=lg.device)
        per_seq = lambda v: v.double().sum(0, keepdim=True)  # noqa: E731
    else:
        seg = torch.searchsorted(cu[1:].contiguous(), torch.arange(T, device=lg.device, dtype=torch.int32), right=True)
        # long sums: differences of running ones, in 64 bits, along the side that is contiguous
        first = cu.to(torch.int64)
        running = lambda v: torch.nn.functional.pad(v.double().t().contiguous().cumsum(-1), (1, 0))  # noqa: E731
        per_seq = lambda v: running(v)[..., first].diff(dim=-1).t()  # noqa: E731
    picked = torch.zeros_like(lg).scatter_add_(1, s["idx"].to(torch.int64), used[:, None].expand(T, k).float())
    n, counts, prob = per_seq(used), per_seq(picked), per_seq(p)
    zero = torch.zeros(S, dtype=torch.float64, device=lg.device)
    inv = torch.where(n > 0, 1 / n.clamp(min=1), zero)
    f = counts * (inv * inv * (E / k))[:, None]
    out = {"counts": counts.to(torch.int32), "tokens": n.to(torch.int32), "prob": prob.float(),
           "loss": (f * prob).sum(1).float(), "z": (inv * per_seq(lse0.double().square())).float(),
           "lse": lse}
    if s["way"] == "step":
        ft = f.float()[seg]
        gl, gz = s["grad_loss"][seg][:, None], (s["grad_z"] * 2 * inv.float())[seg][:, None]
        grad = gl * p * (ft - (ft * p).sum(1, keepdim=True)) + gz * lse0[:, None] * p
        out["grad_logits"] = s["grad_route"] + grad
    return out


def _shared(amax):
    """The exponent that a block of 32 shares: that of its largest magnitude, less 2 (E2M1 reaches 1.5 * 2^2)."""
    _, e = torch.frexp(amax)
    return torch.where(amax > 0, e.to(torch.int32) - 3, torch.full_like(e, -127, dtype=torch.int32)).clamp(-127, 127)


def _nearest(y):
    """The place in _E2M1 nearest to y >= 0, ties to the even place, the last one for all beyond it."""
    mids = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), dtype=torch.float64, device=y.device)
    # bucketize counts the borders below y: one that y may lie on, to be counted too, is moved down a step
    mids[1::2] = torch.nextafter(mids[1::2], torch.zeros_like(mids[1::2]))
    return torch.bucketize(y, mids, out_int32=True)


def _plain_rows(s):
    x, K = s["x"], s["K"]
    v = x.double()
    if s["gated"]:
        # in 64 bits: where a value lies next to the middle of two codes, 32 may take the other one
        gate, up = v[:, :K], v[:, K:]
        v = gate / (1 + torch.exp(-gate)) * up
    b = v.view(x.shape[0], K // 32, 32)
    sh = _shared(b.abs().amax(2))[..., None]
    mag = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)[_nearest(torch.ldexp(b.abs(), -sh)).long()]
    out = {"values": torch.ldexp(torch.where(torch.signbit(b), -mag, mag), sh).view(-1, K).to(torch.bfloat16)}
    if s["gated"] and s["way"] == "step":
        gate, up, ga = x.float()[:, :K], x.float()[:, K:], s["grad"].float()
        sg = 1 / (1 + torch.exp(-gate))
        out["grad_x"] = torch.cat([ga * up * sg * (1 + gate * (1 - sg)), ga * gate * sg], 1).to(x.dtype)
    return out


def _decoded(codes, scales, n, K):
    """fp32 [..., n, K] of packed codes and their scales."""
    t = _E2M1 + tuple(-v for v in _E2M1)
    t = torch.tensor([[t[b >> 4], t[b & 15]] for b in range(256)], device=codes.device)
    v = t[codes.to(torch.int64)].view(-1, 32)
    return torch.ldexp(v, scales.reshape(-1, 1).to(torch.int32) - 127).view(-1, n, K)


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z * (z > 0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _plain_product(s):
    R, E, cap, off, inn, out = s["rows"] + s["tail"], s["E"], s["cap"], s["offsets"], s["inn"], s["out"]
    x = _decoded(s["codes"], s["scales"], s["codes"].shape[0], inn)[0]
    if s["order"] is not None:
        x = x[s["order"].to(torch.int64) // s["k"]]
    bias, dev = s["bias_v"], x.device
    if off is None:
        w = _decoded(s["packed"], s["wscales"], out, inn)
        spread, gather = (lambda v: v[None]), (lambda v: v[0])
    else:
        # the touched experts' weights, and their rows side by side, padded to the longest
        live, off = s["live"], off.to(torch.int64)
        w = _decoded(s["packed"][live], s["wscales"][live], out, inn)
        bias = None if bias is None else bias[live]
        lo, hi = off[live], off[live + 1]
        r = torch.arange(R, device=dev)
        e = torch.searchsorted(hi, r, right=True).clamp_(max=max(live.numel() - 1, 0))
        tail = (r >= off[-1])[:, None]
        at = (lo[:, None] + torch.arange(cap, device=dev)).clamp_(max=R - 1)
        spread = lambda v: v[at]  # noqa: E731
        gather = lambda v: torch.where(tail, torch.zeros((), device=dev), v[e, (r - lo[e]).clamp_(max=cap - 1)])  # noqa: E731
        if not live.numel():
            zero = torch.zeros(R, out, device=dev)
            return {"y": zero.to(_T[s["y"]])} | ({"pre": zero} if s["save"] else {})
    z = torch.bmm(spread(x), w.transpose(1, 2).contiguous())
    if bias is not None:
        z = z + bias[:, None, :]
    a = _act(s["act"], z)
    if s["residual_v"] is not None:
        a = a + spread(s["residual_v"].float())
    return {"y": gather(a).to(_T[s["y"]])} | ({"pre": gather(z)} if s["save"] else {})


# ---- the library's entry points ----

def _own_balance(s):
    import bit_quantized_mixture_nf4_amd as e4b
    f = e4b.moe_balance(s["logits"], s["idx"], cu_tokens=s["cu"], token_mask=s["mask"])
    out = {"counts": f.counts, "tokens": f.tokens, "prob": f.prob, "loss": f.loss, "z": f.z_loss, "lse": f.lse}
    if s["way"] == "step":
        out["grad_logits"] = e4b.moe_balance_backward(f, s["logits"], s["grad_loss"], s["grad_z"], cu_tokens=s["cu"],
                                                      add=s["grad_route"])
    return out


def _own_rows(s):
    import bit_quantized_mixture_nf4_amd as e4b
    out = {"values": e4b.mx4_values(e4b.mx4_rows(s["x"], gated=s["gated"]))}
    if s["gated"] and s["way"] == "step":
        out["grad_x"] = e4b.mx4_rows_backward(s["x"], s["grad"])
    return out


def _own_product(s):
    import bit_quantized_mixture_nf4_amd as e4b
    stack = e4b.QuantStack(s["packed"], None, s["E"], s["out"], s["inn"], "mxfp4", s["wscales"])
    perm = None if s["order"] is None else e4b.Permutation(s["offsets"], s["order"], s["pos"])
    y, pre = e4b.mx_linear(stack, e4b.MxRows(s["codes"], s["scales"]), offsets=None if perm else s["offsets"], perm=perm,
                           bias=s["bias_v"], act=s["act"], residual=s["residual_v"], out_dtype=_T[s["y"]], save=s["save"])
    return {"y": y} | ({"pre": pre} if s["save"] else {})


_PLAIN = {"balance": _plain_balance, "rows": _plain_rows, "product": _plain_product}
_OWN = {"balance": _own_balance, "rows": _own_rows, "product": _own_product}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ---- what a pass cannot do without ----

def work(case):
    c, step = case, case["way"] == "step" if "way" in case else False
    if c["op"] == "balance":
        TE = c["T"] * c["E"] * 4
        n = TE + c["T"] * (c["k"] * 4 + 4 + (1 if c["masked"] else 0)) + c["seqs"] * (c["E"] * 8 + 16)
        # backward: the gradient to add to in, the sum out; the logits are read once for both directions
        return {"bytes": n + (2 * TE if step else 0), "flops": c["T"] * c["E"] * (14 if step else 6)}
    if c["op"] == "rows":
        nK, b = c["n"] * c["K"], (2 if c["dtype"] == "bf16" else 4) * (2 if c["gated"] else 1)
        back = step and c["gated"]
        return {"bytes": nK * (b + 2) + (nK * (2 + b) if back else 0), "flops": nK * (30 if back else 15)}
    R = c["rows"] + c["tail"]
    touched = min(c["touched"] or c["E"], c["rows"])
    n = 17 / 32 * c["inn"] * ((c["rows"] // c["k"] if c["k"] else R) + touched * c["out"])
    n += R * c["out"] * ((2 if c["y"] == "bf16" else 4) + (4 if c["save"] else 0) + (2 if c["residual"] else 0))
    n += (touched * c["out"] * 4 if c["bias"] else 0) + (c["rows"] * 4 if c["k"] else 0)
    return {"bytes": n, "flops": 2 * c["rows"] * c["inn"] * c["out"]}


# ---- the definitions in 64 bits ----

def _exact_balance(s):
    """The losses sequence by sequence, and the gradient by differentiation."""
    f64 = torch.float64
    T, E, k, S = s["T"], s["E"], s["k"], s["seqs"]
    cu = [0, T] if s["cu"] is None else s["cu"].tolist()
    lg = s["logits"].to(f64)
    used = (lg > -math.inf).any(1) if s["mask"] is None else (lg > -math.inf).any(1) & s["mask"]
    leaf = lg.masked_fill(lg == -math.inf, -1e300).requires_grad_(True)
    out = {"counts": None, "tokens": None, "prob": torch.zeros(S, E, dtype=f64, device=DEV),
           "loss": torch.zeros(S, dtype=f64, device=DEV), "z": torch.zeros(S, dtype=f64, device=DEV),
           "lse": torch.full((T,), -math.inf, dtype=f64, device=DEV)}
    total = (leaf * 0).sum()
    with torch.enable_grad():
        for i in range(S):
            t = torch.arange(cu[i], cu[i + 1], device=DEV)
            t = t[used[t]]
            if not t.numel():
                continue
            share = torch.nn.functional.one_hot(s["idx"][t].long(), E).sum((0, 1)).to(f64) / (t.numel() * k)
            mean = torch.softmax(leaf[t], 1).mean(0)
            lse = torch.logsumexp(leaf[t], 1)
            loss, z = E * (share * mean).sum(), lse.square().mean()
            out["prob"][i], out["loss"][i], out["z"][i] = mean.detach() * t.numel(), loss.detach(), z.detach()
            out["lse"][t] = lse.detach()
            total = total + s["grad_loss"][i].to(f64) * loss + s["grad_z"][i].to(f64) * z
        if s["way"] == "step":
            out["grad_logits"] = torch.autograd.grad(total, leaf)[0] + s["grad_route"].to(f64)
    return out


def _exact_rows(s):
    K, f64 = s["K"], torch.float64
    x = s["x"].to(f64)
    with torch.enable_grad():
        leaf = x.clone().requires_grad_(True)
        v = torch.nn.functional.silu(leaf[:, :K]) * leaf[:, K:] if s["gated"] else leaf * 1.0
        out = {}
        if s["gated"] and s["way"] == "step":
            out["grad_x"] = torch.autograd.grad(v, leaf, s["grad"].to(f64))[0]
    b = v.detach().reshape(-1, 32)
    big = b.abs().amax(1, keepdim=True)
    shared = torch.where(big > 0, torch.floor(torch.log2(big)) - 2, torch.full_like(big, -127.0))
    # log2 in floating point may round across a whole number
    shared = torch.where(torch.exp2(shared + 2) > big, shared - 1, shared)
    shared = torch.where(torch.exp2(shared + 3) <= big, shared + 1, shared).clamp(-127, 127)
    y = b / torch.exp2(shared)
    # the step between codes: a half below 2, one below 4, two above
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0)).to(f64)
    out["values"] = ((torch.round(y / step) * step).clamp(-6, 6) * torch.exp2(shared)).view(-1, K)
    return out


def _exact_product(s):
    f64, R, E, inn, out = torch.float64, s["rows"] + s["tail"], s["E"], s["inn"], s["out"]
    if 2 * s["rows"] * inn * out > 1e14:
        return None

    def decoded(codes, scales, n):
        q = torch.stack([codes.long() // 16, codes.long() % 16], dim=-1).reshape(-1, 32)
        m = q % 8
        mag = torch.where(m < 2, m * 0.5, (2 + m % 2) * torch.exp2((m // 2 - 2).to(f64)))
        return (mag * (1 - 2 * (q // 8)) * torch.exp2(scales.reshape(-1, 1).to(f64) - 127)).view(n, inn)

    x = decoded(s["codes"], s["scales"], s["codes"].shape[0])
    off = [0, R] if s["offsets"] is None else s["offsets"].tolist()
    y = torch.zeros(R, out, dtype=f64, device=DEV)
    pre = torch.zeros(R, out, dtype=f64, device=DEV)
    f = torch.nn.functional
    acts = {"none": lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
            "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        at = slice(a, b) if s["order"] is None else s["order"][a:b].long() // s["k"]
        z = x[at] @ decoded(s["packed"][e], s["wscales"][e], out).T
        if s["bias_v"] is not None:
            z = z + s["bias_v"][e].to(f64)
        pre[a:b], y[a:b] = z, acts[s["act"]](z)
        if s["residual_v"] is not None:
            y[a:b] += s["residual_v"][a:b].to(f64)
    return {"y": y} | ({"pre": pre} if s["save"] else {})


def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "rows": _exact_rows, "product": _exact_product}[s["op"]](s)
