"""Float64 definitions of the operators around the expert MLP (numpy).

Routing gradients, the expert order of routed pairs and the way back, products of
expert-sorted rows with a stack and an epilogue, and the norms before and after a
block, each with its gradient.
"""

import math

import numpy as np

f64 = np.float64


def route_backward(idx, w, grad_w, E):
    """d(sum(grad_w * w)) / d logits with w = softmax(logits[idx]), the selection fixed."""
    idx, w, g = np.asarray(idx), np.asarray(w, f64), np.asarray(grad_w, f64)
    out = np.zeros((idx.shape[0], E))
    d = w * (g - (w * g).sum(axis=1, keepdims=True))
    for t in range(idx.shape[0]):
        for j in range(idx.shape[1]):
            if 0 <= idx[t, j] < E:
                out[t, idx[t, j]] += d[t, j]
    return out


def balance(logits, idx, cu=None, mask=None):
    """How evenly a router uses its experts, sequence by sequence: dict of counts [S, E],
    tokens [S], prob [S, E], loss [S], z [S] and lse [T] (-inf for a token not counted)."""
    lg, idx = np.asarray(logits, f64), np.asarray(idx)
    T, E = lg.shape
    k = idx.shape[1]
    cu = [0, T] if cu is None else [min(max(int(c), 0), T) for c in cu]
    S = len(cu) - 1
    counts, tokens, prob = np.zeros((S, E), np.int64), np.zeros(S, np.int64), np.zeros((S, E))
    zsum, lse, loss = np.zeros(S), np.full(T, -np.inf), np.zeros(S)
    for s in range(S):
        for t in range(cu[s], cu[s + 1]):
            if (mask is not None and not mask[t]) or np.all(lg[t] == -np.inf):
                continue
            top = lg[t].max()
            z = np.exp(lg[t] - top)
            lse[t] = top + np.log(z.sum())
            prob[s] += z / z.sum()
            zsum[s] += lse[t] ** 2
            tokens[s] += 1
            for e in idx[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if tokens[s]:
            loss[s] = E / (k * float(tokens[s]) ** 2) * (counts[s] * prob[s]).sum()
            zsum[s] /= tokens[s]
    return {"counts": counts, "tokens": tokens, "prob": prob, "loss": loss, "z": zsum, "lse": lse}


def balance_backward(fwd, logits, k, grad_loss=None, grad_z=None, cu=None, add=None):
    """d(sum(grad_loss loss) + sum(grad_z z)) / d logits, the counts fixed, plus add."""
    lg = np.asarray(logits, f64)
    T, E = lg.shape
    cu = [0, T] if cu is None else [min(max(int(c), 0), T) for c in cu]
    out = np.zeros((T, E)) if add is None else np.asarray(add, f64).copy()
    for s in range(len(cu) - 1):
        for t in range(cu[s], cu[s + 1]):
            if fwd["lse"][t] == -np.inf:
                continue
            N, c = float(fwd["tokens"][s]), np.asarray(fwd["counts"][s], f64)
            z = np.exp(lg[t] - lg[t].max())
            p = z / z.sum()
            if grad_loss is not None:
                out[t] += float(grad_loss[s]) * E / (k * N * N) * p * (c - (c * p).sum())
            if grad_z is not None:
                out[t] += float(grad_z[s]) * 2.0 / N * fwd["lse"][t] * p
    return out


def swiglu(x):
    """silu(g) u of rows [g | u], and its derivatives by g and by u."""
    x = np.asarray(x, f64)
    g, u = np.split(x, 2, axis=1)
    e = np.exp(-np.abs(g))
    s, r = np.where(g < 0, e, 1.0) / (1.0 + e), np.where(g < 0, 1.0, e) / (1.0 + e)  # sigmoid, 1 - sigmoid
    return g * s * u, s * (1.0 + g * r) * u, g * s


def expert_order(idx, E):
    """(offsets [E + 1], sorted_pair [P], pos [T, k]): pairs by expert id, stable; pairs
    whose id lies outside [0, E) last."""
    idx = np.asarray(idx)
    flat = idx.reshape(-1).astype(np.int64)
    buckets = [[] for _ in range(E + 1)]
    for p, e in enumerate(flat):
        buckets[e if 0 <= e < E else E].append(p)
    order = np.array([p for b in buckets for p in b], dtype=np.int32)
    offsets = np.cumsum([0] + [len(b) for b in buckets[:E]]).astype(np.int32)
    pos = np.empty(flat.size, dtype=np.int32)
    pos[order] = np.arange(flat.size, dtype=np.int32)
    return offsets, order, pos.reshape(idx.shape)


def permute(x, idx, E):
    """rows [T k, H]: each pair's token row at its place, zeros for pairs without an expert."""
    offsets, order, _ = expert_order(idx, E)
    rows = np.asarray(x, f64)[order // idx.shape[1]].copy()
    rows[offsets[-1]:] = 0.0
    return rows


def unpermute(rows, offsets, pos, w=None):
    """y[t] = sum_j w[t, j] rows[pos(t, j)] over the pairs that have an expert."""
    T, k = pos.shape
    y = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < offsets[-1]:
                y[t] += (1.0 if w is None else f64(w[t, j])) * np.asarray(rows[pos[t, j]], f64)
    return y


def unpermute_backward(rows, offsets, pos, w, grad_y):
    """(grad_rows, grad_w) of unpermute."""
    T, k = pos.shape
    gy, gr, gw = np.asarray(grad_y, f64), np.zeros((T * k, grad_y.shape[1])), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if 0 <= pos[t, j] < offsets[-1]:
                gr[pos[t, j]] = (1.0 if w is None else f64(w[t, j])) * gy[t]
                gw[t, j] = np.asarray(rows[pos[t, j]], f64) @ gy[t]
    return gr, gw


_erf = np.vectorize(math.erf, otypes=[f64])


def activation(act, z):
    """(act(z), act'(z))"""
    z = np.asarray(z, f64)
    if act == "none":
        return z.copy(), np.ones_like(z)
    if act == "relu":
        return np.maximum(z, 0.0), np.where(np.isnan(z), z, z > 0)
    if act == "silu":
        s = 0.5 * (1.0 + np.tanh(0.5 * z))
        return z * s, s + z * s * (1.0 - s)
    if act == "gelu":
        cdf = 0.5 * (1.0 + _erf(z / math.sqrt(2.0)))
        return z * cdf, cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 0.134145 * z * z)
    raise ValueError(act)


def expert_linear(x, w, offsets=None, bias=None, act="none", residual=None):
    """(y, z) of expert-sorted rows x [R, in] against w [E, out, in]; zeros behind the last expert."""
    R, (E, out, _) = x.shape[0], w.shape
    offsets = [0, R] if offsets is None else offsets
    y, z = np.zeros((R, out)), np.zeros((R, out))
    for e in range(E):
        sl = slice(offsets[e], offsets[e + 1])
        if sl.start == sl.stop:
            continue
        z[sl] = np.asarray(x[sl], f64) @ np.asarray(w[e], f64).T + (0.0 if bias is None else np.asarray(bias[e], f64))
        y[sl] = activation(act, z[sl])[0] + (0.0 if residual is None else np.asarray(residual[sl], f64))
    return y, z


def expert_linear_dgrad(grad_y, z, w, offsets=None, act="none"):
    """(grad_x, grad_bias) with z from expert_linear."""
    R, (E, out, inn) = grad_y.shape[0], w.shape
    offsets = [0, R] if offsets is None else offsets
    gx, gb = np.zeros((R, inn)), np.zeros((E, out))
    for e in range(E):
        sl = slice(offsets[e], offsets[e + 1])
        if sl.start == sl.stop:
            continue
        dz = np.asarray(grad_y[sl], f64) * activation(act, z[sl])[1]
        gx[sl] = dz @ np.asarray(w[e], f64)
        gb[e] = dz.sum(axis=0)
    return gx, gb


def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _gate(gate_token, gate_channel):
    if gate_token is not None:
        return np.asarray(gate_token, f64)[:, None]
    return 1.0 if gate_channel is None else np.asarray(gate_channel, f64)


def block_norm(x, y=None, w_post=None, gate_token=None, gate_channel=None, scale=1.0, w_pre=None, eps=1e-6):
    """(r, h or None)"""
    r = np.asarray(x, f64)
    if y is not None:
        u = np.asarray(y, f64)
        if w_post is not None:
            u = u * _rstd(u, eps) * np.asarray(w_post, f64)
        r = r + scale * _gate(gate_token, gate_channel) * u
    h = None if w_pre is None else r * _rstd(r, eps) * np.asarray(w_pre, f64)
    return r, h


def _norm_backward(g, v, rstd):
    """Gradient of n = v rstd(v) from g = d / d n."""
    n = v * rstd
    return rstd * (g - n * (g * n).mean(axis=1, keepdims=True))


def block_norm_backward(x, grad_r=None, grad_h=None, y=None, w_post=None, gate_token=None, gate_channel=None, scale=1.0,
                        w_pre=None, eps=1e-6):
    """dict of the gradients of sum(grad_r r) + sum(grad_h h)."""
    out = {}
    r, _ = block_norm(x, y, w_post, gate_token, gate_channel, scale, None, eps)
    dr = np.zeros_like(r) if grad_r is None else np.asarray(grad_r, f64).copy()
    if w_pre is not None:
        gh, rs = np.asarray(grad_h, f64), _rstd(r, eps)
        out["grad_w_pre"] = (gh * r * rs).sum(axis=0)
        dr += _norm_backward(gh * np.asarray(w_pre, f64), r, rs)
    out["grad_x"] = dr
    if y is None:
        return out
    yy = np.asarray(y, f64)
    rs = _rstd(yy, eps)
    u = yy if w_post is None else yy * rs * np.asarray(w_post, f64)
    if gate_token is not None:
        out["grad_gate"] = scale * (dr * u).sum(axis=1)
    if gate_channel is not None:
        out["grad_gate"] = scale * (dr * u).sum(axis=0)
    du = scale * _gate(gate_token, gate_channel) * dr
    if w_post is not None:
        out["grad_w_post"] = (du * yy * rs).sum(axis=0)
        du = _norm_backward(du * np.asarray(w_post, f64), yy, rs)
    out["grad_y"] = du
    return out
