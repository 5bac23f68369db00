"""Pins of the float64 definitions around the expert MLP: hand-built cases, central
differences, and agreement with the oracle's routed forward."""

import numpy as np
import pytest

import oracle
from oracle import block


def _diff(f, v, step=1e-6):
    """Central differences of the scalar f over every element of v."""
    g = np.zeros_like(v)
    it = np.nditer(v, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = v[i]
        v[i] = old + step
        hi = f()
        v[i] = old - step
        lo = f()
        v[i] = old
        g[i] = (hi - lo) / (2 * step)
    return g


def test_expert_order_by_hand():
    idx = np.array([[2, 0], [-1, 2], [0, 7], [1, 1]], dtype=np.int32)
    offsets, order, pos = block.expert_order(idx, 3)
    assert offsets.tolist() == [0, 2, 4, 6]
    assert order.tolist() == [1, 4, 6, 7, 0, 3, 2, 5]
    assert pos.tolist() == [[4, 0], [6, 5], [1, 7], [2, 3]]
    rows = block.permute(np.arange(8.0).reshape(4, 2), idx, 3)
    assert rows[:, 0].tolist() == [0, 4, 6, 6, 0, 2, 0, 0] and not rows[6:].any()


def test_route_backward_by_differences():
    rng = np.random.default_rng(0)
    lg, gw = rng.standard_normal((5, 7)), rng.standard_normal((5, 3))
    idx, w = oracle.route(lg, 3)
    def f():
        sel = np.take_along_axis(lg, idx.astype(np.int64), axis=1)
        e = np.exp(sel - sel.max(axis=1, keepdims=True))
        return ((e / e.sum(axis=1, keepdims=True)) * gw).sum()
    np.testing.assert_allclose(block.route_backward(idx, w, gw, 7), _diff(f, lg), atol=1e-8)


def test_unpermute_gradients_by_differences():
    rng = np.random.default_rng(1)
    idx = np.array([[1, 3, -1], [0, 1, 1], [2, 5, 0]])
    offsets, _, pos = block.expert_order(idx, 4)
    rows, w, gy = rng.standard_normal((9, 4)), rng.random((3, 3)), rng.standard_normal((3, 4))
    f = lambda: (block.unpermute(rows, offsets, pos, w) * gy).sum()  # noqa: E731
    gr, gw = block.unpermute_backward(rows, offsets, pos, w, gy)
    np.testing.assert_allclose(gr, _diff(f, rows), atol=1e-8)
    np.testing.assert_allclose(gw, _diff(f, w), atol=1e-8)
    # the plain sum is the gradient of the copies
    x = rng.standard_normal((3, 4))
    g = lambda: (block.permute(x, idx, 4) * rows).sum()  # noqa: E731
    np.testing.assert_allclose(block.unpermute(rows, offsets, pos), _diff(g, x), atol=1e-8)


def test_pieces_make_the_routed_forward():
    """Order, two products and the way back equal the oracle's ungated routed expert MLP."""
    rng = np.random.default_rng(2)
    T, E, k, H, I = 9, 4, 2, 6, 5
    x, lg = rng.standard_normal((T, H)), rng.standard_normal((T, E))
    up, dn = rng.standard_normal((E, I, H)), rng.standard_normal((E, H, I))
    idx, w = oracle.route(lg, k)
    offsets, _, pos = block.expert_order(idx, E)
    a, _ = block.expert_linear(block.permute(x, idx, E), up, offsets, act="silu")
    o, _ = block.expert_linear(a, dn, offsets)
    np.testing.assert_allclose(block.unpermute(o, offsets, pos, w), oracle.moe_forward(x, idx, w, up, dn), atol=1e-12)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_expert_linear_gradients_by_differences(act):
    rng = np.random.default_rng(3)
    x, w, b = rng.standard_normal((7, 4)), rng.standard_normal((3, 5, 4)), rng.standard_normal((3, 5))
    res, gy = rng.standard_normal((7, 5)), rng.standard_normal((7, 5))
    offsets = [0, 2, 2, 6]  # an expert without rows, a row without an expert
    y, z = block.expert_linear(x, w, offsets, b, act, res)
    assert not y[6].any()
    f = lambda: (block.expert_linear(x, w, offsets, b, act, res)[0] * gy).sum()  # noqa: E731
    gx, gb = block.expert_linear_dgrad(gy, z, w, offsets, act)
    np.testing.assert_allclose(gx, _diff(f, x), atol=1e-7)
    np.testing.assert_allclose(gb, _diff(f, b), atol=1e-7)


@pytest.mark.parametrize("has_y,post,gate,pre", [(False, False, None, True), (True, False, None, False),
                                                 (True, True, "token", True), (True, True, "channel", True),
                                                 (True, False, "channel", False), (True, False, "token", True)])
def test_block_norm_gradients_by_differences(has_y, post, gate, pre):
    rng = np.random.default_rng(4)
    T, H = 3, 6
    leaf = {"x": rng.standard_normal((T, H))}
    if has_y:
        leaf["y"] = rng.standard_normal((T, H))
    if post:
        leaf["w_post"] = rng.standard_normal(H)
    if gate:
        leaf["gate_" + gate] = rng.standard_normal(T if gate == "token" else H)
    if pre:
        leaf["w_pre"] = rng.standard_normal(H)
    gr, gh = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def f():
        r, h = block.block_norm(scale=0.7, **leaf)
        return (gr * r).sum() + (0.0 if h is None else (gh * h).sum())

    g = block.block_norm_backward(leaf["x"], gr, gh, scale=0.7, **{n: v for n, v in leaf.items() if n != "x"})
    for name, v in leaf.items():
        want = _diff(f, v)
        got = g["grad_gate" if name.startswith("gate") else "grad_" + name]
        np.testing.assert_allclose(got, want, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_nan_passes_every_activation(act):
    a, d = block.activation(act, np.array([np.nan, -1.0, 2.0]))
    assert np.isnan(a[0]) and (act == "none" or np.isnan(d[0])) and np.isfinite(a[1:]).all() and np.isfinite(d[1:]).all()
