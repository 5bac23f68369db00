"""Pins of the float64 definitions of the router's balance, of gated rows and of microscaled rows:
hand-built cases, central differences and the stacks' conversion."""

import numpy as np
import pytest

import oracle
from oracle import block, mx


def test_an_even_router_has_a_loss_of_one():
    T, E, k = 12, 6, 2
    idx = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    f = block.balance(np.zeros((T, E)), idx)
    assert np.array_equal(f["counts"], [[4] * E]) and f["tokens"][0] == T
    assert np.allclose(f["prob"], T / E) and np.isclose(f["loss"][0], 1.0)
    assert np.allclose(f["lse"], np.log(E)) and np.isclose(f["z"][0], np.log(E) ** 2)


def test_a_router_of_one_expert_has_a_loss_of_its_number():
    lg = np.full((5, 4), -np.inf)
    lg[:, 2] = 3.0
    f = block.balance(lg, np.full((5, 1), 2))
    assert np.isclose(f["loss"][0], 4.0) and np.isclose(f["z"][0], 9.0)


def test_what_is_not_counted():
    rng = np.random.default_rng(0)
    lg = rng.standard_normal((9, 5))
    lg[3] = -np.inf
    lg[7] = np.nan  # masked: whatever it holds
    idx = rng.integers(0, 5, (9, 2))
    idx[1, 0], idx[2, 1] = -1, 5
    mask = np.ones(9, bool)
    mask[7] = False
    f = block.balance(lg, idx, cu=[1, 4, 4, 8], mask=mask)
    assert list(f["tokens"]) == [2, 0, 3] and list(f["counts"].sum(axis=1)) == [2, 0, 6]
    assert f["loss"][1] == 0 and f["z"][1] == 0
    assert [t for t in range(9) if f["lse"][t] == -np.inf] == [0, 3, 7, 8]
    g = block.balance_backward(f, lg, 2, [1.0] * 3, [1.0] * 3, cu=[1, 4, 4, 8])
    assert not g[[0, 3, 7, 8]].any() and np.isfinite(g).all()


def test_balance_gradient_by_differences():
    rng = np.random.default_rng(1)
    T, E, k, cu = 7, 6, 2, [0, 3, 7]
    lg = rng.standard_normal((T, E))
    lg[2, 4] = -np.inf
    idx = np.argsort(-lg, axis=1)[:, :k]
    gl, gz = rng.standard_normal(2), rng.standard_normal(2)
    f = block.balance(lg, idx, cu)
    add = rng.standard_normal((T, E))
    g = block.balance_backward(f, lg, k, gl, gz, cu, add) - add
    loss = lambda v: (gl * (h := block.balance(v, idx, cu))["loss"]).sum() + (gz * h["z"]).sum()  # noqa: E731
    for t in range(T):
        for e in range(E):
            if lg[t, e] == -np.inf:
                assert g[t, e] == 0
                continue
            d = np.zeros_like(lg)
            d[t, e] = 1e-5
            assert abs((loss(lg + d) - loss(lg - d)) / 2e-5 - g[t, e]) < 1e-8


def test_counts_of_two_ranks_give_the_gradient_of_their_joint_loss():
    rng = np.random.default_rng(2)
    lg, k = rng.standard_normal((10, 4)), 2
    idx = np.argsort(-lg, axis=1)[:, :k]
    whole = block.balance(lg, idx)
    want = block.balance_backward(whole, lg, k, [1.0], [0.3])
    parts = [block.balance(lg[s], idx[s]) for s in (slice(0, 4), slice(4, 10))]
    for p, s in zip(parts, (slice(0, 4), slice(4, 10))):
        joint = {**p, "counts": parts[0]["counts"] + parts[1]["counts"], "tokens": parts[0]["tokens"] + parts[1]["tokens"]}
        assert np.allclose(block.balance_backward(joint, lg[s], k, [1.0], [0.3]), want[s])


def test_swiglu_by_differences_and_far_out():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 8)) * 3
    v, dg, du = block.swiglu(x)
    for j in range(8):
        d = np.zeros(8)
        d[j] = 1e-6
        num = (block.swiglu(x + d)[0] - block.swiglu(x - d)[0]) / 2e-6
        assert np.allclose(num[:, j % 4], (dg if j < 4 else du)[:, j % 4], atol=1e-8)
    v, dg, _ = block.swiglu([[-100.0, 200.0, 1e30, 2.0]])
    assert np.isclose(v[0, 0], -100 * np.exp(-100) * 1e30, rtol=1e-12) and v[0, 1] == 400
    assert np.isclose(dg[0, 0], -99 * np.exp(-100) * 1e30, rtol=1e-12)


def test_rows_are_a_stack_of_one_expert():
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((7, 192)) * np.exp(rng.uniform(-60, 60, (7, 1)))).astype(np.float32)
    x[3, 64:96] = 0
    p, s = oracle.quantize_mx(x[None])
    codes, scales = mx.quantize_mx_rows(x)
    assert np.array_equal(codes, p.reshape(7, 96)) and np.array_equal(scales, s.reshape(7, 6))
    assert np.array_equal(mx.mx_rows_values(codes, scales), oracle.dequantize_mx(p, s, 7, 192)[0])


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_a_block_with_no_value_is_nan(bad):
    x = np.ones((2, 64))
    x[1, 40] = bad
    codes, scales = mx.quantize_mx_rows(x)
    assert scales.tolist() == [[125, 125], [125, 255]] and not codes[1, 16:].any()
    v = mx.mx_rows_values(codes, scales)
    assert np.isnan(v[1, 32:]).all() and np.array_equal(v[0], x[0]) and np.array_equal(v[1, :32], x[1, :32])
