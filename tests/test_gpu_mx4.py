"""GPU parity of the microscaled 4-bit rows, their gradient and their product against the oracle.

Codes and scales are exact. The product's operands are exact and its sums fp32: an addition that
rounds is off by U = 2^-24 of its result, one that cuts off by 2 U, so a sum of n terms in any order by
2 n U of the terms' magnitudes; then half a step of the output's type (bf16 2^-8, fp32 U).
"""

import numpy as np
import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
from oracle import block, mx
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def within(got, ref, err, name):
    g = got.detach().cpu().double().numpy()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    bound = (err + HALF[got.dtype] * np.abs(ref)) * (1 + 2.0 ** -6) + 1e-37
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{g[bad][0]} against {ref[bad][0]}, bound {bound[bad][0]:.3e}")


def host(t):
    return t.detach().cpu().double().numpy()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(dtype)


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def same_rows(q, v, name):
    """The codes and scales of float64 values v, byte for byte."""
    codes, scales = mx.quantize_mx_rows(v)
    got_c, got_s = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    bad = np.argwhere(got_s != scales)
    assert not bad.size, f"{name}: scales differ at {bad[0]}: {got_s[tuple(bad[0])]} against {scales[tuple(bad[0])]}"
    bad = np.argwhere(got_c != codes)
    assert not bad.size, f"{name}: codes differ at {bad[0]}: {got_c[tuple(bad[0])]:#x} against {codes[tuple(bad[0])]:#x}"


# ---- rows ----

SIZES = [(1, 64), (3, 128), (5, 192), (64, 2048), (17, 4096), (1001, 320), (2, 14336), (7, 64), (300, 1088), (0, 64)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("n,K", SIZES)
def test_rows_byte_for_byte(n, K, dt):
    announce(f"mx4 rows {n} x {K} {dt}")
    rng = np.random.default_rng(n + K)
    x = rng.standard_normal((n, K)) * np.exp(rng.uniform(-80, 80, (n, 1)))
    x[rng.random((n, K)) < 0.05] = 0.0
    x_d = dev(x, DT[dt])
    q = e4b.mx4_rows(x_d)
    assert q.codes.shape == (n, K // 2) and q.scales.shape == (n, K // 32) and q.rows == n and q.K == K
    same_rows(q, host(x_d), "rows")
    for out in (torch.bfloat16, torch.float32):
        v = e4b.mx4_values(q, out)
        assert v.dtype == out and np.array_equal(host(v), mx.mx_rows_values(q.codes.cpu().numpy(), q.scales.cpu().numpy()))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_every_scale_border_and_tie(dt):
    """Each exponent that a block can share, with every border of two codes, its neighbours, zeros of
    both signs, and subnormal inputs."""
    announce(f"mx4 rows at borders {dt}")
    grid = np.concatenate([np.arange(0, 32) / 4.0, [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.125, 7.96875]])
    step = 2.0 ** -7 if dt == "bf16" else 2.0 ** -23
    grid = np.concatenate([grid, grid * (1 + step), grid * (1 - step)])
    rows = []
    for e in range(-149, 126):
        for top in (4.0, 7.5):  # what fixes the shared exponent
            v = np.resize(grid, 31 * -(-grid.size // 31)).reshape(-1, 31) * 2.0 ** e
            rows.append(np.concatenate([np.full((v.shape[0], 1), top * 2.0 ** e), v], axis=1).reshape(-1))
    rows = np.stack(rows)
    rows = np.pad(rows, ((0, 0), (0, -rows.shape[1] % 64)))
    rows[1::2] *= -1.0
    with np.errstate(over="ignore"):
        x = dev(rows, DT[dt])  # (the last rows reach infinity in bf16: such blocks are NaN)
    same_rows(e4b.mx4_rows(x), host(x), "borders")


def test_rows_equal_the_stacks_conversion():
    x = torch.randn(40, 256, device=DEV) * torch.exp(4 * torch.randn(40, 1, device=DEV))
    s = e4b.quantize(x[None], "mxfp4")
    q = e4b.mx4_rows(x)
    assert torch.equal(q.codes, s.packed.view(40, 128)) and torch.equal(q.scales, s.scales.view(40, 8))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("is_gated", [False, True])
def test_blocks_without_a_value(dt, is_gated):
    """A block that holds an infinity or a NaN reads as NaN, and its neighbours as they are; the product's
    row, too, is NaN throughout and alone."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 256)).astype(np.float32)
    x[1, 40], x[2, 0], x[3, 127], x[4, 64:96] = np.inf, np.nan, -np.inf, np.nan
    if is_gated:
        x[:, 128:] = np.abs(x[:, 128:]) + 0.5
        x[3, 127] = 1e30  # g u beyond fp32
        x[3, 255] = 1e30
    x_d = dev(x, DT[dt])
    q = e4b.mx4_rows(x_d, gated=is_gated)
    with np.errstate(invalid="ignore", over="ignore"):
        v = block.swiglu(host(x_d))[0] if is_gated else host(x_d)
        v = np.where(np.abs(v) > 3.5e38, np.inf, v)
    same_rows(q, v, "rows")
    assert (q.scales == 255).sum().item() == 4
    values = e4b.mx4_values(q)
    assert values.isnan().any(dim=1).tolist() == [False, True, True, True, True, False]
    stack = e4b.quantize(torch.randn(1, 48, q.K, device=DEV), "mxfp4")
    y, _ = e4b.mx_linear(stack, q)
    assert y.isnan().all(dim=1).tolist() == [False, True, True, True, True, False]
    assert not y[[0, 5]].isnan().any()


# ---- gated rows ----


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("n,K", SIZES)
def test_gated_rows_and_their_gradient(n, K, dt):
    """The codes are those of the exact silu(g) u (in 64 bits: its own error reaches a border between two
    codes once in 2^40 values). The gradient's factors are each off by a few steps, the exponential's
    argument by what its second term leaves, below 4 U in all; every product by a step."""
    announce(f"gated rows {n} x {K} {dt}")
    rng = np.random.default_rng(n + K + 1)
    x = rng.standard_normal((n, 2 * K)) * np.exp(rng.uniform(-3, 3, (n, 1)))
    x[rng.random((n, 2 * K)) < 0.02] = 0.0
    x[:, K:] *= np.exp(rng.uniform(-30, 30, (n, 1)))
    x_d = dev(x, DT[dt])
    xh = host(x_d)
    v, dg, du = block.swiglu(xh)
    same_rows(e4b.mx4_rows(x_d, gated=True), v, "gated")
    g, u = xh[:, :K], xh[:, K:]
    e = np.exp(-np.abs(g))
    s, r = np.where(g < 0, e, 1.0) / (1 + e), np.where(g < 0, 1.0, e) / (1 + e)
    for gdt in ("bf16", "fp32"):
        grad = dev(rng.standard_normal((n, K)), DT[gdt])
        ga = host(grad)
        want = np.concatenate([ga * dg, ga * du], axis=1)
        # dg's sum 1 + g (1 - s) may cancel: relative to its terms
        err = np.concatenate([np.abs(ga * u) * s * (1 + np.abs(g) * r), np.abs(ga * du)], axis=1) * 24 * U
        within(e4b.mx4_rows_backward(x_d, grad), want, err, "grad_x")


def test_gated_rows_far_out():
    """Gates at which the exponential leaves fp32's range, factors that bring the product back into it,
    subnormals and zeros."""
    announce("gated rows far out")
    g = np.array([-1e30, -700, -120, -104, -103, -95, -88.5, -87, -80, -65, -64, -63, -20, -1e-30, -1e-42, -0.0, 0.0, 1e-44, 1e-38,
                  1e-3, 17, 64, 65, 88, 104, 1e10, 1e20, -1.2784645, 1.5e-19, -2e-39, 40, -40], np.float32)
    u = np.array([1.0, 1e30, 3e38, -1e-30, 1e-44, 0.0, 2e19, -7.0], np.float32)
    x = np.array([np.concatenate([np.roll(g, k), np.full(32, b), g * 0 + a, g * 0 + a])
                  for a in u for b in (1.0, -3.0) for k in (0, 5)], np.float32)
    x_d = dev(x, torch.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        v, dg, du = block.swiglu(x)
        v = np.where(np.abs(v) > np.finfo(np.float32).max, np.inf, v)
    same_rows(e4b.mx4_rows(x_d, gated=True), v, "gated")
    # a block a value: every far value alone fixes its scale
    wide = np.zeros((g.size * u.size, 128), np.float32)
    wide[:, 0], wide[:, 64] = np.repeat(g, u.size), np.tile(u, g.size)
    with np.errstate(over="ignore"):
        v, dg, du = block.swiglu(wide)
        v = np.where(np.abs(v) > np.finfo(np.float32).max, np.inf, v)
    same_rows(e4b.mx4_rows(dev(wide, torch.float32), gated=True), v, "alone")
    grad = np.zeros((wide.shape[0], 64), np.float32)
    grad[:, 0] = 0.75
    want = np.concatenate([grad * dg, grad * du], axis=1)
    got = host(e4b.mx4_rows_backward(dev(wide, torch.float32), dev(grad, torch.float32)))
    # dg's terms are s and s |g| (1 - s): for g < 0 s <= e^-|g| and 1 - s <= 1, else s <= 1 and
    # 1 - s <= e^-|g|; beyond fp32's normal range on either side only the limit counts
    gg, uu, ga = np.abs(wide[:, :64]).astype(np.float64), np.abs(wide[:, 64:]).astype(np.float64), grad.astype(np.float64)
    e = np.exp(-gg)
    terms = np.concatenate([ga * uu * np.where(wide[:, :64] < 0, e * (1 + gg), 1 + gg * e), np.abs(want[:, 64:])], axis=1)
    fin = np.abs(want) < 3.3e38
    bad = fin & ~(np.abs(got - want) <= 24 * U * np.minimum(terms, 1e39) + 2.0 ** -120)
    assert not bad.any(), (np.argwhere(bad)[0], got[bad][0], want[bad][0])
    assert np.isinf(got[np.abs(want) > 3.5e38]).all()


def test_gated_gradient_by_differences():
    x = torch.randn(4, 128, device=DEV, dtype=torch.float64)
    ga = torch.randn(4, 64, device=DEV)
    got = host(e4b.mx4_rows_backward(x.float(), ga))
    xh, gh = host(x.float()), host(ga)
    for i, j in ((0, 0), (1, 63), (2, 64), (3, 127), (0, 31)):
        d = np.zeros_like(xh)
        d[i, j] = 1e-6
        num = (gh * (block.swiglu(xh + d)[0] - block.swiglu(xh - d)[0])).sum() / 2e-6
        assert abs(num - got[i, j]) <= 1e-6 * (1 + abs(num))


# ---- the product ----


@pytest.mark.parametrize("is_gated", [False, True])
def test_rows_beyond_32_bits(is_gated):
    """More than 2^32 values: the last rows have the bits that they have alone."""
    announce(f"mx rows beyond 32 bits gated={is_gated}")
    n, K = 4200007, 1088
    x = torch.empty(n, K * (1 + is_gated), device=DEV, dtype=torch.bfloat16).normal_()
    q = e4b.mx4_rows(x, gated=is_gated)
    alone = e4b.mx4_rows(x[-24:].clone(), gated=is_gated)
    assert torch.equal(q.codes[-24:], alone.codes) and torch.equal(q.scales[-24:], alone.scales)
    v = e4b.mx4_values(q)
    assert torch.equal(bits(v[-24:]), bits(e4b.mx4_values(alone)))
    if is_gated:
        g = e4b.mx4_rows_backward(x, v)
        assert torch.equal(bits(g[-24:]), bits(e4b.mx4_rows_backward(x[-24:].clone(), v[-24:].clone())))


def _stack(E, out, inn, seed, lo=118, hi=123):
    rng = np.random.default_rng(seed)
    packed = rng.integers(0, 256, (E, out * inn // 2), dtype=np.uint8)
    scales = rng.integers(lo, hi, (E, out * inn // 32), dtype=np.uint8)
    st = e4b.QuantStack(torch.from_numpy(packed).to(DEV), None, E, out, inn, "mxfp4", torch.from_numpy(scales).to(DEV))
    w = np.stack([mx.mx_rows_values(packed[e].reshape(out, inn // 2), scales[e].reshape(out, inn // 32)) for e in range(E)])
    return st, w


def _counts(E, rows, rng, empty=()):
    p = rng.random(E) + 0.1
    p[list(empty)] = 0
    return rng.multinomial(rows, p / p.sum())


def _act_errors(act, z, z_err):
    """The error of act(z) for one of z: |act'| <= 1.2, and a few steps of exp, erf and the quotient."""
    if act in ("none", "relu"):
        return z_err
    return 1.2 * z_err + 16 * U * (np.abs(z) + z * z * (np.abs(z) < 4))


PRODUCTS = [
    # E, rows, tail, in, out, act, bias, residual, y
    (1, 1, 0, 64, 1, "none", True, False, "fp32"), (1, 8, 0, 2048, 128, "none", False, False, "bf16"),
    (1, 5, 0, 192, 17, "gelu", True, True, "bf16"), (4, 13, 3, 128, 96, "silu", True, False, "fp32"),
    (128, 64, 0, 256, 80, "none", False, False, "bf16"), (3, 40, 0, 320, 260, "relu", True, True, "bf16"),
    (2, 0, 0, 64, 64, "none", True, False, "bf16"), (4, 0, 9, 64, 64, "silu", False, False, "fp32"),
    (1, 33, 2, 4096, 48, "gelu_tanh", True, False, "bf16"), (9, 200, 0, 2112, 300, "silu", True, False, "bf16"),
    (1, 300, 0, 512, 1030, "none", True, True, "fp32"), (1024, 50, 2, 64, 8, "none", True, False, "bf16"),
    (1, 700, 0, 1024, 513, "gelu", True, True, "bf16"), (5, 1500, 7, 448, 700, "relu", True, True, "bf16"),
    (2, 2500, 9, 128, 1000, "silu", True, True, "bf16"), (1, 2100, 0, 576, 2300, "none", False, False, "bf16"),
    (3, 3000, 5, 704, 1028, "gelu_tanh", True, True, "fp32"), (8, 4000, 0, 1024, 520, "none", True, False, "bf16"),
    (1, 1025, 3, 64, 1, "none", True, True, "fp32"), (1, 5000, 0, 64, 256, "silu", False, False, "bf16"),
    (6, 6000, 11, 1152, 1288, "none", True, True, "bf16"), (2, 4100, 0, 2048, 1027, "gelu", True, False, "fp32"),
]


@pytest.mark.parametrize("E,rows,tail,inn,out,act,with_bias,with_res,yt", PRODUCTS)
def test_product(E, rows, tail, inn, out, act, with_bias, with_res, yt):
    announce(f"mx product E={E} rows={rows}+{tail} {inn}->{out} {act} bias={with_bias} res={with_res} {yt}")
    rng = np.random.default_rng(rows + out)
    stack, w = _stack(E, out, inn, out + inn)
    R = rows + tail
    offsets = np.concatenate([[0], np.cumsum(_counts(E, rows, rng, (0,) if E > 2 else ()))]).astype(np.int32)
    off_d = torch.from_numpy(offsets).to(DEV) if E > 1 or tail else None
    x = rng.standard_normal((R, inn)) * np.exp(rng.standard_normal((R, 1)))
    x[rows:] = np.nan  # rows of no expert
    q = e4b.mx4_rows(dev(x, torch.bfloat16))
    xh = np.nan_to_num(mx.mx_rows_values(q.codes.cpu().numpy(), q.scales.cpu().numpy()))
    bias = dev(rng.standard_normal((E, out)) * 0.1, torch.float32) if with_bias else None
    res = dev(rng.standard_normal((R, out)), torch.bfloat16) if with_res else None
    bh, rh = None if bias is None else host(bias), None if res is None else host(res)
    y, pre = e4b.mx_linear(stack, q, offsets=off_d, bias=bias, act=act, residual=res, out_dtype=DT[yt], save=True)
    y_ref, z_ref = block.expert_linear(xh, w, offsets, bh, act, rh)
    zmag = block.expert_linear(np.abs(xh), np.abs(w), offsets, None if bh is None else np.abs(bh))[1]
    z_err = 2 * (inn + 4) * U * zmag
    within(pre, z_ref, z_err, "pre")
    live = (np.arange(R) < rows)[:, None]
    y_err = _act_errors(act, z_ref, z_err) + 2 * U * (np.abs(y_ref) + (0 if rh is None else np.abs(rh)))
    within(y, y_ref, y_err * live, "y")
    y2, none = e4b.mx_linear(stack, q, offsets=off_d, bias=bias, act=act, residual=res, out_dtype=DT[yt])
    assert none is None and torch.equal(bits(y2), bits(y))


# Products in every tiling, with rows enough for it: 128 x 128 tiles found by a map, 64 x 64 ones of many experts, and
# 256 x 256 ones, one a workgroup and several in turn, of 2 to 9 K-steps of 256 (whose scales come for 4 at a time).
LARGE = [
    (1024, 2990, 5, 128, 520, "relu", True, True, "bf16"), (700, 2500, 0, 192, 264, "none", False, False, "fp32"),
    (1, 4100, 0, 512, 2816, "none", False, False, "bf16"), (3, 5000, 0, 1280, 2312, "none", True, False, "bf16"),
    (5, 12000, 33, 768, 2048, "none", True, False, "bf16"), (2, 9000, 0, 512, 2504, "silu", True, True, "bf16"),
    (7, 9500, 130, 2304, 2056, "gelu", True, False, "fp32"), (300, 40000, 1, 1024, 2048, "none", False, True, "bf16"),
]


@pytest.mark.parametrize("E,rows,tail,inn,out,act,with_bias,with_res,yt", LARGE)
def test_product_in_every_tiling(E, rows, tail, inn, out, act, with_bias, with_res, yt):
    """The reference is summed by torch in 64 bits, on the GPU: numpy would take minutes."""
    announce(f"mx product E={E} rows={rows}+{tail} {inn}->{out} {act} bias={with_bias} res={with_res} {yt}")
    rng = np.random.default_rng(rows + out)
    stack, w = _stack(E, out, inn, out + inn)
    R, f64 = rows + tail, torch.float64
    offsets = np.concatenate([[0], np.cumsum(_counts(E, rows, rng, (0, E - 1) if E > 2 else ()))]).astype(np.int32)
    off_d = torch.from_numpy(offsets).to(DEV) if E > 1 or tail else None
    q = e4b.mx4_rows(dev(rng.standard_normal((R, inn)) * np.exp(rng.standard_normal((R, 1))), torch.bfloat16))
    x = torch.from_numpy(np.float32(mx.mx_rows_values(q.codes.cpu().numpy(), q.scales.cpu().numpy()))).to(DEV)
    bias = dev(rng.standard_normal((E, out)) * 0.1, torch.float32) if with_bias else None
    res = dev(rng.standard_normal((R, out)), torch.bfloat16) if with_res else None
    y, pre = e4b.mx_linear(stack, q, offsets=off_d, bias=bias, act=act, residual=res, out_dtype=DT[yt], save=True)
    y2, none = e4b.mx_linear(stack, q, offsets=off_d, bias=bias, act=act, residual=res, out_dtype=DT[yt])
    assert none is None and torch.equal(bits(y2), bits(y))
    assert not bits(y[rows:]).any() and not bits(pre[rows:]).any()
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        we, xe = torch.from_numpy(np.float32(w[e])).to(DEV).to(f64).t().contiguous(), x[a:b].to(f64)
        be = torch.zeros(out, device=DEV, dtype=f64) if bias is None else bias[e].to(f64)
        z = host(xe @ we + be)
        z_err = 2 * (inn + 4) * U * host(xe.abs() @ we.abs() + be.abs())
        within(pre[a:b], z, z_err, f"pre of expert {e}")
        ye, r = block.activation(act, z)[0], 0.0 if res is None else host(res[a:b])
        within(y[a:b], ye + r, _act_errors(act, z, z_err) + 2 * U * (np.abs(ye + r) + np.abs(r)), f"y of expert {e}")


@pytest.mark.parametrize("T,k,E,inn,out", [(3000, 4, 5, 768, 2048), (1200, 8, 300, 128, 2048)])
def test_gathered_in_large_tiles(T, k, E, inn, out):
    test_product_gathered_by_token(T, k, E, inn, out, 0.1)


def test_lists_that_lead_nowhere_in_large_tiles():
    test_lists_that_lead_nowhere_stay_inside(4, 12000, 512, 2048)


def test_tokens_beyond_32_bits():
    """Gathered rows of more than 2^32 bytes of codes."""
    announce("mx product gathered beyond 32 bits")
    T, inn, out = 8200, 2 ** 20, 64
    codes = torch.zeros(T, inn // 2, device=DEV, dtype=torch.uint8)
    scales = torch.full((T, inn // 32), 127, device=DEV, dtype=torch.uint8)
    stack, _ = _stack(1, out, inn, 12)
    g = torch.Generator(device=DEV).manual_seed(1)
    some = [0, 1, 4095, 4096, 8191, 8192, 8199]
    for t in some:
        codes[t] = torch.randint(0, 256, (inn // 2,), generator=g, device=DEV, dtype=torch.uint8)
    q = e4b.MxRows(codes, scales)
    perm = e4b.moe_permute(torch.zeros(T, 1, dtype=torch.int32, device=DEV), 1, torch.zeros(T, 8, device=DEV, dtype=torch.bfloat16))[1]
    y, _ = e4b.mx_linear(stack, q, perm=perm, out_dtype=torch.float32)
    alone, _ = e4b.mx_linear(stack, e4b.MxRows(codes[some], scales[some]), out_dtype=torch.float32)
    mag = 6 * 2.0 ** -5 * 6 * inn  # of the terms
    assert (y[some] - alone).abs().max().item() <= 4 * inn * U * mag
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[some] = False
    assert not y[rest].any() and alone.abs().max(dim=1).values.gt(0).all()


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
@pytest.mark.parametrize("inn,out", [(128, 64), (192, 300)])
def test_product_row_counts(rows, inn, out):
    announce(f"mx product rows={rows} {inn}->{out}")
    rng = np.random.default_rng(rows)
    stack, w = _stack(1, out, inn, 1)
    q = e4b.mx4_rows(dev(rng.standard_normal((rows, inn)), torch.bfloat16))
    y, _ = e4b.mx_linear(stack, q, out_dtype=torch.float32)
    xh = mx.mx_rows_values(q.codes.cpu().numpy(), q.scales.cpu().numpy())
    within(y, block.expert_linear(xh, w)[0], 2 * (inn + 4) * U * block.expert_linear(np.abs(xh), np.abs(w))[0], "y")


@pytest.mark.parametrize("T,k,E,inn,out,drop", [(1, 1, 1, 64, 16, 0.0), (9, 2, 4, 128, 33, 0.3), (8, 8, 128, 256, 80, 0.0),
                                                (300, 4, 7, 192, 200, 0.2), (1100, 2, 3, 320, 520, 0.1), (5, 3, 2, 64, 64, 1.0),
                                                (700, 8, 16, 1024, 264, 0.0), (2000, 3, 2, 64, 1030, 0.0), (0, 2, 4, 64, 64, 0.0)])
def test_product_gathered_by_token(T, k, E, inn, out, drop):
    """Rows read where their tokens lie give the bits of rows that were copied into expert order."""
    announce(f"mx product gathered T={T} k={k} E={E} {inn}->{out}")
    rng = np.random.default_rng(T + out)
    stack, _ = _stack(E, out, inn, 5)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    x = dev(rng.standard_normal((T, inn)), torch.bfloat16)
    rows, perm = e4b.moe_permute(torch.from_numpy(ids).to(DEV), E, x)
    bias = dev(rng.standard_normal((E, out)), torch.float32)
    y, pre = e4b.mx_linear(stack, e4b.mx4_rows(x), perm=perm, bias=bias, act="silu", save=True)
    y2, pre2 = e4b.mx_linear(stack, e4b.mx4_rows(rows), offsets=perm.offsets, bias=bias, act="silu", save=True)
    assert y.shape == (T * k, out) and torch.equal(bits(y), bits(y2)) and torch.equal(bits(pre), bits(pre2))
    live = int(perm.offsets[-1])
    assert not bits(y[live:]).any() and not bits(pre[live:]).any()


@pytest.mark.parametrize("E,rows,inn,out", [(4, 64, 128, 96), (4, 1200, 192, 520)])
def test_lists_that_lead_nowhere_stay_inside(E, rows, inn, out):
    """Offsets that do not ascend or leave the rows, and an order that names no pair."""
    announce(f"mx product bad lists rows={rows}")
    stack, _ = _stack(E, out, inn, 2)
    q = e4b.mx4_rows(torch.randn(rows, inn, device=DEV))
    big = torch.full((rows + 32, out), 7.0, device=DEV)  # the output with guard rows behind it
    for lists in ([0, 40, 10, rows, rows], [0, 16, 32, 48, 2 ** 31 - 1], [-7, -1, rows, rows, rows], [rows, 0, rows, 0, rows]):
        off = torch.tensor(lists, dtype=torch.int32, device=DEV)
        e4b.mx_linear(stack, q, offsets=off, out_dtype=torch.float32, out=big[:rows], save=True)
    order = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows,), device=DEV, dtype=torch.int64).to(torch.int32)
    perm = e4b.Permutation(torch.tensor([0, 5, 9, rows, rows], dtype=torch.int32, device=DEV), order,
                           torch.zeros(rows // 2, 2, dtype=torch.int32, device=DEV))
    e4b.mx_linear(stack, e4b.MxRows(q.codes[:rows // 2], q.scales[:rows // 2]), perm=perm, out_dtype=torch.float32, out=big[:rows])
    torch.cuda.synchronize()
    assert big[rows:].eq(7.0).all() and big[:rows].isfinite().all()


@pytest.mark.parametrize("rows,inn,out", [(20, 256, 96), (300, 128, 520), (2100, 448, 2304)])
def test_residual_added_in_place(rows, inn, out):
    rng = np.random.default_rng(rows)
    stack, _ = _stack(1, out, inn, 3)
    q = e4b.mx4_rows(dev(rng.standard_normal((rows, inn)), torch.bfloat16))
    res = dev(rng.standard_normal((rows, out)), torch.bfloat16)
    want = e4b.mx_linear(stack, q, act="silu", residual=res)[0]
    got = e4b.mx_linear(stack, q, act="silu", residual=res, out=res)[0]
    assert got.data_ptr() == res.data_ptr() and torch.equal(bits(got), bits(want))


def test_products_of_extreme_scales():
    """Scales from one end to the other: sums near fp32's largest values and below its smallest."""
    announce("mx product of extreme scales")
    stack, w = _stack(1, 32, 128, 9, lo=190, hi=192)
    q = e4b.mx4_rows(torch.randn(32, 128, device=DEV) * 2.0 ** 30)
    xh = mx.mx_rows_values(q.codes.cpu().numpy(), q.scales.cpu().numpy())
    y, _ = e4b.mx_linear(stack, q, out_dtype=torch.float32)
    within(y, xh @ w[0].T, 2 * 132 * U * (np.abs(xh) @ np.abs(w[0]).T), "large")
    stack, w = _stack(1, 32, 128, 10, lo=0, hi=3)
    y, _ = e4b.mx_linear(stack, e4b.mx4_rows(torch.randn(32, 128, device=DEV) * 2.0 ** -60), out_dtype=torch.float32)
    assert not y.any()  # 2^-180 has no fp32 value


def test_offsets_beyond_32_bits():
    """A stack of more than 2^32 codes, and outputs of more than 2^31 values."""
    announce("mx product beyond 32 bits")
    E, out, inn = 3, 65536, 49152
    g = torch.Generator(device=DEV).manual_seed(0)
    packed = torch.randint(0, 256, (E, out * inn // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(118, 123, (E, out * inn // 32), generator=g, device=DEV, dtype=torch.uint8)
    stack = e4b.QuantStack(packed, None, E, out, inn, "mxfp4", scales)
    q = e4b.mx4_rows(torch.randn(5, inn, device=DEV))
    off = torch.tensor([0, 1, 2, 5], dtype=torch.int32, device=DEV)
    y, _ = e4b.mx_linear(stack, q, offsets=off, out_dtype=torch.float32)
    last = e4b.QuantStack(packed[2, -64 * inn // 2:][None], None, 1, 64, inn, "mxfp4", scales[2, -64 * inn // 32:][None])
    alone, _ = e4b.mx_linear(last, e4b.MxRows(q.codes[2:], q.scales[2:]), out_dtype=torch.float32)
    mag = e4b.mx4_values(e4b.MxRows(q.codes[2:], q.scales[2:]), torch.float32).abs().sum(dim=1).max().item() * 6 * 2.0 ** -5
    assert (y[2:, -64:] - alone).abs().max().item() <= 4 * inn * U * mag
    del y, packed, scales, stack
    rows, out, inn = 40000, 65536, 64
    stack, _ = _stack(1, out, inn, 11)
    q = e4b.mx4_rows(torch.randn(rows, inn, device=DEV))
    y, _ = e4b.mx_linear(stack, q)
    tail = e4b.MxRows(q.codes[-104:], q.scales[-104:])
    alone, _ = e4b.mx_linear(stack, tail)
    assert torch.equal(bits(y[-104:]), bits(alone))  # (64 products a sum: one instruction's, in any tiling)


def test_refusals_on_the_device():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    q = e4b.mx4_rows(x)
    stack, _ = _stack(2, 64, 64, 0)
    one, _ = _stack(1, 64, 64, 0)
    nf4 = e4b.quantize(torch.zeros(1, 64, 64, device=DEV), "nf4")
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    perm = e4b.moe_permute(ids, 2)[1]
    ones = torch.ones(64, device=DEV)
    bad = [
        lambda: e4b.mx4_rows(x[:, :32]),
        lambda: e4b.mx4_rows(x[:, ::2].contiguous()),
        lambda: e4b.mx4_rows(x.view(-1)),
        lambda: e4b.mx4_rows(x, gated=True),  # K = 32
        lambda: e4b.mx4_rows_backward(torch.zeros(4, 128, device=DEV), x[:3]),
        lambda: e4b.mx4_values(e4b.MxRows(q.codes, q.scales[:3])),
        lambda: e4b.mx4_values(e4b.MxRows(q.codes[:, :16].contiguous(), q.scales)),
        lambda: e4b.mx4_values(q, torch.float16),
        lambda: e4b.mx_linear(stack, q),  # two experts, no offsets
        lambda: e4b.mx_linear(nf4, q),
        lambda: e4b.mx_linear(stack, q, offsets=off[:2]),
        lambda: e4b.mx_linear(stack, q, offsets=off, perm=perm),
        lambda: e4b.mx_linear(one, q, perm=perm),  # an order of two experts
        lambda: e4b.mx_linear(stack, e4b.MxRows(q.codes[:3], q.scales[:3]), perm=perm),
        lambda: e4b.mx_linear(stack, e4b.mx4_rows(torch.zeros(4, 128, device=DEV)), offsets=off),
        lambda: e4b.mx_linear(stack, q, offsets=off, act="tanh"),
        lambda: e4b.mx_linear(stack, q, offsets=off, bias=ones),
        lambda: e4b.mx_linear(stack, q, offsets=off, residual=x[:3]),
        lambda: e4b.mx_linear(stack, q, offsets=off, out_dtype=torch.float16),
        lambda: e4b.mx_linear(stack, q, offsets=off, out=x[:2]),
        lambda: e4b.mx_linear(one, q, residual=x, out=x.float(), out_dtype=torch.bfloat16),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} was not refused")


# ---- together ----


def _tensors(*vs):
    return [t for v in vs for t in (v if isinstance(v, (list, tuple)) else [v]) if t is not None]


class Experts:
    """A router kept even and its experts in 4 bits, trained through, as a user joins them."""

    def __init__(self, T=160, H=256, I=192, E=8, k=2, seed=0):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.router = e4b.quantize(dev(rng.standard_normal((1, E, H)) * 0.1, torch.float32), "bf16")
        self.up, self.up_w = _stack(E, 2 * I, H, seed + 1)
        self.dn, self.dn_w = _stack(E, H, I, seed + 2)
        self.x = dev(rng.standard_normal((T, H)), torch.bfloat16)
        self.grad = dev(rng.standard_normal((T, H)), torch.bfloat16)
        self.mask = torch.from_numpy(rng.random(T) > 0.1).to(DEV)
        self.cu = torch.tensor([0, T // 3, T // 2, T], dtype=torch.int32, device=DEV)
        self.weights = torch.full((3,), 0.01, device=DEV), torch.full((3,), 1e-3, device=DEV)

    def forward(self):
        s = self
        s.logits, _ = e4b.expert_linear(s.router, s.x, out_dtype=torch.float32)
        s.idx, s.w = e4b.moe_route(s.logits, s.k)
        s.bal = e4b.moe_balance(s.logits, s.idx, cu_tokens=s.cu, token_mask=s.mask)
        _, s.perm = e4b.moe_permute(s.idx, s.E)
        s.q = e4b.mx4_rows(s.x)
        s.gu, _ = e4b.mx_linear(s.up, s.q, perm=s.perm)
        s.a = e4b.mx4_rows(s.gu, gated=True)
        s.o, _ = e4b.mx_linear(s.dn, s.a, offsets=s.perm.offsets)
        s.y = e4b.moe_unpermute(s.perm, s.o, s.w)
        return [s.y, s.bal.loss, s.bal.z_loss]

    def backward(self):
        s = self
        go, gw = e4b.moe_unpermute_backward(s.perm, s.o, s.grad, s.w)
        ga, _ = e4b.expert_linear_dgrad(s.dn, go, offsets=s.perm.offsets)
        ggu = e4b.mx4_rows_backward(s.gu, ga)
        grows, _ = e4b.expert_linear_dgrad(s.up, ggu, offsets=s.perm.offsets)
        gl = e4b.moe_route_backward(s.idx, s.w, gw, s.E)
        gl = e4b.moe_balance_backward(s.bal, s.logits, *s.weights, cu_tokens=s.cu, add=gl, out=gl)
        gx, _ = e4b.expert_linear_dgrad(s.router, gl)
        return [e4b.moe_permute_backward(s.perm, grows), gx, gl]


def test_experts_in_4_bits_forward_and_backward():
    """The chain in 64 bits from each tensor that the library rounded (the rows' codes among them), so
    that no code lies on the other side of a border: every output is one rounding to its type and its
    sums' steps away, bounded by 2^-7 of the largest value where no sum cancels to less."""
    announce("experts in 4 bits forward and backward")
    s = Experts()
    y, loss, z = s.forward()
    grows, gx_router, gl = s.backward()
    off, pos, idx = (t.cpu().numpy() for t in (s.perm.offsets, s.perm.pos, s.idx))
    order = s.perm.sorted_pair.cpu().numpy()
    close = lambda got, want, name: tuple([  # noqa: E731
        np.testing.assert_array_less(np.max(np.abs(host(got) - want)), 2.0 ** -7 * np.max(np.abs(want)), err_msg=name)])
    same_rows(s.q, host(s.x), "x")
    xq = host(e4b.mx4_values(s.q))
    gu, _ = block.expert_linear(xq[order // s.k], s.up_w, off)
    close(s.gu, gu, "gate_up")
    same_rows(s.a, block.swiglu(host(s.gu))[0], "a")
    o, _ = block.expert_linear(host(e4b.mx4_values(s.a)), s.dn_w, off)
    close(s.o, o, "down")
    close(y, block.unpermute(host(s.o), off, pos, host(s.w)), "y")
    bal = block.balance(host(s.logits), idx, s.cu.cpu().numpy(), s.mask.cpu().numpy())
    close(loss, bal["loss"], "loss")
    close(z, bal["z"], "z")
    go, gw = block.unpermute_backward(host(s.o), off, pos, host(s.w), host(s.grad))
    zero = np.zeros_like
    ga = block.expert_linear_dgrad(go, zero(go), s.dn_w, off)[0]
    _, dg, du = block.swiglu(host(s.gu))
    ggu = np.concatenate([ga * dg, ga * du], axis=1)
    rows = block.expert_linear_dgrad(ggu, zero(ggu), s.up_w, off)[0]
    err = np.max(np.abs(host(grows) - block.unpermute(rows, off, pos)))
    # three tensors between are rounded to bf16: grad_a, grad of [g | u] and the rows
    assert err <= 4 * 2.0 ** -8 * np.max(np.abs(block.unpermute(np.abs(rows), off, pos)))
    want = block.route_backward(idx, host(s.w), gw, s.E)
    want = block.balance_backward(bal, host(s.logits), s.k, *[host(t) for t in s.weights], s.cu.cpu().numpy(), want)
    close(gl, want, "grad_logits")


def test_two_runs_and_another_stream():
    s = Experts(T=333, seed=3)
    want = _tensors(s.forward(), s.backward())
    again = _tensors(s.forward(), s.backward())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = _tensors(s.forward(), s.backward())
    torch.cuda.current_stream().wait_stream(stream)
    for p, q, r in zip(want, again, got):
        assert torch.equal(bits(p), bits(q)) and torch.equal(bits(p), bits(r))


def test_captured_and_replayed():
    announce("experts in 4 bits in a graph")
    s, eager = Experts(T=700, seed=4), Experts(T=700, seed=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.forward()
        s.backward()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _tensors(s.forward(), s.backward())
    for rep in range(4):
        x = torch.randn(700, 256, device=DEV).to(torch.bfloat16)
        s.x.copy_(x)
        eager.x.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        want = _tensors(eager.forward(), eager.backward())
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(out, want)):
            assert torch.equal(bits(p), bits(q)), (rep, i)


@pytest.mark.parametrize("E,rows,inn,out", [(1, 3, 256, 64), (6, 60, 192, 640), (3, 900, 320, 2000), (4, 5000, 128, 520),
                                            (4, 12000, 768, 2048)])
def test_product_captured_in_every_tiling(E, rows, inn, out):
    """New rows and new offsets between replays; both graphs of a workspace."""
    announce(f"mx product in a graph E={E} rows={rows} {inn}->{out}")
    rng = np.random.default_rng(rows)
    stack, _ = _stack(E, out, inn, 4)
    q = e4b.mx4_rows(dev(rng.standard_normal((rows, inn)), torch.bfloat16))
    off = torch.zeros(E + 1, device=DEV, dtype=torch.int32)
    bias = dev(rng.standard_normal((E, out)), torch.float32)
    ws = torch.empty(max(256, e4b.mx_linear_workspace_bytes(stack, rows)), device=DEV, dtype=torch.uint8)
    run = lambda: e4b.mx_linear(stack, q, offsets=off, bias=bias, act="relu", save=True, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out_t = run()
        graphs.append((graph, out_t))
    for rep in range(4):
        new = e4b.mx4_rows(dev(rng.standard_normal((rows, inn)), torch.bfloat16))
        q.codes.copy_(new.codes)
        q.scales.copy_(new.scales)
        off.copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(_counts(E, rows - rep, rng))]).astype(np.int32)))
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for _, got in graphs:
            for a, b in zip(got, want):
                assert torch.equal(bits(a), bits(b)), rep
