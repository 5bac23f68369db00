"""Values at the edges of the operators around the expert MLP: NaN and infinities that a
diverged model has in live rows, far tails, skewed routings, every tiling's row counts.

Tolerances as in test_gpu_block: counted in steps U = 2^-24 of fp32 and half steps of the
output's type, derived beside each test.
"""

import functools
import math

import numpy as np
import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
from gpu_util import DEV, announce
from oracle import block
from plan_util import ROWS, T128, T256, TALL, linear_plan
from test_gpu_block import U, _norm_inputs, _stack, bits, dev, host, within

pytestmark = pytest.mark.gpu


# few rows, 128 x 128 tiles cut along k, 256 x 128, 256 x 256
TILINGS = [(1, 20, 128, 96), (1, 300, 2048, 520), (1, 2100, 448, 2300), (2, 3500, 192, 4104)]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("E,rows,inn,out", TILINGS)
def test_nan_passes_every_activation(E, rows, inn, out, act):
    """A NaN in a live row's x, in a bias or in a gradient shows in everything that it enters, and
    in nothing else: the other elements keep their bits."""
    announce(f"NaN through {act} E={E} rows={rows} {inn} -> {out}")
    rng = np.random.default_rng(rows)
    stack, _ = _stack(E, out, inn, "nf4", 3)
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device=DEV) if E > 1 else None
    x = dev(rng.standard_normal((rows, inn)), torch.bfloat16)
    bias = dev(rng.standard_normal((E, out)) * 0.1, torch.float32)
    gy = dev(rng.standard_normal((rows, out)), torch.bfloat16)
    y, pre = e4b.expert_linear(stack, x, off, bias, act, save=True)
    gx, gb = e4b.expert_linear_dgrad(stack, gy, offsets=off, act=act, pre=pre, grad_bias=True)

    r, c = rows - 3, out // 2  # a row of the last expert, a column
    bad_x, bad_b = x.clone(), bias.clone()
    bad_x[r, 5] = float("nan")
    bad_b[0, c] = float("nan")
    y2, pre2 = e4b.expert_linear(stack, bad_x, off, bad_b, act, save=True)
    n0 = rows // 2 if E > 1 else rows  # rows of expert 0
    want = torch.zeros(rows, out, dtype=torch.bool, device=DEV)
    want[r] = True
    want[:n0, c] = True
    assert torch.equal(y2.isnan(), want) and torch.equal(pre2.isnan(), want)
    assert torch.equal(bits(y2)[~want], bits(y)[~want])

    # the gradient of a row whose pre-activation is NaN (an activation's), then of a NaN gradient
    if act != "none":
        bad_pre = pre.clone()
        bad_pre[r] = float("nan")
        gx2, gb2 = e4b.expert_linear_dgrad(stack, gy, offsets=off, act=act, pre=bad_pre, grad_bias=True)
        assert gx2[r].isnan().all() and gb2[E - 1].isnan().all()
        keep = torch.arange(rows, device=DEV) != r
        assert torch.equal(bits(gx2)[keep], bits(gx)[keep]) and torch.equal(bits(gb2)[:E - 1], bits(gb)[:E - 1])
    low = int(pre[r].argmin())  # where max(z, 0) is flat: NaN times 0
    assert pre[r, low] < 0
    bad_gy = gy.clone()
    bad_gy[r, low] = float("nan")
    gx2, gb2 = e4b.expert_linear_dgrad(stack, bad_gy, offsets=off, act=act, pre=pre, grad_bias=True)
    assert gx2[r].isnan().all() and gb2[E - 1, low].isnan() and int(gb2.isnan().sum()) == 1
    keep = torch.arange(rows, device=DEV) != r
    assert torch.equal(bits(gx2)[keep], bits(gx)[keep])


@pytest.mark.parametrize("T,H,dt", [(5, 264, "bf16"), (9, 33, "fp32"), (3, 4104, "fp32"), (600, 512, "bf16"), (2, 16384, "bf16")])
@pytest.mark.parametrize("gate", [None, "token", "channel"])
@pytest.mark.parametrize("post", [False, True])
def test_block_norm_gradient_without_pre_norm_of_an_overflowed_block(T, H, dt, gate, post):
    """Without w_pre, r = x + scale g u: grad_x is grad_r whatever y holds, and without w_post
    grad_y = scale g grad_r. An infinity, a NaN or a product beyond fp32 in y reaches only what y is
    a factor of: its row's token gate, its column's channel gate."""
    announce(f"norm backward of an overflowed y T={T} H={H} {dt} gate={gate} post={post}")
    rng = np.random.default_rng(H)
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    x, y = dev(rng.standard_normal((T, H)), dtype), dev(rng.standard_normal((T, H)), torch.bfloat16)
    gr = dev(rng.standard_normal((T, H)), dtype)
    kw = {"scale": 4.0}
    if post:
        kw["w_post"] = dev(1 + 0.1 * rng.standard_normal(H), torch.float32)
    g = 1.0
    if gate:
        g = dev(1 + rng.random(T if gate == "token" else H), torch.float32)
        kw["gate_" + gate] = g
        g = g[:, None] if gate == "token" else g
    clean = e4b.block_norm_backward(e4b.block_norm(x, y=y, **kw), x, gr, y=y, **kw)
    row, cols = T - 2, [1, H // 2, H - 1]
    bad = y.clone()
    bad[row, cols] = torch.tensor([float("inf"), float("nan"), 3e38], dtype=torch.bfloat16, device=DEV)
    f = e4b.block_norm(x, y=bad, **kw)
    b = e4b.block_norm_backward(f, x, gr, y=bad, **kw)
    assert torch.equal(bits(b.grad_x), bits(gr))
    keep = torch.arange(T, device=DEV) != row
    assert torch.equal(bits(b.grad_y)[keep], bits(clean.grad_y)[keep])
    if post:  # the row's own statistic is lost: nothing to expect of its grad_y
        return
    # grad_y is one product of three (two of them exact powers) rounded to bf16: as without the bad values
    assert torch.equal(bits(b.grad_y), bits(clean.grad_y))
    if gate == "token":
        assert torch.equal(bits(b.grad_gate)[keep], bits(clean.grad_gate)[keep]) and not b.grad_gate[row].isfinite()
    elif gate == "channel":
        ok = torch.ones(H, dtype=torch.bool, device=DEV)
        ok[cols] = False
        assert torch.equal(bits(b.grad_gate)[ok], bits(clean.grad_gate)[ok])
        assert b.grad_gate[cols[0]].isinf() and b.grad_gate[cols[1]].isnan()


def _act_values(act, z):
    """(act(z), act'(z)) as the kernels compute them in fp32, one value each: zero weights and the
    bias z give the forward, a kept pre-activation z and grad_y = 1 the bias gradient."""
    n = z.shape[0]
    stack = e4b.quantize(torch.zeros(1, n, 64, device=DEV), "bf16")
    zd = dev(z[None], torch.float32)
    y, pre = e4b.expert_linear(stack, torch.zeros(1, 64, dtype=torch.bfloat16, device=DEV), bias=zd, act=act,
                               out_dtype=torch.float32, save=True)
    assert torch.equal(pre, zd)
    _, gb = e4b.expert_linear_dgrad(stack, torch.ones(1, n, device=DEV), act=act, pre=zd, grad_bias=True)
    return host(y)[0], host(gb)[0]


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_activations_of_the_largest_values(act):
    """Far from 0 every activation is z or 0 and its slope 1 or 0, up to the largest finite fp32."""
    z = np.float32([100.0, 1e6, 1e13, 1.8e19, 1.9e19, 1e20, 1e30, 3.4e38])
    y, d = _act_values(act, np.concatenate([z, -z]))
    n = len(z)
    assert np.array_equal(y[:n], z.astype(np.float64)) and not y[n:].any()
    assert np.array_equal(d[:n], np.ones(n)) and not d[n:].any()


def test_gelu_far_below_zero():
    """z Phi(z) and its slope to a relative accuracy where they are small: erfc(x) e^(x^2) is fitted to
    1.4 U and evaluated within 8 (7 multiply-adds of terms that partly cancel, a reciprocal); x = |z| / sqrt 2
    is off by 2 U, so the exponent -x^2 by 5 x^2 U and its scaling to base 2 by 2 more: 3.5 z^2 U; the
    exponential, the halving product and z's own add 4. The slope Phi + z phi adds the density's
    error, the same exponential's, to each of two terms that do not cancel below -2."""
    z = np.linspace(-12.5, -0.25, 4099).astype(np.float32)
    y, d = _act_values("gelu", z)
    zz = z.astype(np.float64)
    phi = np.array([0.5 * math.erfc(-v / math.sqrt(2.0)) for v in zz])
    rel = (4 * zz * zz + 24) * U
    bad = np.abs(y - zz * phi) > rel * np.abs(zz * phi)
    assert not bad.any(), (zz[bad][0], y[bad][0], (zz * phi)[bad][0])
    dens = zz * np.exp(-0.5 * zz * zz) / math.sqrt(2.0 * math.pi)
    bad = np.abs(d - (phi + dens)) > rel * (phi + np.abs(dens))
    assert not bad.any(), (zz[bad][0], d[bad][0], (phi + dens)[bad][0])


# E, rows, in, out, the expert that takes all but a few rows, the forward's tiles
SKEWED = [(128, 1024, 256, 128, 77, ROWS), (4, 5000, 64, 96, 2, ROWS), (2, 700, 512, 130, 0, ROWS), (512, 4000, 128, 64, 511, ROWS),
          (3, 200, 192, 96, 1, ROWS), (16, 600, 1088, 1024, 5, T128), (3, 1900, 448, 2304, 1, TALL), (2, 3500, 192, 4104, 1, T256)]


@pytest.mark.parametrize("E,rows,inn,out,hot,tiles", SKEWED)
def test_one_hot_expert_of_many(E, rows, inn, out, hot, tiles):
    """Nearly every row on one expert, in every tiling: each element against 64 bits, and rows of no
    expert as zeros."""
    announce(f"hot expert {hot} of {E}, rows={rows} {inn} -> {out}")
    rng = np.random.default_rng(E + rows)
    R = rows + 7
    assert linear_plan(E, R, inn, out)[0] == tiles
    stack, w = _stack(E, out, inn, "nf4", 5)
    counts = np.zeros(E, dtype=np.int64)
    counts[(hot + 1) % E] = counts[(hot * 7 + 3) % E] = 3
    counts[hot] = 0
    counts[hot] = rows - counts.sum()
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    off = torch.from_numpy(offsets).to(DEV)
    x = dev(rng.standard_normal((R, inn)), torch.bfloat16)
    bias = dev(rng.standard_normal((E, out)) * 0.1, torch.float32)
    y, pre = e4b.expert_linear(stack, x, off, bias, out_dtype=torch.float32, save=True)
    ref = block.expert_linear(host(x), w, offsets, host(bias))[0]
    mag = block.expert_linear(np.abs(host(x)), np.abs(w), offsets, np.abs(host(bias)))[0]
    within(y, ref, mag * (inn + 4) * U, "y")
    assert torch.equal(y, pre) and not bits(y[rows:]).any()
    gy = dev(rng.standard_normal((R, out)), torch.bfloat16)
    gx, gb = e4b.expert_linear_dgrad(stack, gy, offsets=off, grad_bias=True)
    gyh = host(gy)
    gyh[rows:] = 0.0
    gx_ref, gb_ref = block.expert_linear_dgrad(gyh, gyh, w, offsets)
    within(gx, gx_ref, block.expert_linear_dgrad(np.abs(gyh), gyh, np.abs(w), offsets)[0] * (out + 4) * U, "grad_x")
    within(gb, gb_ref, block.expert_linear_dgrad(np.abs(gyh), gyh, w, offsets)[1] * (rows + 8) * U, "grad_bias")


def _time(call):
    best = float("inf")
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def test_a_hot_expert_takes_no_longer_than_the_same_rows_alone():
    """100000 rows of one of four experts spread over the chip as those of a single expert do (19 us;
    in a fixed number of row slices per expert they took 1200). Ten times is a bound on the spread of
    the work, not on its speed."""
    announce("time of a hot expert")
    rows = 100000
    x = torch.randn(rows, 64, device=DEV).to(torch.bfloat16)
    off = torch.tensor([0, 0, rows, rows, rows], dtype=torch.int32, device=DEV)
    one, four = _stack(1, 64, 64, "nf4", 6)[0], _stack(4, 64, 64, "nf4", 6)[0]

    alone, hot = _time(lambda: e4b.expert_linear(one, x)), _time(lambda: e4b.expert_linear(four, x, off))
    assert hot < 10 * alone, (hot, alone)


# E, rows, those of an expert, in, out, y, the forward's tiles
TAILS = [(3, 3000, 5, 64, 129, "bf16", ROWS), (1, 500, 0, 64, 64, "bf16", ROWS), (3, 3001, 1, 64, 33, "fp32", ROWS),
         (2, 700, 9, 1024, 1023, "bf16", T128), (2, 700, 699, 1024, 1024, "fp32", T128), (3, 1907, 11, 448, 2303, "bf16", TALL),
         (2, 3507, 300, 192, 4104, "bf16", T256)]


@pytest.mark.parametrize("E,R,live,inn,out,yt,tiles", TAILS)
def test_most_rows_of_no_expert(E, R, live, inn, out, yt, tiles):
    """Every row from offsets[E] on is zeros in y, the pre-activation and grad_x, to the last element
    and no further; the rows before are those of the same call without them."""
    announce(f"{R - live} of {R} rows of no expert, {inn} -> {out} {yt}")
    rng = np.random.default_rng(R)
    assert linear_plan(E, R, inn, out)[0] == tiles
    stack, w = _stack(E, out, inn, "nf4", 7)
    offsets = np.linspace(0, live, E + 1).astype(np.int32)
    off = torch.from_numpy(offsets).to(DEV)
    x = dev(rng.standard_normal((R, inn)), torch.bfloat16)
    x[live:] = float("nan")
    dtype = {"bf16": torch.bfloat16, "fp32": torch.float32}[yt]
    big = torch.full((R + 3, out), 7.0, dtype=dtype, device=DEV)
    y, pre = e4b.expert_linear(stack, x, off, out_dtype=dtype, save=True, out=big[:R])
    assert not bits(y[live:]).any() and not bits(pre[live:]).any() and big[R:].eq(7.0).all()
    xh = host(x)
    xh[live:] = 0.0
    ref = block.expert_linear(xh, w, offsets)[0]
    mag = block.expert_linear(np.abs(xh), np.abs(w), offsets)[0]
    within(y, ref, mag * (inn + 4) * U, "y")
    gy = dev(rng.standard_normal((R, out)), torch.bfloat16)
    gy[live:] = float("inf")
    gx, _ = e4b.expert_linear_dgrad(stack, gy, offsets=off)
    assert not bits(gx[live:]).any() and (live < 2 or bits(gx[:live]).any())


def test_rows_of_no_expert_cost_no_more_than_rows_of_one():
    """100000 rows of no expert are cleared by the whole chip (four workgroups took 1200 us, the same rows
    of an expert 19). Ten times is a bound on the spread of the work, not on its speed."""
    announce("time of rows of no expert")
    rows = 100100
    x = torch.randn(rows, 64, device=DEV).to(torch.bfloat16)
    off = torch.tensor([0, 100], dtype=torch.int32, device=DEV)
    stack = _stack(1, 64, 64, "nf4", 6)[0]
    alone, none = _time(lambda: e4b.expert_linear(stack, x)), _time(lambda: e4b.expert_linear(stack, x, off))
    assert none < 10 * alone, (none, alone)


@functools.lru_cache(maxsize=None)
def _wide_stack(out, inn):
    return _stack(1, out, inn, "nf4", 8)


# rows, the forward's tiles, in, out; the products of 4096 -> 1100 are cut along k
COUNTS = [(127, T128, 320, 16520), (128, T128, 320, 16520), (129, TALL, 320, 16520), (255, TALL, 320, 16520),
          (256, TALL, 320, 16520), (257, T128, 320, 16520), (384, T128, 320, 16520), (385, T256, 320, 16520),
          (511, T256, 320, 16520), (512, T256, 320, 16520), (513, T256, 320, 16520), (127, T128, 4096, 1100),
          (128, T128, 4096, 1100), (129, T128, 4096, 1100), (256, T128, 4096, 1100), (257, T128, 4096, 1100)]


@pytest.mark.parametrize("rows,tiles,inn,out", COUNTS)
def test_counts_at_which_a_row_tile_begins_or_ends(rows, tiles, inn, out):
    """Against 64 bits, in the tiles that the count is meant to reach; a row's bits do not depend on
    where it stands among the rows."""
    announce(f"{rows} rows of {inn} -> {out}")
    plan = linear_plan(1, rows, inn, out)
    assert plan[0] == tiles and (plan[2] > 1) == (inn == 4096)
    stack, w = _wide_stack(out, inn)
    x = dev(np.random.default_rng(rows).standard_normal((rows, inn)), torch.bfloat16)
    y, _ = e4b.expert_linear(stack, x, out_dtype=torch.float32)
    ref = block.expert_linear(host(x), w)[0]
    within(y, ref, block.expert_linear(np.abs(host(x)), np.abs(w))[0] * (inn + 4) * U, "y")
    back, _ = e4b.expert_linear(stack, x.flip(0).contiguous(), out_dtype=torch.float32)
    assert torch.equal(bits(back.flip(0)), bits(y))


@pytest.mark.parametrize("rows,tiles", [(127, T128), (128, T128), (129, TALL), (256, TALL), (257, T128), (384, T128),
                                        (385, T256), (512, T256), (513, T256)])
def test_counts_at_which_a_row_tile_of_the_gradient_begins_or_ends(rows, tiles):
    announce(f"gradient of {rows} rows of 16512 -> 320")
    assert linear_plan(1, rows, 16512, 320)[1] == tiles
    stack, w = _wide_stack(320, 16512)
    gy = dev(np.random.default_rng(rows).standard_normal((rows, 320)), torch.bfloat16)
    gx, gb = e4b.expert_linear_dgrad(stack, gy, grad_bias=True)
    gyh = host(gy)
    ref, gb_ref = block.expert_linear_dgrad(gyh, gyh, w)
    mag, gb_mag = block.expert_linear_dgrad(np.abs(gyh), gyh, np.abs(w))
    within(gx, ref, mag * (320 + 4) * U, "grad_x")
    within(gb, gb_ref, gb_mag * (rows + 8) * U, "grad_bias")
    back, _ = e4b.expert_linear_dgrad(stack, gy.flip(0).contiguous())
    assert torch.equal(bits(back.flip(0)), bits(gx))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H", [(1, 32, 16383), (3, 9, 8192), (17, 17, 2337), (130, 8, 640), (1030, 9, 136), (4096, 9, 24),
                                   (5000, 3, 1), (999, 32, 16), (333, 5, 17), (700, 2, 128), (4097, 17, 8)])
def test_way_back_of_few_tokens_and_of_narrow_rows(T, k, H, dt):
    """The gradients against 64 bits however a token's slots are spread over waves, and y."""
    announce(f"way back T={T} k={k} H={H} {dt}")
    rng = np.random.default_rng(T + H)
    ids = rng.integers(-1, 6, (T, k)).astype(np.int32)
    _, perm = e4b.moe_permute(torch.from_numpy(ids).to(DEV), 6)
    offsets, pos = perm.offsets.cpu().numpy(), perm.pos.cpu().numpy()
    live = int(offsets[-1])
    rows, gy = dev(rng.standard_normal((T * k, H)), dt), dev(rng.standard_normal((T, H)), dt)
    rows[live:] = float("nan")
    w = dev(rng.random((T, k)), torch.float32)
    rh = np.nan_to_num(host(rows))
    on = pos < live
    place = np.where(on, pos, 0)
    at = rh[place] * on[..., None]
    y = e4b.moe_unpermute(perm, rows, w)
    within(y, (at * host(w)[..., None]).sum(1), (np.abs(at) * host(w)[..., None]).sum(1) * (k + 1) * U, "y")
    gr, gw = e4b.moe_unpermute_backward(perm, rows, gy, w)
    gyh = host(gy)[:, None, :]
    within(gw, (at * gyh).sum(2), (np.abs(at * gyh)).sum(2) * (H + 2) * U, "grad_w")
    ref = np.zeros((T * k, H))
    ref[pos[on]] = (host(w)[..., None] * gyh)[on]
    within(gr, ref, np.abs(ref) * U, "grad_rows")
    gr2, _ = e4b.moe_unpermute_backward(perm, None, gy, w, grad_w=False)
    assert torch.equal(bits(gr2), bits(gr))


def test_way_back_spreads_over_the_chip():
    """A gradient of one token with many slots, and narrow rows of many tokens, against the same pairs as
    tokens of one slot and as wide rows (1200 us against 12 and 211 against 10 where a wave takes
    a token and a workgroup a row; 25 and 26 now). Ten times bounds the spread, not the speed."""
    announce("time of the way back")

    def args(T, k, H):
        ids = torch.randint(0, 64, (T, k), device=DEV, dtype=torch.int32)
        return e4b.moe_permute(ids, 64)[1], torch.randn(T * k, H, device=DEV), torch.rand(T, k, device=DEV), torch.randn(T, H, device=DEV)

    def back(T, k, H):
        p, rows, w, gy = args(T, k, H)
        return _time(lambda: e4b.moe_unpermute_backward(p, rows, gy, w))

    def forth(T, k, H):
        p, rows, w, _ = args(T, k, H)
        return _time(lambda: e4b.moe_unpermute(p, rows, w))

    assert back(1, 32, 16383) < 10 * back(32, 1, 16383)
    assert forth(48482, 27, 3) < 10 * forth(190, 27, 768)


@pytest.mark.parametrize("H", [4097, 5120, 8191, 8192, 8200, 9634, 12288, 16383, 16384])
@pytest.mark.parametrize("dt,has_y,post,gate,pre", [("bf16", True, True, "token", True), ("fp32", True, True, "channel", True),
                                                    ("fp32", True, False, None, False), ("bf16", True, True, "channel", False),
                                                    ("fp32", False, False, None, True), ("bf16", True, False, "token", False)])
def test_long_rows(H, dt, has_y, post, gate, pre):
    """Rows beyond 4096 columns, more of them than workgroups, with guards behind every output: the
    gradients against differentiation in 64 bits, to the steps that test_block_norm_and_its_gradient
    derives (H + 24 of a row's sums, four of them; T + 16 of a column's)."""
    T = 300
    announce(f"long rows H={H} {dt} y={has_y} post={post} gate={gate} pre={pre}")
    x, kw, gr, gh = _norm_inputs(T, H, dt, has_y, post, gate, pre)
    f = e4b.block_norm(x, scale=0.5, **kw)
    g = e4b.block_norm_backward(f, x, gr, gh, scale=0.5, **kw)
    leaf = {n: v.double().cpu().requires_grad_(True) for n, v in [("x", x)] + list(kw.items())}

    def rms(v, w):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w

    r = leaf["x"] * 1.0
    if has_y:
        u = rms(leaf["y"], leaf["w_post"]) if post else leaf["y"]
        gv = {"token": lambda: leaf["gate_token"][:, None], "channel": lambda: leaf["gate_channel"], None: lambda: 1.0}[gate]()
        r = r + 0.5 * gv * u
    loss = (r * gr.double().cpu()).sum()
    if pre:
        loss = loss + (rms(r, leaf["w_pre"]) * gh.double().cpu()).sum()
    names = list(leaf)
    ref = dict(zip(names, torch.autograd.grad(loss, [leaf[n] for n in names])))
    for name, got in (("x", g.grad_x), ("y", g.grad_y), ("w_post", g.grad_w_post), ("w_pre", g.grad_w_pre),
                      ("gate_" + str(gate), g.grad_gate)):
        if name not in ref:
            assert got is None
            continue
        want = ref[name].numpy()
        if name in ("x", "y"):  # each row by its own magnitude (row 1, of zeros, has a far larger gradient)
            mag = np.sqrt((want ** 2).mean(axis=1, keepdims=True))
        else:
            mag = np.sqrt((want ** 2).mean())
        steps = 4 * (H + 24) + (T + 16 if name in ("w_post", "w_pre", "gate_channel") else 0)
        within(got, want, 16 * mag * steps * U, name)


def test_long_rows_take_no_multiple_of_short_ones():
    """The gradient of 4 M elements in rows of 16383 against rows of 4096: 5 times is a bound on scratch
    and idle lanes, not on speed (8 with a kernel that spilled)."""
    announce("time of long rows")

    def back(T, H):
        x, kw, gr, gh = _norm_inputs(T, H, "fp32", True, True, "channel", True)
        f = e4b.block_norm(x, **kw)
        return _time(lambda: e4b.block_norm_backward(f, x, gr, gh, **kw))

    short, long = back(4096, 4096), back(1024, 16383)
    assert long < 5 * short, (long, short)


def test_odd_long_rows_forward_take_no_multiple_of_short_ones():
    """r = x + y of 74 M elements in rows of 12358 against rows of 4096: 2.4 times bounds the registers that
    single elements take (2.9 with a guard and an address for each, 1.7 without)."""
    announce("time of odd long rows, forward")

    def forth(T, H):
        x, kw, _, _ = _norm_inputs(T, H, "fp32", True, False, None, False)
        return _time(lambda: e4b.block_norm(x, **kw))

    short, long = forth(18102, 4096), forth(6000, 12358)
    assert long < 2.4 * short, (long, short)


# products in every tiling (with and without shares of k, foreign rows), forward and gradient
PRODUCTS = [(4, 90, 0, 256, 192), (1, 300, 0, 2048, 520), (3, 1900, 7, 448, 2304), (2, 3500, 9, 192, 4104), (1, 700, 0, 1024, 2048)]


def _product(E, rows, tail, inn, out, seed):
    rng = np.random.default_rng(seed)
    R = rows + tail
    off = torch.linspace(0, rows, E + 1, device=DEV).to(torch.int32) if E > 1 or tail else None
    return {"off": off, "x": dev(rng.standard_normal((R, inn)), torch.bfloat16),
            "gy": dev(rng.standard_normal((R, out)), torch.float32), "bias": dev(rng.standard_normal((E, out)), torch.float32)}


def _step(stack, s, ws=(None, None)):
    y, _ = e4b.expert_linear(stack, s["x"], s["off"], s["bias"], "gelu", workspace=ws[0])
    gx, gb = e4b.expert_linear_dgrad(stack, s["gy"], s["x"], s["off"], s["bias"], "gelu", grad_bias=True, workspace=ws[1])
    return [y, gx, gb]


@pytest.mark.parametrize("E,rows,tail,inn,out", PRODUCTS)
def test_workspace_contents_do_not_matter(E, rows, tail, inn, out):
    announce(f"workspaces of NaN, {rows} rows of {inn} -> {out}")
    stack, _ = _stack(E, out, inn, "nf4", 9)
    s = _product(E, rows, tail, inn, out, 1)
    want = _step(stack, s)
    need = (e4b.expert_linear_workspace_bytes(stack, rows + tail), e4b.expert_linear_dgrad_workspace_bytes(stack, rows + tail, True))
    ws = [torch.full((n // 4 + 1,), float("nan"), device=DEV) for n in need]
    for p, q in zip(want, _step(stack, s, ws)):
        assert torch.equal(bits(p), bits(q))


def test_larger_calls_captured_and_replayed():
    """Every tiling, the order of several passes with rows both ways, and long norms in one graph,
    replayed on new inputs with eager runs between."""
    announce("larger calls in a graph")
    stacks = [_stack(E, out, inn, "nf4", 9)[0] for E, _, _, inn, out in PRODUCTS]
    norms = [_norm_inputs(300, H, dt, True, True, gate, True) for H, dt, gate in
             ((8192, "bf16", "token"), (12288, "fp32", "channel"), (4099, "fp32", "token"))]
    ids = torch.zeros(9000, 4, dtype=torch.int32, device=DEV)
    rows_in = torch.zeros(9000, 264, dtype=torch.bfloat16, device=DEV)
    few = torch.zeros(3, 30, dtype=torch.int32, device=DEV)
    few_in = torch.zeros(3, 1032, dtype=torch.bfloat16, device=DEV)
    lg = torch.zeros(5000, 300, device=DEV)
    prods = [_product(*p, 0) for p in PRODUCTS]

    def refresh(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in [s[n] for s in prods for n in ("x", "gy", "bias")] + [rows_in, few_in, lg] + [n[0] for n in norms] + [
                v for n in norms for v in (n[2], n[3], n[1]["y"])]:
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        for t in (ids, few):
            t.copy_(torch.randint(-1, 40, t.shape, generator=g, device=DEV))

    def run():
        out = [t for stack, s in zip(stacks, prods) for t in _step(stack, s)]
        for i, x in ((ids, rows_in), (few, few_in)):
            rows, perm = e4b.moe_permute(i, 40, x)
            w = torch.full(i.shape, 0.5, device=DEV)
            out += [rows, perm.offsets, perm.pos, e4b.moe_unpermute(perm, rows, w), *e4b.moe_unpermute_backward(perm, rows, x, w)]
        idx, w = e4b.moe_route(lg, 7)
        out += [idx, w, e4b.moe_route_backward(idx, w, w, 300)]
        for x, kw, gr, gh in norms:
            f = e4b.block_norm(x, **kw)
            b = e4b.block_norm_backward(f, x, gr, gh, **kw)
            out += [f.r, f.h, b.grad_x, b.grad_y, b.grad_gate, b.grad_w_post, b.grad_w_pre]
        return out

    refresh(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for rep in range(1, 4):
        refresh(rep)
        g.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(out, want)):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), (rep, i)
