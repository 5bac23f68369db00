"""GPU parity of the operators around the expert MLP against oracle.block (float64).

Tolerances are worst-case bounds, element by element: half a step of the output's
type relative to the value (bf16 2^-8, fp32 2^-24), plus n 2^-24 times the sum of
the terms' magnitudes for an fp32 sum of n of them, plus the few steps of exp, erf,
a quotient or a square root. Copies, orders and zeros are exact.
"""

import numpy as np
import pytest
import torch

import oracle
import bit_quantized_mixture_nf4_amd as e4b
from oracle import block
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def within(got, ref, err, name):
    """|got - ref| <= err + half a step of got's type, everywhere."""
    half = HALF[got.dtype]
    g = got.detach().cpu().double().numpy()
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    bound = (err + half * np.abs(ref)) * (1 + 2.0 ** -6) + 1e-37
    bad = ~(np.abs(g - ref) <= bound)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                           f"{g[bad][0]} against {ref[bad][0]}, bound {bound[bad][0]:.3e}")


def host(t):
    return t.detach().cpu().double().numpy()


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(dtype)


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


# ---- the router ----


@pytest.mark.parametrize("T,E,k,masked", [(1, 1, 1, False), (3, 8, 2, True), (64, 60, 5, False), (257, 128, 8, True),
                                          (33, 1024, 32, True), (5, 65, 32, False), (0, 8, 2, False),
                                          (300, 256, 16, False), (70, 400, 12, True), (4097, 200, 9, True),
                                          (4100, 511, 16, True)])
def test_route_and_its_gradient(T, E, k, masked):
    announce(f"route T={T} E={E} k={k} masked={masked}")
    rng = np.random.default_rng(T + E)
    lg = rng.standard_normal((T, E)).astype(np.float32)
    if T > 1:
        lg[1] = lg[1, 0]  # ties go to the lower id
    if masked:
        lg[rng.random((T, E)) < 0.5] = -np.inf
        lg[-1] = -np.inf
    idx, w = e4b.moe_route(dev(lg, torch.float32), k)
    assert idx.shape == (T, k) and idx.dtype == torch.int32
    want = np.argsort(-lg.astype(np.float64), axis=1, kind="stable")[:, :k]
    assert np.array_equal(idx.cpu().numpy(), want)
    sel = np.take_along_axis(lg.astype(np.float64), want, axis=1)
    top = sel[:, :1]
    z = np.where(np.isneginf(sel), 0.0, np.exp(np.where(np.isneginf(sel), 0.0, sel) - np.where(np.isneginf(top), 0.0, top)))
    tot = z.sum(axis=1, keepdims=True)
    ref = np.where(tot > 0, z / np.where(tot > 0, tot, 1.0), 0.0)
    # exp's argument is off by half a step of a difference below 16, exp and the quotient by a few
    within(w, ref, ref * (k + 24) * U, "w")
    gw = rng.standard_normal((T, k)).astype(np.float32)
    gl = e4b.moe_route_backward(idx, w, dev(gw, torch.float32), E)
    wf = host(w)
    ref = block.route_backward(want, wf, gw, E)
    mag = np.zeros((T, E))
    np.put_along_axis(mag, want, wf * (np.abs(gw) + (wf * np.abs(gw)).sum(axis=1, keepdims=True)), axis=1)
    within(gl, ref, mag * (k + 4) * U, "grad_logits")


def test_route_of_unusable_logits_keeps_valid_ids():
    lg = torch.randn(6, 70, device=DEV)
    lg[0] = float("nan")
    lg[1, ::2] = -float("nan")
    lg[2, 5] = float("inf")
    lg[3] = float("inf")
    lg.view(torch.int32)[4] = -1  # the NaN of all ones
    idx, _ = e4b.moe_route(lg, 32)
    idx = idx.cpu().numpy()
    assert idx.min() >= 0 and idx.max() < 70
    for t in (0, 1, 2, 3, 5):
        assert len(set(idx[t])) == 32


def test_route_equals_the_routed_forward():
    """The routing that the expert MLP makes from the same logits, bit for bit."""
    from gpu_util import Problem
    from workloads import get_config

    pb = Problem(get_config("tiny"), seed=3, with_grad=False)
    _, idx, w, _ = e4b.moe_forward(pb.layer, pb.x_d, pb.cfg.k, logits=pb.logits_d)
    idx2, w2 = e4b.moe_route(pb.logits_d, pb.cfg.k)
    assert torch.equal(idx, idx2) and torch.equal(bits(w), bits(w2))


def test_route_backward_repeated_and_foreign_ids():
    idx = torch.tensor([[1, 1, -1], [4, 0, 2]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.5, 0.25, 0.25], [0.5, 0.25, 0.25]], device=DEV)
    g = torch.tensor([[1.0, 2.0, 4.0], [1.0, 2.0, 4.0]], device=DEV)
    ref = block.route_backward(idx.cpu().numpy(), host(w), host(g), 4)
    gl = e4b.moe_route_backward(idx, w, g, 4)
    within(gl, ref, np.full(ref.shape, 32 * U), "grad_logits")
    assert gl[1].abs().sum() == (gl[1, 0].abs() + gl[1, 2].abs())


# ---- expert order and back ----

ORDERS = [(1, 1, 1, 8, "bf16", 0.0), (5, 2, 3, 33, "bf16", 0.4), (8, 8, 128, 2048, "bf16", 0.0),
          (3, 32, 4, 64, "fp32", 0.2), (700, 3, 7, 100, "fp32", 0.1), (513, 8, 64, 2056, "bf16", 0.0),
          (9000, 4, 17, 24, "bf16", 0.1), (40, 2, 1024, 16, "fp32", 0.0), (17, 4, 5, 4097, "fp32", 1.0),
          (1030, 4, 9, 40, "bf16", 0.0), (0, 2, 4, 16, "bf16", 0.0)]


def _ids(T, k, E, drop, rng):
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < drop] = rng.choice([-1, E, E + 5, -2 ** 31, 2 ** 31 - 1])
    return ids


@pytest.mark.parametrize("T,k,E,H,dt,drop", ORDERS)
def test_permute_and_back(T, k, E, H, dt, drop):
    announce(f"permute T={T} k={k} E={E} H={H} {dt} drop={drop}")
    rng = np.random.default_rng(T * k + H)
    dtype = DT[dt]
    ids = _ids(T, k, E, drop, rng)
    x = dev(rng.standard_normal((T, H)), dtype)
    rows, perm = e4b.moe_permute(torch.from_numpy(ids).to(DEV), E, x)
    offsets, order, pos = block.expert_order(ids, E)
    for got, want in ((perm.offsets, offsets), (perm.sorted_pair, order), (perm.pos, pos)):
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want)
    live = int(offsets[-1])
    want = x[torch.from_numpy(order[:live] // k).long().to(DEV)]
    assert torch.equal(bits(rows[:live]), bits(want)) and not bits(rows[live:]).any()
    none, perm2 = e4b.moe_permute(torch.from_numpy(ids).to(DEV), E)
    assert none is None and torch.equal(perm2.pos, perm.pos)

    # pairs without an expert: whatever their rows hold stays out of every sum
    g = dev(rng.standard_normal((T * k, H)), dtype)
    gh = np.abs(host(g))
    gh[live:] = 0.0
    g[live:] = float("nan")
    ref = block.unpermute(np.nan_to_num(host(g)), offsets, pos)
    mag = block.unpermute(gh, offsets, pos)
    within(e4b.moe_permute_backward(perm, g), ref, mag * k * U, "grad_x")
    w = dev(rng.random((T, k)), torch.float32)
    ref = block.unpermute(np.nan_to_num(host(g)), offsets, pos, host(w))
    mag = block.unpermute(gh, offsets, pos, host(w))
    within(e4b.moe_unpermute(perm, g, w), ref, mag * (k + 1) * U, "y")

    gy = dev(rng.standard_normal((T, H)), dtype)
    gr, gw = e4b.moe_unpermute_backward(perm, g, gy, w)
    gr_ref, gw_ref = block.unpermute_backward(np.nan_to_num(host(g)), offsets, pos, host(w), host(gy))
    _, gw_mag = block.unpermute_backward(gh, offsets, pos, host(w), np.abs(host(gy)))
    within(gr, gr_ref, np.abs(gr_ref) * U, "grad_rows")
    assert not bits(gr[live:]).any()
    within(gw, gw_ref, gw_mag * (H + 2) * U, "grad_w")
    gr2, none = e4b.moe_unpermute_backward(perm, None, gy, w, grad_w=False)
    assert none is None and torch.equal(bits(gr2), bits(gr))
    gr3, _ = e4b.moe_unpermute_backward(perm, g, gy)
    ref = block.unpermute_backward(np.nan_to_num(host(g)), offsets, pos, None, host(gy))[0]
    assert np.array_equal(host(gr3), ref)  # weights of 1: copies


def test_permute_many_pairs_of_one_expert():
    """Several passes over the ids (more than 32768 pairs), nearly all of one expert."""
    announce("permute 70001 pairs, one hot expert")
    ids = np.full((70001, 1), 5, dtype=np.int32)
    ids[::1000] = 2
    ids[-1] = 6
    _, perm = e4b.moe_permute(torch.from_numpy(ids).to(DEV), 7)
    offsets, order, pos = block.expert_order(ids, 7)
    for got, want in ((perm.offsets, offsets), (perm.sorted_pair, order), (perm.pos, pos)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_unpermute_ignores_places_outside_the_rows():
    announce("unpermute with places outside the rows")
    offsets = torch.tensor([0, 2, 3], dtype=torch.int32, device=DEV)
    pos = torch.tensor([[0, -1], [2, 2 ** 31 - 1], [3, 1]], dtype=torch.int32, device=DEV)
    perm = e4b.Permutation(offsets, torch.zeros(6, dtype=torch.int32, device=DEV), pos)
    rows = torch.arange(6 * 16, device=DEV, dtype=torch.float32).view(6, 16)
    y = e4b.moe_unpermute(perm, rows)
    assert torch.equal(y, torch.stack([rows[0], rows[2], rows[1]]))
    # offsets beyond the rows do not make more of them
    far = e4b.Permutation(torch.tensor([0, 2, 2 ** 31 - 1], dtype=torch.int32, device=DEV), perm.sorted_pair, pos)
    assert torch.equal(e4b.moe_unpermute(far, rows), torch.stack([rows[0], rows[2], rows[3] + rows[1]]))
    gr, gw = e4b.moe_unpermute_backward(perm, rows, torch.ones(3, 16, device=DEV))
    assert torch.equal(gw != 0, torch.tensor([[True, False], [True, False], [False, True]], device=DEV))
    assert not gr[3].any() and gr[:3].eq(1).all()


# ---- products with a stored stack ----


def _stack(E, out, inn, codebook, seed):
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((E, out, inn)) * 0.05).astype(np.float32)
    view = oracle.bf16_bits_to_f32(oracle.bf16_rne_bits(oracle.stored_weights(w, codebook).reshape(E * out, inn)))
    return e4b.quantize(torch.from_numpy(w).to(DEV), codebook), view.reshape(E, out, inn).astype(np.float64)


def _counts(E, rows, rng, empty=()):
    c = np.bincount(rng.integers(0, E, rows), minlength=E)
    for e in empty:
        c[(e + 1) % E] += c[e]
        c[e] = 0
    return c


# codebook, E, rows, tail, in, out, act, bias, residual, y
LINEARS = [
    ("nf4", 1, 1, 0, 64, 64, "none", False, False, "bf16"),
    ("bf16", 1, 8, 0, 2048, 60, "none", True, False, "fp32"),
    ("nf4", 1, 300, 0, 320, 200, "silu", True, True, "bf16"),
    ("fp4", 6, 137, 5, 192, 320, "gelu", True, False, "bf16"),
    ("mxfp4", 5, 64, 0, 448, 129, "gelu_tanh", True, True, "fp32"),
    ("int8", 4, 515, 1, 128, 72, "relu", False, True, "bf16"),
    ("fp8", 3, 33, 40, 256, 1000, "silu", True, False, "fp32"),
    ("nf4", 128, 64, 0, 512, 256, "silu", True, False, "bf16"),
    ("nf4", 2, 1000, 0, 1024, 512, "gelu", True, True, "bf16"),
    ("bf16", 7, 900, 3, 64, 17, "none", True, True, "bf16"),
    ("nf4", 1024, 50, 2, 64, 8, "none", True, False, "bf16"),
    ("fp8", 1, 257, 0, 576, 1, "relu", True, False, "fp32"),
    ("nf4", 3, 0, 0, 64, 64, "silu", True, False, "bf16"),
    ("mxfp4", 4, 0, 9, 64, 64, "none", True, False, "bf16"),
    ("nf4", 1, 17, 0, 4096, 96, "none", True, True, "bf16"),
    ("mxfp4", 9, 40, 0, 2112, 300, "silu", True, False, "bf16"),
    ("bf16", 2, 1500, 0, 256, 776, "silu", True, True, "bf16"),
    ("int8", 8, 48, 0, 1024, 256, "none", False, False, "fp32"),
    # 128-row tiles, cut along k and not
    ("nf4", 1, 700, 0, 1024, 2048, "gelu", True, True, "bf16"),
    ("fp4", 1, 600, 3, 1088, 2049, "silu", True, False, "fp32"),
    ("bf16", 3, 500, 9, 1024, 1000, "relu", True, True, "bf16"),
    ("mxfp4", 2, 1030, 0, 512, 1100, "gelu_tanh", False, False, "bf16"),
    ("int8", 1, 1300, 0, 320, 1024, "none", True, False, "bf16"),
    ("nf4", 5, 3000, 2, 64, 1100, "silu", True, False, "bf16"),
    ("fp8", 1, 3001, 0, 128, 1001, "none", True, True, "fp32"),
    ("nf4", 1, 700, 0, 2048, 2048, "gelu", True, True, "bf16"),
    ("fp4", 1, 650, 3, 2112, 2049, "silu", True, False, "fp32"),
    ("mxfp4", 2, 1500, 0, 1024, 1500, "gelu_tanh", False, False, "bf16"),
    ("bf16", 3, 500, 9, 1024, 1100, "relu", True, True, "bf16"),
    ("int8", 1, 1300, 0, 448, 1024, "none", True, False, "bf16"),
    ("fp8", 1, 3001, 0, 192, 1001, "none", True, True, "fp32"),
    # 256-row tiles, forward and gradient
    ("nf4", 2, 2500, 7, 128, 4096, "silu", True, True, "bf16"),
    ("bf16", 1, 2049, 0, 64, 4360, "gelu", True, False, "fp32"),
    ("fp8", 3, 2600, 0, 128, 3968, "none", False, True, "bf16"),
    ("mxfp4", 2, 2300, 1, 192, 4224, "relu", True, False, "bf16"),
    ("nf4", 2, 2500, 5, 4096, 128, "none", True, False, "bf16"),
    ("int8", 1, 2200, 0, 4224, 192, "gelu_tanh", True, False, "bf16"),
    ("mxfp4", 3, 2600, 0, 3968, 64, "none", False, False, "fp32"),
    ("bf16", 2, 2304, 0, 4096, 128, "silu", True, False, "bf16"),
    ("nf4", 2, 3500, 4, 192, 4104, "gelu", True, True, "bf16"),
    # 256 x 128 tiles, forward and gradient
    ("nf4", 1, 2100, 0, 448, 2300, "gelu", True, True, "bf16"),
    ("bf16", 1, 2100, 0, 128, 2304, "none", True, True, "fp32"),
    ("fp8", 3, 1900, 7, 128, 2322, "silu", True, False, "bf16"),
    ("int8", 1, 1793, 1, 192, 2304, "relu", False, True, "bf16"),
    ("fp4", 1, 2100, 3, 512, 2312, "gelu_tanh", True, False, "bf16"),
    ("mxfp4", 2, 3000, 0, 704, 4101, "silu", True, False, "fp32"),
    ("bf16", 1, 2100, 0, 2304, 192, "silu", True, False, "bf16"),
    ("nf4", 2, 1900, 3, 2304, 100, "gelu", True, True, "bf16"),
    ("mxfp4", 3, 1900, 1, 2112, 64, "none", True, False, "bf16"),
    ("int8", 1, 2100, 0, 2176, 60, "relu", True, False, "fp32"),
]


def _act_errors(act, z, z_err):
    """(error of act(z), of act'(z)) for an error of z: |act'| <= 1.2, |act''| <= 1.1, and a few
    steps of exp, erf and the quotient (relative to 1 + |z|, which bounds every term)."""
    if act == "none":
        return z_err, 0 * z
    if act == "relu":  # a sign that z's error can flip
        return z_err, (np.abs(z) <= z_err).astype(np.float64)
    return 1.2 * z_err + 16 * U * (np.abs(z) + z * z * (np.abs(z) < 4)), 1.1 * z_err + 32 * U * (1 + np.abs(z)) ** 2


@pytest.mark.parametrize("cb,E,rows,tail,inn,out,act,with_bias,with_res,yt", LINEARS)
def test_expert_linear_and_its_gradient(cb, E, rows, tail, inn, out, act, with_bias, with_res, yt):
    announce(f"linear {cb} E={E} rows={rows}+{tail} {inn}->{out} {act} bias={with_bias} res={with_res} {yt}")
    rng = np.random.default_rng(rows + out)
    stack, w = _stack(E, out, inn, cb, out + inn)
    R = rows + tail
    counts = _counts(E, rows, rng, empty=(0,) if E > 2 else ())
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    off_d = torch.from_numpy(offsets).to(DEV) if E > 1 or tail else None
    x = dev(rng.standard_normal((R, inn)), torch.bfloat16)
    x[rows:] = float("nan")  # rows of no expert
    bias = dev(rng.standard_normal((E, out)) * 0.1, torch.float32) if with_bias else None
    res = dev(rng.standard_normal((R, out)), torch.bfloat16) if with_res else None
    xh = np.nan_to_num(host(x))
    bh = None if bias is None else host(bias)
    rh = None if res is None else host(res)
    y, pre = e4b.expert_linear(stack, x, offsets=off_d, bias=bias, act=act, residual=res, out_dtype=DT[yt], save=True)
    y_ref, z_ref = block.expert_linear(xh, w, offsets, bh, act, rh)
    zmag = block.expert_linear(np.abs(xh), np.abs(w), offsets, None if bh is None else np.abs(bh))[1]
    z_err = (inn + 4) * U * zmag
    within(pre, z_ref, z_err, "pre")
    live = (np.arange(R) < rows)[:, None]
    a_err, da_err = _act_errors(act, z_ref, z_err)
    y_err = a_err + 2 * U * (np.abs(y_ref) + (0 if rh is None else np.abs(rh)))
    within(y, y_ref, y_err * live, "y")
    y2, none = e4b.expert_linear(stack, x, offsets=off_d, bias=bias, act=act, residual=res, out_dtype=DT[yt])
    assert none is None and torch.equal(bits(y2), bits(y))

    gy = dev(rng.standard_normal((R, out)), DT[yt])
    gy[rows:] = float("inf")
    gyh = np.where(live, host(gy), 0.0)
    gx, gb = e4b.expert_linear_dgrad(stack, gy, offsets=off_d, act=act, pre=pre, grad_bias=True)
    gx_ref, gb_ref = block.expert_linear_dgrad(gyh, z_ref, w, offsets, act)
    dz = np.abs(gyh * block.activation(act, z_ref)[1])
    dz_err = np.abs(gyh) * da_err + 2 * U * dz
    # dz is rounded to bf16 as the product's operand, then out products are summed
    back = lambda v: block.expert_linear_dgrad(v, z_ref, np.abs(w), offsets)[0]  # noqa: E731
    within(gx, gx_ref, back(dz_err * (1 + 2.0 ** -8) + dz * (2.0 ** -8 + (out + 4) * U)), "grad_x")
    col = lambda v: block.expert_linear_dgrad(v, z_ref, w, offsets)[1]  # noqa: E731
    within(gb, gb_ref, col(dz_err + dz * (rows + 8) * U), "grad_bias")
    if act != "none":  # without the kept pre-activation: the same bits
        gx2, gb2 = e4b.expert_linear_dgrad(stack, gy, x=x, offsets=off_d, bias=bias, act=act, grad_bias=True)
        assert torch.equal(bits(gx2), bits(gx)) and torch.equal(bits(gb2), bits(gb))
    else:
        gx2, none = e4b.expert_linear_dgrad(stack, gy, offsets=off_d)
        assert none is None and torch.equal(bits(gx2), bits(gx))


@pytest.mark.parametrize("rows", [1, 2, 9, 16, 17, 31, 33, 64, 65, 127, 128, 129, 255, 256, 257, 511])
def test_expert_linear_row_counts(rows):
    """One dense stack over every count at which a tile of rows begins or ends; each row's result is
    the one it has alone in the batch."""
    announce(f"linear rows={rows}")
    rng = np.random.default_rng(rows)
    stack, w = _stack(1, 160, 256, "nf4", 1)
    x = dev(rng.standard_normal((rows, 256)), torch.bfloat16)
    y, _ = e4b.expert_linear(stack, x, out_dtype=torch.float32)
    ref, _ = block.expert_linear(host(x), w)
    mag, _ = block.expert_linear(np.abs(host(x)), np.abs(w))
    within(y, ref, mag * 260 * U, "y")


@pytest.mark.parametrize("lists", [[0, 40, 10, 64, 64], [0, 16, 32, 48, 9999], [-7, -1, 64, 64, 64], [64, 0, 64, 0, 64]])
def test_expert_linear_clamps_bad_offsets(lists):
    """Offsets that do not ascend or leave the rows stay inside the buffers."""
    announce(f"linear offsets {lists}")
    stack, _ = _stack(4, 96, 128, "nf4", 2)
    x = torch.randn(64, 128, device=DEV).to(torch.bfloat16)
    off = torch.tensor(lists, dtype=torch.int32, device=DEV)
    big = torch.full((96, 96), 7.0, device=DEV)  # the output with guard rows behind it
    e4b.expert_linear(stack, x, offsets=off, out_dtype=torch.float32, out=big[:64])
    gx, gb = e4b.expert_linear_dgrad(stack, big[:64].contiguous(), offsets=off, grad_bias=True)
    torch.cuda.synchronize()
    assert big[64:].eq(7.0).all() and gx.shape == (64, 128) and gb.shape == (4, 96)


# ---- the norms ----

NORMS = [
    (1, 8, "bf16", True, True, None, True), (3, 33, "bf16", True, True, "token", True),
    (17, 100, "fp32", True, False, "channel", True), (64, 512, "bf16", True, True, "channel", True),
    (5, 1000, "bf16", False, False, None, True), (2, 1, "fp32", True, True, "token", True),
    (33, 2048, "bf16", True, True, "token", True), (70, 2056, "fp32", True, True, "channel", True),
    (9, 4097, "fp32", True, True, "token", True), (700, 264, "bf16", True, False, "token", False),
    (4200, 64, "fp32", True, True, "channel", True), (2, 16384, "bf16", True, True, "channel", True),
    (3, 16383, "fp32", True, True, None, True), (6, 8191, "bf16", True, True, "channel", True),
    (513, 1024, "bf16", True, True, None, False), (11, 4096, "bf16", True, True, "token", True),
    (300, 8192, "bf16", True, False, None, True), (0, 64, "bf16", True, True, "channel", True),
    (0, 64, "fp32", True, True, "token", True),
]


def _norm_inputs(T, H, dt, has_y, post, gate, pre):
    rng = np.random.default_rng(T + H)
    x = dev(rng.standard_normal((T, H)), DT[dt])
    if T > 2:
        x[1] = 0  # a row of zeros
    kw = {}
    if has_y:
        kw["y"] = dev(rng.standard_normal((T, H)), torch.bfloat16)
        if T > 2:
            kw["y"][1] = 0
    if post:
        kw["w_post"] = dev(1 + 0.1 * rng.standard_normal(H), torch.float32)
    if gate:
        kw["gate_" + gate] = dev(rng.standard_normal(T if gate == "token" else H), torch.float32)
    if pre:
        kw["w_pre"] = dev(1 + 0.1 * rng.standard_normal(H), torch.float32)
    gr = dev(rng.standard_normal((T, H)), DT[dt])
    gh = dev(rng.standard_normal((T, H)), torch.bfloat16) if pre else None
    return x, kw, gr, gh


@pytest.mark.parametrize("E,rows,inn,out", [(1, 20, 128, 96), (1, 300, 2048, 520), (3, 900, 1024, 1001), (1, 2100, 448, 2300),
                                            (2, 3500, 192, 4104)])
def test_residual_added_in_place(E, rows, inn, out):
    """y may be written over the residual, in every tiling; over the rows of x it may not."""
    announce(f"in place E={E} rows={rows} {inn} -> {out}")
    rng = np.random.default_rng(rows)
    stack, _ = _stack(E, out, inn, "nf4", 3)
    x = dev(rng.standard_normal((rows, inn)), torch.bfloat16)
    res = dev(rng.standard_normal((rows, out)), torch.bfloat16)
    off = torch.linspace(0, rows - 5, E + 1, device=DEV).to(torch.int32) if E > 1 else None
    want = e4b.expert_linear(stack, x, off, act="silu", residual=res)[0]
    got = e4b.expert_linear(stack, x, off, act="silu", residual=res, out=res)[0]
    assert got.data_ptr() == res.data_ptr() and torch.equal(bits(got), bits(want))
    square, _ = _stack(1, inn, inn, "nf4", 4)
    with pytest.raises(ValueError, match="overlap"):
        e4b.expert_linear(square, x, out=x)


@pytest.mark.parametrize("T,H,dt,has_y,post,gate,pre", NORMS)
def test_block_norm_and_its_gradient(T, H, dt, has_y, post, gate, pre):
    announce(f"norm T={T} H={H} {dt} y={has_y} post={post} gate={gate} pre={pre}")
    x, kw, gr, gh = _norm_inputs(T, H, dt, has_y, post, gate, pre)
    hk = {n: host(v) for n, v in kw.items()}
    scale = float(np.float32(0.7)) if has_y else 1.0
    f = e4b.block_norm(x, scale=scale, **kw)
    xh = host(x)
    r_ref, h_ref = block.block_norm(xh, scale=scale, **hk)
    # a mean of H squares, its root and the products after it; r loses half a step of its terms
    n = H + 16
    gate_v = block._gate(hk.get("gate_token"), hk.get("gate_channel"))
    u = np.zeros_like(xh)
    if has_y:
        u = hk["y"] * (block._rstd(hk["y"], 1e-6) * hk["w_post"] if post else 1.0)
        r_err = n * U * np.abs(scale * gate_v * u) + 2 * U * (np.abs(xh) + np.abs(scale * gate_v * u))
        within(f.r, r_ref, r_err, "r")
    else:
        assert f.r is x
        r_err = 0.0 * xh
    M = np.abs(xh) + np.abs(scale * gate_v * u)  # what r's error is relative to
    rs = block._rstd(r_ref, 1e-6) if T else np.zeros((0, 1))
    if pre:
        # r's own error also moves the statistic: relative to the row's root mean square
        rel = np.sqrt((r_err ** 2).mean(axis=1, keepdims=True)) * rs if T else np.zeros((0, 1))
        h_err = np.abs(hk["w_pre"]) * rs * (r_err + np.abs(r_ref) * (n * U + rel))
        within(f.h, h_ref, h_err, "h")
    else:
        assert f.h is None

    g = e4b.block_norm_backward(f, x, gr, gh, scale=scale, **kw)
    grh, ghh = host(gr), None if gh is None else host(gh)
    ref = block.block_norm_backward(xh, grh, ghh, scale=scale, **hk)
    # magnitudes of the terms of every gradient, with M in place of |r| where r may cancel; each is
    # off by at most the steps of its statistics and sums: c of them
    c = 4 * (H + 24) * U
    a = lambda v: np.abs(v)  # noqa: E731
    drm = a(grh)
    if pre:
        cm, nm = a(ghh * hk["w_pre"]), M * rs
        drm = drm + rs * (cm + nm * (cm * nm).mean(axis=1, keepdims=True)) if T else drm
        within(g.grad_w_pre, ref["grad_w_pre"], (a(ghh) * nm).sum(axis=0) * (c + (T + 16) * U), "grad_w_pre")
    else:
        assert g.grad_w_pre is None
    within(g.grad_x, ref["grad_x"], c * drm, "grad_x")
    if not has_y:
        assert g.grad_y is None and g.grad_gate is None and g.grad_w_post is None
        return
    if gate:
        gm = scale * drm * a(u)
        within(g.grad_gate, ref["grad_gate"], gm.sum(axis=1) * c if gate == "token" else gm.sum(axis=0) * (c + (T + 16) * U),
               "grad_gate")
    dum = scale * a(gate_v) * drm
    if post:
        ry = block._rstd(hk["y"], 1e-6) if T else np.zeros((0, 1))
        mm = a(hk["y"]) * ry
        within(g.grad_w_post, ref["grad_w_post"], (dum * mm).sum(axis=0) * (c + (T + 16) * U), "grad_w_post")
        bm = dum * a(hk["w_post"])
        dum = ry * (bm + mm * (bm * mm).mean(axis=1, keepdims=True)) if T else dum
    within(g.grad_y, ref["grad_y"], c * dum, "grad_y")
    # without the column gradients the others keep their bits
    g2 = e4b.block_norm_backward(f, x, gr, gh, scale=scale, weight_grads=False, **kw)
    assert g2.grad_w_pre is None and g2.grad_w_post is None
    assert torch.equal(bits(g2.grad_x), bits(g.grad_x)) and torch.equal(bits(g2.grad_y), bits(g.grad_y))


def test_block_norm_without_grad_r():
    x, kw, _, gh = _norm_inputs(7, 136, "bf16", True, True, "token", True)
    f = e4b.block_norm(x, **kw)
    a = e4b.block_norm_backward(f, x, None, gh, **kw)
    b = e4b.block_norm_backward(f, x, torch.zeros_like(x), gh, **kw)
    for name in ("grad_x", "grad_y", "grad_gate", "grad_w_post", "grad_w_pre"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_refusals_on_the_device():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    ones = torch.ones(64, device=DEV)
    ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    stack, _ = _stack(2, 64, 64, "nf4", 0)
    bad = [
        lambda: e4b.moe_route(torch.zeros(4, 8, device=DEV), 9),
        lambda: e4b.moe_route(torch.zeros(4, 8, device=DEV).t(), 2),
        lambda: e4b.moe_permute(ids, 0, x),
        lambda: e4b.moe_permute(ids, 8, x[:3]),
        lambda: e4b.moe_permute(ids, 8, x[:, ::2]),
        lambda: e4b.moe_permute(ids.view(-1), 8, x),
        lambda: e4b.moe_unpermute(e4b.moe_permute(ids, 8)[1], x),
        lambda: e4b.expert_linear(stack, x),  # two experts, no offsets
        lambda: e4b.expert_linear(stack, x, offsets=ids.view(-1)[:2]),
        lambda: e4b.expert_linear(stack, x, offsets=ids.view(-1)[:3], act="tanh"),
        lambda: e4b.expert_linear(stack, x, offsets=ids.view(-1)[:3], bias=ones),
        lambda: e4b.expert_linear(stack, x, offsets=ids.view(-1)[:3], out_dtype=torch.float16),
        lambda: e4b.expert_linear_dgrad(stack, x, offsets=ids.view(-1)[:3], workspace=torch.empty(8, device=DEV)),
        lambda: e4b.expert_linear_dgrad(stack, x, offsets=ids.view(-1)[:3], act="silu"),
        lambda: e4b.block_norm(x),
        lambda: e4b.block_norm(x, w_post=ones),
        lambda: e4b.block_norm(x, y=x, gate_token=ones),
        lambda: e4b.block_norm(x, y=x, gate_token=ones[:4], gate_channel=ones),
        lambda: e4b.block_norm(x, w_pre=ones, eps=0.0),
        lambda: e4b.block_norm_backward(e4b.block_norm(x, w_pre=ones), x, x, w_pre=ones),
        lambda: e4b.block_norm_backward(e4b.block_norm(x, y=x), x, y=x),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


# ---- together ----


class Block:
    """Norm, router, experts with biases and another activation, and the way back, as a user joins them."""

    def __init__(self, T=150, H=256, I=192, E=8, k=2, seed=0):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.router, self.router_w = _stack(1, E, H, "bf16", 11)
        self.up, self.up_w = _stack(E, I, H, "nf4", 12)
        self.dn, self.dn_w = _stack(E, H, I, "nf4", 13)
        f = lambda *s: dev(rng.standard_normal(s) * 0.1, torch.float32)  # noqa: E731
        self.b_up, self.b_dn = f(E, I), f(E, H)
        self.w_in, self.w_post = 1 + f(H), 1 + f(H)
        self.x = dev(rng.standard_normal((T, H)), torch.bfloat16)
        self.gate = dev(rng.random(T), torch.float32)
        self.grad = dev(rng.standard_normal((T, H)), torch.bfloat16)

    def forward(self):
        s = self
        s.n0 = e4b.block_norm(s.x, w_pre=s.w_in)
        s.logits, _ = e4b.expert_linear(s.router, s.n0.h, out_dtype=torch.float32)
        s.idx, s.w = e4b.moe_route(s.logits, s.k)
        rows, s.perm = e4b.moe_permute(s.idx, s.E, s.n0.h)
        a, s.pre = e4b.expert_linear(s.up, rows, offsets=s.perm.offsets, bias=s.b_up, act="gelu", save=True)
        s.o, _ = e4b.expert_linear(s.dn, a, offsets=s.perm.offsets, bias=s.b_dn)
        s.y = e4b.moe_unpermute(s.perm, s.o, s.w)
        s.n1 = e4b.block_norm(s.x, y=s.y, w_post=s.w_post, gate_token=s.gate, scale=0.5)
        return s.n1.r

    def backward(self):
        s = self
        g1 = e4b.block_norm_backward(s.n1, s.x, s.grad, y=s.y, w_post=s.w_post, gate_token=s.gate, scale=0.5)
        go, gw = e4b.moe_unpermute_backward(s.perm, s.o, g1.grad_y, s.w)
        ga, gb_dn = e4b.expert_linear_dgrad(s.dn, go, offsets=s.perm.offsets, grad_bias=True)
        grows, gb_up = e4b.expert_linear_dgrad(s.up, ga, offsets=s.perm.offsets, act="gelu", pre=s.pre, grad_bias=True)
        gh = e4b.moe_permute_backward(s.perm, grows)
        gl = e4b.moe_route_backward(s.idx, s.w, gw, s.E)
        gh2, _ = e4b.expert_linear_dgrad(s.router, gl)
        g0 = e4b.block_norm_backward(s.n0, s.x, g1.grad_x, gh + gh2, w_pre=s.w_in)
        return {"grad_x": g0.grad_x, "grad_w_in": g0.grad_w_pre, "grad_w_post": g1.grad_w_post, "grad_gate": g1.grad_gate,
                "grad_b_up": gb_up, "grad_b_dn": gb_dn, "grad_logits": gl}

    def reference(self):
        s, off, pos, idx = self, self.perm.offsets.cpu().numpy(), self.perm.pos.cpu().numpy(), self.idx.cpu().numpy()
        x, w_in, w_post, gate = host(s.x), host(s.w_in), host(s.w_post), host(s.gate)
        _, h = block.block_norm(x, w_pre=w_in)
        lg, _ = block.expert_linear(h, s.router_w)
        sel = np.take_along_axis(lg, idx.astype(np.int64), axis=1)
        w = np.exp(sel - sel.max(axis=1, keepdims=True))
        w /= w.sum(axis=1, keepdims=True)
        rows = block.permute(h, idx, s.E)
        a, z = block.expert_linear(rows, s.up_w, off, host(s.b_up), "gelu")
        o, _ = block.expert_linear(a, s.dn_w, off, host(s.b_dn))
        y = block.unpermute(o, off, pos, w)
        r, _ = block.block_norm(x, y, w_post, gate_token=gate, scale=0.5)
        g1 = block.block_norm_backward(x, host(s.grad), None, y, w_post, gate_token=gate, scale=0.5)
        go, gw = block.unpermute_backward(o, off, pos, w, g1["grad_y"])
        ga, gb_dn = _dgrad_none(go, s.dn_w, off)
        grows, gb_up = block.expert_linear_dgrad(ga, z, s.up_w, off, "gelu")
        gl = block.route_backward(idx, w, gw, s.E)
        gh = block.unpermute(grows, off, pos) + gl @ s.router_w[0]
        g0 = block.block_norm_backward(x, g1["grad_x"], gh, w_pre=w_in)
        return r, {"grad_x": g0["grad_x"], "grad_w_in": g0["grad_w_pre"], "grad_w_post": g1["grad_w_post"],
                   "grad_gate": g1["grad_gate"], "grad_b_up": gb_up, "grad_b_dn": gb_dn, "grad_logits": gl}


def _dgrad_none(gy, w, off):
    return block.expert_linear_dgrad(gy, np.zeros_like(gy), w, off)


def test_a_block_of_them_forward_and_backward():
    """The chain against the same chain in 64 bits. Each tensor between two calls is rounded to bf16
    once: 5 on the way to r, 7 more on the way back, each at most 2^-8 of its value; 12 2^-8 of the
    largest value bounds what they add up to where no sum cancels."""
    announce("a block forward and backward")
    b = Block()
    r = b.forward()
    grads = b.backward()
    r_ref, ref = b.reference()
    for name, got, want in [("r", r, r_ref)] + [(n, grads[n], ref[n]) for n in ref]:
        err = np.max(np.abs(host(got) - want))
        assert err <= 12 * 2.0 ** -8 * np.max(np.abs(want)), (name, err, np.max(np.abs(want)))


def test_two_runs_are_the_same():
    b = Block(T=333, seed=1)
    one = [b.forward()] + list(b.backward().values())
    two = [b.forward()] + list(b.backward().values())
    for p, q in zip(one, two):
        assert torch.equal(bits(p), bits(q))


def test_on_another_stream():
    b = Block(T=90, seed=2)
    want = [b.forward()] + list(b.backward().values())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [b.forward()] + list(b.backward().values())
    torch.cuda.current_stream().wait_stream(s)
    for p, q in zip(want, got):
        assert torch.equal(bits(p), bits(q))


def test_captured_and_replayed():
    """One graph of the whole block, replayed on new inputs with eager runs between the replays."""
    announce("block in a graph")
    b, eager = Block(T=120, seed=3), Block(T=120, seed=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.forward()
        b.backward()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [b.forward()] + list(b.backward().values())
    for rep in range(4):
        x = torch.randn(120, 256, device=DEV).to(torch.bfloat16)
        b.x.copy_(x)
        eager.x.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        want = [eager.forward()] + list(eager.backward().values())
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(out, want)):
            assert torch.equal(bits(p), bits(q)), (rep, i)
