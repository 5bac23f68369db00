"""GPU tests of the microscaled 4-bit operators at their edges: factors that leave fp32's range where the result
does not, parts of longer rows."""

import numpy as np
import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
from oracle import mx
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def host(t):
    return t.detach().cpu().double().numpy()


def silu_parts(g):
    """(derivative of silu, the magnitudes of its terms, silu) in 64 bits, with their limits at infinite g."""
    with np.errstate(invalid="ignore"):
        e = np.exp(-np.abs(g))
        s, r = np.where(g < 0, e, 1.0) / (1 + e), np.where(g < 0, 1.0, e) / (1 + e)
        gr = np.where(r == 0, 0.0, g * r)
        slope = np.where(s == 0, 0.0, s * (1 + gr))
        terms = np.where(s == 0, 0.0, s * (1 + np.abs(gr)))
        return slope, terms, np.where(s == 0, -0.0, g * s)


def check_gated_gradient(g, u, ga, dtype):
    """One value of [g | u] and of the gradient a block, so that none has a neighbour's company. Each factor is
    off by a few steps (24 U of the terms in all), the result by half a step of its type, or of its least subnormal one."""
    x = torch.zeros(g.size, 128, device=DEV)
    grad = torch.zeros(g.size, 64, device=DEV)
    x[:, 0], x[:, 64], grad[:, 0] = (torch.from_numpy(v.astype(np.float32)).to(DEV) for v in (g, u, ga))
    x, grad = x.to(dtype), grad.to(dtype)
    got = host(e4b.mx4_rows_backward(x, grad))
    g, u, ga = host(x)[:, 0], host(x)[:, 64], host(grad)[:, 0]
    slope, terms, silu = silu_parts(g)
    info = torch.finfo(dtype)
    with np.errstate(invalid="ignore", over="ignore"):
        want = np.stack([ga * u * slope, ga * silu], axis=1)
        size = np.stack([np.abs(ga * u) * terms, np.abs(ga * silu)], axis=1)
        err = 24 * U * size + HALF[dtype] * np.abs(want) * (1 + 2.0 ** -6) + info.smallest_normal * info.eps
        have = got[:, [0, 64]]
        # what lies beyond the type's largest value by more than its own error is infinite
        far = np.isinf(want) | (np.abs(want) - err > info.max)
        near = ~far & (np.abs(want) + err >= info.max)
        ok = np.where(far, have == np.sign(want) * np.inf, np.abs(have - want) <= err)
        ok |= np.isnan(want) & np.isnan(have)
        ok |= near & (np.abs(have) >= info.max * (1 - HALF[dtype]))
    bad = np.argwhere(~ok)
    assert not bad.size, (f"{len(bad)} of {ok.size} off, first g={g[bad[0, 0]]} u={u[bad[0, 0]]} grad={ga[bad[0, 0]]}: "
                          f"{have[tuple(bad[0])]} against {want[tuple(bad[0])]}")
    assert not np.delete(got, [0, 64], axis=1).any()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_gated_gradient_of_the_largest_gates(dt):
    """Where silu is the identity, or constant, to the last gate that a type holds, and at infinite ones; a NaN is
    passed on."""
    announce(f"gated gradient of the largest gates {dt}")
    g = np.array([80, 88, 100, 104, 127, 128, 129, 1e4, 1e30, 2.3e38, 2.35e38, 2.37e38, 2.4e38, 3.3e38, np.inf, np.nan,
                  -1e30, -2.4e38, -3.3e38, -np.inf])
    u, ga = np.array([1.0, -7.0, 0.375, 0.0, 1e-20, 3e20]), np.array([0.75, -2.0, 1e-30, 0.0])
    g, u, ga = (v.reshape(-1) for v in np.meshgrid(g, u, ga, indexing="ij"))
    check_gated_gradient(g, u, ga, DT[dt])


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_gated_gradient_of_factors_that_leave_the_range(dt):
    """grad u, or silu of a least gate, beyond fp32's range or with few bits left in it, and the result within it."""
    announce(f"gated gradient of factors that leave the range {dt}")
    g = np.array([-90, -64.5, -64, -63.5, -50, -40, -30, -10, -1.2784645, -1, -0.25, -1e-30, -2e-31, -1e-36, -1e-39, -1e-42,
                  0.0, -0.0, 1.4e-45, 7e-45, 1e-41, 1e-38, 1e-20, 0.5, 1, 20, 60, 90, 2e38])
    far = np.array([0.0, 1e-45, 1e-42, 3e-39, 1e-37, 1e-30, 1e-20, 1e-15, 1.0, 1e15, 1e20, 1e30, 3e38])
    g, u, ga = (v.reshape(-1) for v in np.meshgrid(g, np.concatenate([far, -far]), far, indexing="ij"))
    check_gated_gradient(g, u, ga, DT[dt])


def test_gated_gradient_next_to_such_factors():
    """The values beside one that takes the way in 64 bits keep their bits."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(64, 512, device=DEV, generator=gen)
    grad = torch.randn(64, 256, device=DEV, generator=gen)
    want = e4b.mx4_rows_backward(x, grad)
    at = torch.arange(64, device=DEV)
    x2, grad2 = x.clone(), grad.clone()
    x2[at, 3 * at], x2[at, 256 + 3 * at], grad2[at, 3 * at] = -40.0, 1e20, 1e20
    got = e4b.mx4_rows_backward(x2, grad2)
    assert got[at, 3 * at].isfinite().all() and got[at, 3 * at].lt(-1e23).all()
    other = torch.ones_like(got, dtype=torch.bool)
    other[at, 3 * at] = other[at, 256 + 3 * at] = False
    assert torch.equal(got[other].view(torch.int32), want[other].view(torch.int32))


@pytest.mark.parametrize("K", [64, 192, 512])
def test_parts_of_longer_rows(K):
    """Rows from any one on, with the bits of a copy."""
    announce(f"mx rows in parts K={K}")
    gen = torch.Generator(device=DEV).manual_seed(K)
    q = e4b.mx4_rows(torch.randn(120, K, device=DEV, generator=gen))
    stack = e4b.quantize(torch.randn(1, 48, K, device=DEV, generator=gen), "mxfp4")
    for first, n in ((1, 7), (2, 100), (5, 64), (8, 1)):
        part = e4b.MxRows(q.codes[first:first + n], q.scales[first:first + n])
        copy = e4b.MxRows(part.codes.clone(), part.scales.clone())
        assert torch.equal(e4b.mx4_values(part).view(torch.int16), e4b.mx4_values(copy).view(torch.int16))
        y, want = e4b.mx_linear(stack, part)[0], e4b.mx_linear(stack, copy)[0]
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
        ids = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
        y = e4b.mx_linear(stack, part, perm=e4b.moe_permute(ids, 1)[1])[0]
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_values_of_every_code_and_scale(dt):
    """All 16 codes under all 256 scales; 255 is NaN whatever the codes are."""
    announce(f"mx values of every code and scale {dt}")
    codes = np.resize(np.arange(256, dtype=np.uint8), (256, 32))  # a row holds 64 values, two blocks
    codes = np.stack([np.roll(codes[0], s) for s in range(256)])
    codes[:, :16] = (np.arange(16) * 17)[None, :] ^ (np.arange(256) % 2 * 15)[:, None]
    scales = np.stack([np.arange(256), np.arange(256)[::-1]], axis=1).astype(np.uint8)
    q = e4b.MxRows(torch.from_numpy(codes).to(DEV), torch.from_numpy(np.ascontiguousarray(scales)).to(DEV))
    with np.errstate(over="ignore"):  # 2 to 6 times 2^127, and 4 and 6 times 2^126, are infinite in either type
        want = mx.mx_rows_values(codes, scales).astype(np.float32)
    got = host(e4b.mx4_values(q, DT[dt]))
    bad = np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))
    assert not bad.size, (f"{len(bad)} of {got.size} off, first under scale {scales[bad[0, 0], bad[0, 1] // 32]}: "
                          f"{got[tuple(bad[0])]} against {want[tuple(bad[0])]}")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_gated_rows_of_the_largest_gates(dt):
    """Their codes: silu is the identity there, or nothing; what leaves fp32's range is infinite and its block NaN."""
    announce(f"gated rows of the largest gates {dt}")
    g = np.array([100, 127, 128, 129, 1e30, 2.3e38, 2.37e38, 3.3e38, np.inf, np.nan, -100, -128, -1e30, -2.4e38, -np.inf])
    u = np.array([0.0, 1.0, -0.5, 1.4e-45, 1e-38, 1e-10, 3e20, -3.3e38])
    g, u = (v.reshape(-1) for v in np.meshgrid(g, u, indexing="ij"))
    x = np.zeros((g.size, 128), np.float32)
    x[:, 0], x[:, 64] = g, u  # alone in its block
    x[:, 32:64], x[:, 96:] = 3.0, np.arange(32)  # and beside others
    x[:, 37], x[:, 101] = g, u
    x_d = torch.from_numpy(x).to(DEV).to(DT[dt])
    xh = host(x_d)
    with np.errstate(invalid="ignore", over="ignore"):
        v = silu_parts(xh[:, :64])[2] * xh[:, 64:]
        v = np.where(np.abs(v) > np.finfo(np.float32).max, np.inf, v)
    codes, scales = mx.quantize_mx_rows(v)
    q = e4b.mx4_rows(x_d, gated=True)
    for got, want, name in ((q.scales, scales, "scales"), (q.codes, codes, "codes")):
        bad = np.argwhere(got.cpu().numpy() != want)
        assert not bad.size, (name, g[bad[0, 0]], u[bad[0, 0]], got[tuple(bad[0])].item(), want[tuple(bad[0])])
