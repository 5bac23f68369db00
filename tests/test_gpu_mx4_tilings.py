"""GPU tests of the microscaled product in each tiling, which the host's plan is asked for: K-steps by whole panels of
scales, and where a block without a value shows."""

import numpy as np
import pytest
import torch

import bit_quantized_mixture_nf4_amd as e4b
import test_gpu_mx4 as mx4
from gpu_util import DEV, announce
from test_mx_plan import ROWS, T64, T128, T256, mx_plan

pytestmark = pytest.mark.gpu


# 256 x 256 tiles whose K-steps of 256 fill the panels of four steps' scales exactly (4, 8, 16 and 20 steps): several
# tiles a workgroup, and one.
WHOLE_PANELS = [
    (40, 40000, 1, 1024, 2048, "none", True, False, "bf16"), (7, 9500, 130, 2048, 2056, "silu", True, True, "bf16"),
    (1, 5000, 0, 4096, 4096, "none", False, False, "bf16"), (4, 9000, 3, 4096, 2048, "none", True, False, "fp32"),
    (3, 8000, 0, 1024, 2312, "gelu_tanh", False, True, "bf16"), (2, 8000, 1, 5120, 1800, "none", False, False, "bf16"),
]


@pytest.mark.parametrize("E,rows,tail,inn,out,act,with_bias,with_res,yt", WHOLE_PANELS)
def test_products_of_whole_panels(E, rows, tail, inn, out, act, with_bias, with_res, yt):
    assert mx_plan(E, rows + tail, inn, out).tiles == T256
    mx4.test_product_in_every_tiling(E, rows, tail, inn, out, act, with_bias, with_res, yt)


@pytest.mark.parametrize("T,k,E,inn,out,drop", [(5000, 8, 40, 1024, 2048, 0.0), (4700, 2, 7, 2048, 2056, 0.1),
                                                (4600, 2, 3, 4096, 2048, 0.0), (3000, 4, 6, 1280, 2312, 0.2)])
def test_gathered_products_of_several_panels(T, k, E, inn, out, drop):
    assert mx_plan(E, T * k, inn, out, k).tiles == T256
    mx4.test_product_gathered_by_token(T, k, E, inn, out, drop)


@pytest.mark.parametrize("E,rows,inn,out,act,tiles", [
    (1, 7, 192, 48, "none", ROWS), (5, 60, 2048, 80, "silu", ROWS), (9, 200, 2112, 300, "none", T64),
    (700, 2500, 192, 264, "gelu", T64), (3, 3005, 704, 1028, "silu", T128), (6, 6011, 1152, 1288, "none", T128),
    (5, 12033, 768, 2048, "none", T256), (40, 40001, 1024, 2048, "none", T256), (7, 9630, 2304, 2056, "silu", T256),
    (1, 5000, 4096, 4096, "none", T256)])
def test_blocks_without_a_value_in_every_tiling(E, rows, inn, out, act, tiles):
    """A NaN scale of a row makes that row of the product NaN throughout, one of a weight row that column of its
    expert, and everything else keeps its bits."""
    announce(f"mx product with NaN blocks E={E} rows={rows} {inn}->{out}")
    assert mx_plan(E, rows, inn, out).tiles == tiles
    rng = np.random.default_rng(rows)
    gen = torch.Generator(device=DEV).manual_seed(rows)
    packed = torch.randint(0, 256, (E, out * inn // 2), generator=gen, device=DEV, dtype=torch.uint8)
    scales = torch.randint(118, 123, (E, out * inn // 32), generator=gen, device=DEV, dtype=torch.uint8)
    offsets = np.concatenate([[0], np.cumsum(mx4._counts(E, rows, rng))]).astype(np.int32)
    off = torch.from_numpy(offsets).to(DEV) if E > 1 else None
    q = e4b.mx4_rows(torch.randn(rows, inn, device=DEV, generator=gen))
    res = torch.randn(rows, out, device=DEV, generator=gen).to(torch.bfloat16)

    def product(x_scales, w_scales):
        stack = e4b.QuantStack(packed, None, E, out, inn, "mxfp4", w_scales)
        return e4b.mx_linear(stack, e4b.MxRows(q.codes, x_scales), offsets=off, act=act, residual=res, save=True)

    want = product(q.scales, scales)
    assert not any(t.isnan().any() for t in want)
    # rows at the ends of tiles and experts, blocks from the first to the last
    some = sorted({min(r, rows - 1) for r in (0, 3, 15, 16, 63, 64, 127, 128, 255, 256, 300, rows // 2, rows - 1)}
                  | {int(offsets[E // 2]) % rows})
    x_scales = q.scales.clone()
    for i, r in enumerate(some):
        x_scales[r, (i * (inn // 32 - 1)) // max(len(some) - 1, 1)] = 255
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[some] = True
    for got, ref in zip(product(x_scales, scales), want):
        assert got[bad].isnan().all() and torch.equal(mx4.bits(got[~bad]), mx4.bits(ref[~bad]))
    # columns of two experts
    w_scales = scales.clone().view(E, out, inn // 32)
    bad = torch.zeros(rows, out, dtype=torch.bool, device=DEV)
    for e in {E // 2, E - 1}:
        for i, c in enumerate(sorted({min(c, out - 1) for c in (0, 5, 63, 64, 127, 255, 256, out - 1)})):
            w_scales[e, c, (7 * i) % (inn // 32) if i else inn // 32 - 1] = 255
            bad[offsets[e]:offsets[e + 1], c] = True
    for got, ref in zip(product(q.scales, w_scales.view(E, -1)), want):
        assert got[bad].isnan().all() and torch.equal(mx4.bits(got[~bad]), mx4.bits(ref[~bad]))
