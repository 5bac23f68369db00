"""The host-side plan of the microscaled products: launches that the card can take, one workspace for
rows in place and gathered ones, and the tilings that the GPU tests are meant to reach (no GPU)."""

import ctypes

import pytest

import bit_quantized_mixture_nf4_amd as e4b
from bit_quantized_mixture_nf4_amd import _lib

ROWS, T64, T128, T256 = 0, 1, 2, 3  # few rows, tiles


class Plan(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_int32), ("by_offsets", ctypes.c_bool), ("rows", ctypes.c_int64),
                ("off_tile_map", ctypes.c_size_t), ("ws_bytes", ctypes.c_size_t)]


def mx_plan(E, rows, inn, out, top_k=0):
    plan = e4b.load()._ZN3e4b14plan_mx_linearEPK9e4b_stacklibiiPNS_12MxLinearPlanE  # e4b::plan_mx_linear
    plan.restype = ctypes.c_int32
    plan.argtypes = [ctypes.POINTER(_lib.E4bStack), ctypes.c_int64, ctypes.c_int32, ctypes.c_bool, ctypes.c_int32,
                     ctypes.c_int32, ctypes.c_void_p]
    st = _lib.E4bStack(0x10000, None, E, out, inn, 32, e4b.CODEBOOKS["mxfp4"], 0x10000)  # never read here
    p = Plan()
    status = plan(ctypes.byref(st), rows, max(top_k, 1), top_k > 0, _lib.E4B_ACT_NONE, _lib.E4B_BF16, ctypes.byref(p))
    return status if status != _lib.E4B_OK else p


@pytest.mark.parametrize("E,rows,inn,out,tiles,by_offsets", [
    (1, 8, 2048, 4096, ROWS, True), (8, 128, 768, 2048, T64, True), (128, 64, 2048, 1536, T64, True),
    (9, 200, 2112, 300, T64, True), (5, 1507, 448, 700, T64, True), (1024, 2995, 128, 520, T64, False),
    (300, 9600, 128, 2048, T64, False), (3, 3005, 704, 1028, T128, True), (8, 4000, 1024, 520, T128, True),
    (6, 6011, 1152, 1288, T128, False), (2, 4100, 2048, 1027, T128, False), (1, 4100, 512, 2816, T256, False),
    (5, 12033, 768, 2048, T256, False), (7, 9630, 2304, 2056, T256, False), (300, 40001, 1024, 2048, T128, False),
    (40, 40001, 1024, 2048, T256, False)])
def test_tilings(E, rows, inn, out, tiles, by_offsets):
    p = mx_plan(E, rows, inn, out)
    assert (p.tiles, p.ws_bytes == 0) == (tiles, tiles == ROWS or by_offsets)


@pytest.mark.parametrize("E", [1, 3, 64, 513, 1024])
@pytest.mark.parametrize("rows", [1, 17, 100, 4096, 4097, 9000, 170000, 1 << 20])
@pytest.mark.parametrize("inn,out", [(64, 64), (64, 640000), (512, 1 << 20), (4096, 28672), (1 << 20, 8), (128, 300000)])
def test_accepted_products_fit_a_launch(E, rows, inn, out):
    """A dimension of a launch has fewer than 2^32 threads (256 a workgroup, and at most 1024 that clear rows)."""
    p = mx_plan(E, rows, inn, out)
    if isinstance(p, int):
        return
    if p.tiles in (T64, T128):
        bm = 64 if p.tiles == T64 else 128
        groups = (rows + (bm - 1) * min(E, rows)) // bm * -(-out // bm)
        assert (-(-groups // 8) * 8 + (1024 if p.by_offsets else 0)) * 256 < 1 << 32
    if p.tiles == T256:
        assert inn % 256 == 0 and inn >= 512 and out % 8 == 0
        assert (rows + 255 * min(E, rows)) // 256 * -(-out // 256) < 1 << 32


@pytest.mark.parametrize("E,rows,inn,out,top_k", [(8, 64, 2048, 4096, 8), (64, 32768, 2048, 2048, 8), (3, 9000, 704, 1028, 2),
                                                  (1, 8200, 1 << 20, 64, 1), (2, 1 << 20, 1 << 15, 640, 2), (1024, 65536, 64, 64, 4)])
def test_workspace_is_enough_for_gathered_rows(E, rows, inn, out, top_k):
    """It is asked for by rows alone."""
    there, gathered = mx_plan(E, rows, inn, out), mx_plan(E, rows, inn, out, top_k)
    assert gathered.ws_bytes <= there.ws_bytes
    if rows // top_k * (inn // 2) >= 1 << 32:
        assert gathered.tiles == ROWS
