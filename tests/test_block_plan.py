"""The host-side plan of the stored-weight products: launches that the card can take (no GPU)."""

import pytest

from plan_util import T128, T256, TALL, linear_plan

THREADS = {T128: 256, TALL: 512, T256: 512}
ROWS_OF = {T128: 128, TALL: 256, T256: 256}
COLS_OF = {T128: 128, TALL: 128, T256: 256}


def grid_threads(E, rows, cols, tiles, splits):
    """Threads of the launch: every expert may end in a partial tile; workgroups come in eights."""
    bm = ROWS_OF[tiles]
    row_tiles = (rows + (bm - 1) * min(E, rows)) // bm
    groups = row_tiles * -(-cols // COLS_OF[tiles]) * splits
    return -(-groups // 8) * 8 * THREADS[tiles]


@pytest.mark.parametrize("E,rows,small,large", [(1024, 170000, 64, 640000), (1024, 200000, 64, 820000), (700, 140000, 64, 900000),
                                                (1, 1 << 20, 64, 1 << 17), (1024, 9000, 64, 1 << 20), (64, 1 << 18, 64, 1 << 19),
                                                (1, 1 << 22, 128, 1 << 16), (300, 60000, 128, 1 << 20)])
def test_accepted_products_fit_a_launch(E, rows, small, large):
    """A dimension of a launch has fewer than 2^32 threads."""
    for inn, out in ((small, large), (large, small)):
        p = linear_plan(E, rows, inn, out)
        if isinstance(p, int):  # refused
            continue
        fwd, bwd, fs, bs = p
        if fwd in THREADS:
            assert grid_threads(E, rows, out, fwd, fs) < 1 << 32, (inn, out, p)
        assert grid_threads(E, rows, inn, bwd, bs) < 1 << 32, (inn, out, p)
