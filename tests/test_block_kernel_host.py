"""The tiled Block_FP8 GEMM's kernels on the CPU: every address that a
direct-to-LDS load reads lies inside its array, outputs are stored inside their
rows, and the product is right whichever wavefront runs first and whether loads
arrive at once or only when a wait asks for them."""
import os

import numpy as np
import pytest

from tests.block_cases import dequant_blocks, dequant_rows, draw_codes, draw_scales, groups
from tests.kernel_host import gemm as host

pytestmark = pytest.mark.skipif(not os.path.exists(host.CLANG), reason="no clang")

ORDERS = [(False, False), (True, False), (False, True), (True, True)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return host.build(str(tmp_path_factory.mktemp("block_gemm")))


def inputs(M, N, K, E=None, seed=0):
    g = np.random.default_rng([seed, M, N, K])
    e = () if E is None else (E,)
    return (draw_codes(g, M, K), draw_scales(g, M, groups(K)), draw_codes(g, *e, N, K),
            draw_scales(g, *e, groups(N), groups(K)))


def assert_near(y, x, w, what):
    """The bound of the GPU tests: a bf16 rounding, and sums within 2^-14 of
    the sum of |products|."""
    Y, S = x @ w.T, np.abs(x) @ np.abs(w).T
    bad = ~(np.abs(y - Y) <= 2.0 ** -8 * 1.01 * np.abs(Y) + 2.0 ** -14 * 1.01 * S + 1e-38)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, at {np.argwhere(bad)[:4].tolist()}"


def check(lib, tile, M, N, K, orders=ORDERS, **kw):
    c = inputs(M, N, K)
    for descending, late in orders:
        y, faults, text = host.run(lib, tile, *c, descending=descending, late=late, **kw)
        assert faults == 0, text
        assert_near(y, dequant_rows(*c[:2]), dequant_blocks(*c[2:]), f"{tile} {kw}")


def check_grouped(lib, tile, counts, N, K, T, orders=ORDERS, **kw):
    off = np.r_[0, np.cumsum(counts)]
    c = inputs(T or off[-1], N, K, len(counts))
    rows = None if T is None else np.random.default_rng(1).integers(0, T, off[-1])
    for descending, late in orders:
        y, faults, text = host.run(lib, tile, *c, offsets=off, rows=rows, descending=descending,
                                   late=late, **kw)
        assert faults == 0, text
        for e in range(len(counts)):
            at = np.arange(off[e], off[e + 1])
            x = at if rows is None else rows[at]
            assert_near(y[at], dequant_rows(c[0][x], c[1][x]), dequant_blocks(c[2][e], c[3][e]),
                        f"{tile} expert {e}")


# Loops from one step to more than the deepest staging and a group of steps.
@pytest.mark.parametrize("tile,M,N", [("16x128", 17, 130), ("64x64", 70, 130),
                                      ("64x128", 70, 130), ("128x128", 130, 140)])
@pytest.mark.parametrize("K,packed", [(128, False), (256, True), (1408, False), (1408, True),
                                      (1424, False)])
def test_tile(lib, tile, M, N, K, packed):
    check(lib, tile, M, N, K, packed=packed)


@pytest.mark.parametrize("parts", [1, 2, 4])
@pytest.mark.parametrize("K,packed", [(128, True), (640, False), (640, True), (656, False)])
def test_largest_tile(lib, parts, K, packed):
    check(lib, "256x256", 300, 300, K, orders=ORDERS[::3], parts=parts, packed=packed)


@pytest.mark.parametrize("tile,M,N", [("16x128", 17, 130), ("64x64", 70, 130),
                                      ("64x128", 70, 130), ("128x128", 130, 140)])
@pytest.mark.parametrize("split_k", [2, 4])
def test_split(lib, tile, M, N, split_k):
    check(lib, tile, M, N, 1424, split_k=split_k, orders=ORDERS[::3])


def test_split_flag_outlives_the_output_tile(lib):
    """Wavefronts that run ahead after the split's hand-off must not overwrite
    what the others have yet to read: with a tile whose first outputs are zero
    (four weight rows of zeros) all outputs are still stored."""
    c = inputs(130, 140, 1408)
    c[2][:4] = 0
    for tile in ("64x128", "128x128"):
        for descending, late in ORDERS:
            y, faults, text = host.run(lib, tile, *c, split_k=2, descending=descending, late=late)
            assert faults == 0, text
            assert_near(y, dequant_rows(*c[:2]), dequant_blocks(*c[2:]), tile)


@pytest.mark.parametrize("K", range(16, 128, 16))
@pytest.mark.parametrize("parts", [1, 2, 4])
def test_single_short_step_reads_inside(lib, K, parts):
    """K ends inside the only step, and the last row is in the last weight tile
    of the largest tile: no load may reach past the rows' ends."""
    check(lib, "256x256", 300, 512, K, orders=ORDERS[:1], parts=parts)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("tile,counts,N,T", [
    ("16x128", [5, 0, 30], 130, 9), ("64x128", [5, 0, 70, 1], 200, 40),
    ("128x128", [150, 0, 3], 200, None), ("256x256", [300, 3, 0, 150], 300, 20)])
def test_grouped(lib, tile, counts, N, T, packed):
    check_grouped(lib, tile, counts, N, 384, T, packed=packed, orders=ORDERS[::3])


@pytest.mark.parametrize("counts,N,T", [([140], 256 * 129, None), ([70, 300], 256 * 33, 9)])
def test_grouped_single_short_step_reads_inside(lib, counts, N, T):
    """The largest tile at full and at half size, whole and in pieces."""
    check_grouped(lib, "256x256", counts, N, 64, T, orders=ORDERS[:1])


def test_a_read_past_the_end_is_seen(lib):
    for tile in host.TILES:
        c = inputs(130, 256, 256)
        assert host.run(lib, tile, *c, hide=16, parts=1)[1] > 0, tile


def test_launchers_refuse_tiles_that_are_not_built(lib):
    """(another tile's kernel on this one's grid would compute something else)"""
    ids = {name: t[0] for name, t in host.TILES.items()}
    for packed in (0, 1):
        for id_ in ids.values():
            assert lib.emu_launch(id_, 0, packed) == 0
            assert lib.emu_launch(id_, 1, packed) == (1 if id_ == ids["64x64"] else 0)
        for id_ in (-1, len(ids)):
            assert lib.emu_launch(id_, 0, packed) == 1 and lib.emu_launch(id_, 1, packed) == 1
