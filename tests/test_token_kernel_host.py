"""The tiled GEMM of the token-scaled formats on the CPU: every address that a
direct-to-LDS load reads lies inside its array, outputs are stored inside their
rows, and the product is right whichever wavefront runs first and whether loads
arrive at once or only when a wait asks for them."""
import os

import numpy as np
import pytest

from tests.kernel_host import token_gemm as host
from tests.token_cases import FORMATS, assert_product, codes, scales

pytestmark = pytest.mark.skipif(not os.path.exists(host.CLANG), reason="no clang")

ORDERS = [(False, False), (True, False), (False, True), (True, True)]
SMALL = [("16x128", 17, 130), ("64x64", 70, 130), ("64x128", 70, 130), ("128x128", 130, 140)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return host.build(str(tmp_path_factory.mktemp("token_gemm")))


def check(lib, fmt, tile, M, N, K, orders=ORDERS, **kw):
    g = np.random.default_rng([M, N, K])
    c = codes(g, fmt, M, K), scales(g, M), codes(g, fmt, N, K), scales(g, N)
    for descending, late in orders:
        y, faults, text = host.run(lib, fmt, tile, *c, descending=descending, late=late, **kw)
        assert faults == 0, text
        assert_product(fmt, y, *c, f"{tile} {kw}")


# Loops from one step to more than the deepest staging and a group of steps.
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tile,M,N", SMALL)
@pytest.mark.parametrize("K,packed", [(128, False), (256, True), (1408, False), (1424, False)])
def test_tile(lib, fmt, tile, M, N, K, packed):
    check(lib, fmt, tile, M, N, K, packed=packed, orders=ORDERS[::3])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("parts", [1, 2, 4])
@pytest.mark.parametrize("K,packed", [(128, True), (640, False), (656, False)])
def test_largest_tile(lib, fmt, parts, K, packed):
    check(lib, fmt, "256x256", 300, 300, K, orders=ORDERS[::3], parts=parts, packed=packed)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tile,M,N", SMALL)
def test_split(lib, fmt, tile, M, N):
    check(lib, fmt, tile, M, N, 1424, split_k=4, orders=ORDERS[::3])


@pytest.mark.parametrize("K", range(16, 128, 32))
@pytest.mark.parametrize("parts", [1, 2, 4])
def test_single_short_step_reads_inside(lib, K, parts):
    check(lib, "W8A8_INT8", "256x256", 300, 512, K, orders=ORDERS[:1], parts=parts)


@pytest.mark.parametrize("tile", host.TILES)
def test_one_row(lib, tile):
    """One token and one weight row: every load but the first of each repeats."""
    check(lib, "W8A8_INT8", tile, 1, 1, 144, orders=ORDERS[::3], parts=1)


def test_a_read_past_the_end_is_seen(lib):
    g = np.random.default_rng(0)
    c = codes(g, "W8A8_INT8", 130, 256), scales(g, 130), codes(g, "W8A8_INT8", 256, 256), scales(g, 256)
    for tile in host.TILES:
        for name in ("xq", "sx", "wq", "sw"):
            assert host.run(lib, "W8A8_INT8", tile, *c, hide=name, parts=1)[1] > 0, (tile, name)


def test_launcher_refuses_tiles_that_are_not_built(lib):
    for fmt in host.FMT.values():
        for packed in (0, 1):
            assert all(lib.emu_launch(fmt, t, packed) == 0 for t in range(len(host.TILES)))
            assert lib.emu_launch(fmt, -1, packed) == lib.emu_launch(fmt, len(host.TILES), packed) == 1
