"""What runs a shape of the token-scaled GEMM (token_plans.py), without a GPU, and
that the shapes together reach every kernel that is built for it."""
import pytest

from tests.token_cases import FORMATS
from tests.token_plans import LARGE, SHAPES, SMALL_M


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES)
def test_plan(w8, fmt, shape):
    M, N, K, packed = shape
    p = w8.token_gemm_plan(fmt, M, N, K, packed=packed)
    assert ((p["tile_m"], p["tile_n"]), p["split_k"], p["parts"]) == SHAPES[shape]
    split = p["split_k"] > 1 and (p["tile_m"], p["tile_n"]) != SMALL_M
    if (p["tile_m"], p["tile_n"]) != SMALL_M:
        assert (w8.token_gemm_workspace_size(fmt, M, N, K, packed=packed) > 0) == split


def test_every_kernel_is_reached():
    tiles = {(tile, packed) for (*_, packed), (tile, _, _) in SHAPES.items()}
    assert tiles >= {(t, p) for t in ((16, 128), (64, 64), (64, 128), (128, 128), LARGE)
                     for p in (False, True)}
    parts = {(parts, packed) for (*_, packed), (tile, _, parts) in SHAPES.items() if tile == LARGE}
    assert parts == {(n, p) for n in (1, 2, 4) for p in (False, True)}
    split = {tile for tile, k, _ in SHAPES.values() if k > 1}
    assert split >= {(16, 128), (64, 64), (128, 128)}


def test_a_plan_for_every_size(w8):
    """No shape within the limits is without one, and launches stay in range."""
    for fmt in FORMATS:
        for M in (1, 2, 31, 32, 33, 100, 1000, 4097, 100000, (1 << 22) - 1):
            for N in (1, 17, 300, 5000, 70000):
                for K in (16, 48, 128, 1040, 8192, 131056):
                    p = w8.token_gemm_plan(fmt, M, N, K)
                    assert p["split_k"] in (1, 2, 4, 8, 16) and p["parts"] in (1, 2, 4)
                    assert p["workgroups"] > 0 or p["tile_m"] == 0
