"""The plan functions of the Block_FP8 GEMMs: what runs which shape, that the
GPU tests' shapes reach every kernel that is built, refusals (no GPU)."""
import ctypes

import pytest

from tests.block_plans import DENSE, EVERY_TILE, GROUPED, LARGE

OK, INVALID = 0, 1
TILES = {(16, 128), (64, 64), (64, 128), (128, 128), LARGE}


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


def tile(p):
    return p["tile_m"], p["tile_n"]


@pytest.mark.parametrize("shape", DENSE)
def test_dense(w8, shape):
    M, N, K, packed = shape
    p = w8.block_gemm_plan(M, N, K, packed=packed)
    assert (tile(p), p["split_k"], p["parts"]) == DENSE[shape]
    tiles = -(-M // p["tile_m"]) * -(-N // p["tile_n"])
    whole = tiles if p["parts"] == 1 else tiles // 256 * 256
    assert p["workgroups"] == (whole + p["parts"] * (tiles - whole)) * p["split_k"]
    ws = w8.block_gemm_workspace_size(M, N, K, packed=packed)
    partials = tiles * p["split_k"] * p["tile_m"] * p["tile_n"] * 4
    assert ws == (partials + (2 << 20) if p["split_k"] > 1 else 0)


def test_dense_shapes_reach_every_kernel():
    reached = {(tile, split > 1, parts, packed)
               for (*_, packed), (tile, split, parts) in DENSE.items()}
    want = {(t, split, 1, packed) for t in TILES - {LARGE} for split in (False, True)
            for packed in (False, True)}
    want |= {(LARGE, False, parts, packed) for parts in (1, 2, 4) for packed in (False, True)}
    assert reached == want
    # one step that K ends inside of: the largest tile in all its forms
    assert {parts for (_, _, K, _), (t, _, parts) in DENSE.items() if K < 128 and t == LARGE} \
        == {1, 2, 4}


@pytest.mark.parametrize("K", [272, 384])
def test_every_tile_by_rows(w8, K):
    for M, (t, parts) in EVERY_TILE.items():
        p = w8.block_gemm_plan(M, 4200, K)
        assert (tile(p), p["split_k"], p["parts"]) == (t, 1, parts)
    assert {t for t, _ in EVERY_TILE.values()} == TILES


def test_grouped(w8):
    reached = set()
    for counts, N, K, T, t in GROUPED:
        n = sum(counts)
        p = w8.grouped_gemm_plan(len(counts), T or n, N, K, n_rows=n)
        assert tile(p) == t and p["split_k"] == 1, (counts, N, K)
        reached |= {(t, False)} | ({(t, True)} if K % 128 == 0 else set())
    assert reached == {(t, packed) for t in TILES - {(64, 64)} for packed in (False, True)}


def test_rows_far_apart_leave_the_largest_tile(w8):
    """It addresses gathered rows by 32-bit offsets from the first."""
    assert tile(w8.grouped_gemm_plan(1, 4095, 2100, 256, n_rows=4200, ldq=1 << 20)) == LARGE
    assert tile(w8.grouped_gemm_plan(1, 4096, 2100, 256, n_rows=4200, ldq=1 << 20)) == (128, 128)


def test_small_m_and_nothing(w8):
    for shape in ((1, 2048, 2048), (0, 2048, 2048)):
        p = w8.block_gemm_plan(*shape)
        assert tile(p) == (0, 0) and p["split_k"] == 1 and p["workgroups"] == 0
    assert tile(w8.block_gemm_plan(1, 4608, 7168)) != (0, 0)
    assert w8.grouped_gemm_plan(8, 0, 2048, 2048, n_rows=0)["workgroups"] == 0


def test_refusals(w8):
    lib, p = w8._lib, w8._capi.BlockPlan(7)
    for args in ((-1, 512, 1024, 0), (1 << 22, 512, 1024, 0), (48, 0, 1024, 0), (48, 512, 1000, 0),
                 (48, 512, 1024, 2), (48, 512, 1040, 1)):
        assert lib.w8_block_gemm_plan(*args, ctypes.byref(p)) == INVALID
    assert lib.w8_block_gemm_plan(48, 512, 1024, 0, None) == INVALID
    for args in ((0, 9, 512, 1024, 1024, 9), (65537, 9, 512, 1024, 1024, 9),
                 (4, -1, 512, 1024, 1024, 9), (4, 9, 0, 1024, 1024, 9), (4, 9, 512, 1032, 1032, 9),
                 (4, 9, 512, 1024, 1008, 9), (4, 9, 512, 1024, 1032, 9),
                 (4, 9, 512, 1024, (1 << 23) + 16, 9), (4, 9, 512, 1024, 1024, -1)):
        assert lib.w8_grouped_gemm_plan(*args, ctypes.byref(p)) == INVALID
        assert lib.w8_last_error()
    assert lib.w8_grouped_gemm_plan(4, 9, 512, 1024, 1024, 9, None) == INVALID
    assert p.tile_m == 7  # nothing was written
