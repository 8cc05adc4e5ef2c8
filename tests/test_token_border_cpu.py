"""Which kernel runs a token-scaled product of up to 32 tokens, without a GPU: the
small-M GEMM (a plan without a tile) or the tiles, on both sides of the border."""
import pytest

from tests.token_cases import FORMATS


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K,row,packed", [
    # above 16 tokens: 2^23 weights in either layout
    (17, 4096, 2048, True, True), (32, 896, 8192, True, True), (32, 4112, 2048, False, False),
    (17, 1792, 5120, False, False), (32, 8192, 1024, True, True),
    # up to 16: 24 * 2^20 weights row-major, any packed
    (16, 3584, 5120, True, True), (16, 6143, 4096, True, True), (16, 6144, 4096, False, True),
    (8, 4608, 7168, False, True), (1, 5120, 8192, False, True), (16, 16384, 8192, False, True),
    # above 32 never
    (33, 16, 128, False, False)])
def test_border(w8, fmt, M, N, K, row, packed):
    assert (w8.token_gemm_plan(fmt, M, N, K)["tile_m"] == 0) == row
    assert (w8.token_gemm_plan(fmt, M, N, K, packed=True)["tile_m"] == 0) == packed


@pytest.mark.parametrize("M,N,K", [(32, 4096, 2048), (17, 2048, 2048), (16, 8192, 8192)])
def test_block_fp8_keeps_its_own(w8, M, N, K):
    """Its border was measured on its kernels."""
    assert w8.block_gemm_plan(M, N, K)["tile_m"] != 0
    assert w8.block_gemm_plan(M, N, K, packed=True)["tile_m"] != 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_packed_size_has_a_plan_and_a_workspace(w8, fmt):
    for M in (1, 7, 8, 16, 17, 32):
        for N, K in ((1, 128), (17, 130944), (1 << 24, 128), (70001, 8192), (300000, 1024)):
            w8.token_gemm_plan(fmt, M, N, K, packed=True)
            assert w8.token_gemm_workspace_size(fmt, M, N, K, packed=True) >= 0
