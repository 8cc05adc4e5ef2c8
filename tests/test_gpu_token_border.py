"""Token-scaled products on both sides of the border between the small-M GEMM and
the tiles: the same definition either way, W8A8_INT8 bit for bit."""
import numpy as np
import pytest
import torch

from tests.block_cases import on_device
from tests.token_cases import FORMATS, assert_product, bits_of, codes, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(17, 4096, 2048), (32, 1030, 8064), (32, 2560, 3456),
                                   (16, 6144, 4096), (9, 7000, 4224), (1, 3600, 8192)])
def test_product(w8, fmt, M, N, K):
    print(f"[case] {fmt} {M} x {N} x {K}", flush=True)
    g = np.random.default_rng([M, N, K])
    c = codes(g, fmt, M, K), scales(g, M), codes(g, fmt, N, K), scales(g, N)
    t = torch.int8 if fmt == "W8A8_INT8" else torch.float8_e4m3fn
    xq, sx, wq, sw = (on_device(v) for v in c)
    xq, wq = xq.view(t), wq.view(t)
    for w in (wq, w8.pack_weight(fmt, wq)):
        assert_product(fmt, bits_of(w8.token_gemm(fmt, xq, sx, w, sw)), *c)
