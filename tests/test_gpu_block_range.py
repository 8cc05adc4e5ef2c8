"""The row operators at the ends of the number range (GPU)."""
import numpy as np
import pytest

from tests.block_cases import assert_codes, bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


@pytest.mark.parametrize("gate", [-80, -87, -87.5, -88, -88.5, -89, -92, -95, -100, -104, -150,
                                  -1e30, -3.3e38])
def test_far_negative_gates(w8, gate):
    """Whole groups of gates whose silu, g exp(g), is tiny: as long as fp32
    holds the product (to g = -103.9) it is not lost, whatever 1 / (1 +
    exp(-g)) does on the way.  dv: 2^-20 of the value as for other gates, and
    the spacing 2^-149 of the smallest numbers, of the value and (448 of them)
    of the scale."""
    g = np.random.default_rng(7)
    gates, gv = bf16(np.full((3, 256), gate) * (1 + 0.002 * g.random((3, 256))))
    x, xv = bf16(g.standard_normal((3, 256)))
    q, s = w8.block_quantize(x, gate=gates)
    # (below half of that spacing fp32's products are 0)
    want = (gv * np.exp(gv) * xv).astype(np.float32).astype(np.float64)
    assert_codes(q, s, want, np.abs(want) * 2.0 ** -20 + 449 * 2.0 ** -149)
