"""The row operators at the ends of the number range (GPU)."""
import numpy as np
import pytest
import torch

from tests.block_cases import DEV, E4M3, GROUP, assert_codes, bf16, groups

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


def codes_agree(zq, sz, z):
    """Codes and scales tell the same numbers as z: NaN or infinite scales
    exactly for the groups where z has such values, and zeros for zeros."""
    M, D = z.shape
    pad = torch.zeros(M, groups(D) * GROUP, device=DEV)
    pad[:, :D] = z.float()
    finite = torch.isfinite(pad.view(M, -1, GROUP)).all(dim=2)
    assert torch.equal(torch.isfinite(sz), finite)
    v = torch.from_numpy(E4M3[zq.view(torch.uint8).cpu().numpy()]).to(DEV)
    v = v * sz.double().repeat_interleave(GROUP, dim=1)[:, :D]
    keep = finite.repeat_interleave(GROUP, dim=1)[:, :D]
    assert (v[keep & (z == 0)] == 0).all()
    empty = finite & (pad.view(M, -1, GROUP) == 0).all(dim=2)
    assert (sz[empty] == 1).all()


# one wave a row, several, a last group of few
@pytest.mark.parametrize("D", [256, 400, 1160, 9000])
@pytest.mark.parametrize("rdtype", [torch.bfloat16, torch.float32])
def test_norm_codes_follow_the_norm(w8, D, rdtype):
    """Rows whose factor 1 / sqrt(mean h^2 + eps) is NaN (a NaN in the row, in
    another group than the zeros), infinite (zeros with eps = 0) or 0 (an
    infinity, or squares that fp32 does not hold)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    h = torch.randn(7, D, generator=g, device=DEV).to(rdtype)
    h[0, 5], h[2, 7], h[4, 3] = float("nan"), float("inf"), float("-inf")
    h[3] = 0
    h[5] *= 2.0 ** 90
    h[:, 128:256] = 0
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    y = torch.zeros(7, D, dtype=torch.bfloat16, device=DEV)
    for eps in (0.0, 1e-6):
        _, zq, sz, z = w8.residual_norm(y, h, w, eps=eps, quantize=True, with_z=True)
        assert torch.isnan(z[0]).all() and (z[5] == 0).all()
        assert torch.isnan(z[3]).all() if eps == 0 else (z[3] == 0).all()
        codes_agree(zq, sz, z)
        assert torch.isnan(sz[0]).all()
        # the rows between are as they are alone
        alone = w8.residual_norm(y[6:], h[6:].clone(), w, eps=eps, quantize=True)
        assert torch.equal(zq[6].view(torch.uint8), alone[1][0].view(torch.uint8))
        assert torch.equal(sz[6], alone[2][0])
