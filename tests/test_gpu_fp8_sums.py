"""FP8_Dynamic sums on the GPU are as exact as the matrix instruction's products:
its rounding (2^-16 of a result in the root mean square, for codes of normally
distributed values) does not grow with the steps that are added up."""
import numpy as np
import pytest
import torch

from tests.block_cases import DEV
from tests.test_gpu_moe_layer import FORMATS, Layer, sized

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


def normal_codes(g, n, K):
    v = torch.randn(n, K, generator=g, device=DEV)
    s = v.abs().amax(dim=1) / 448
    return (v / s[:, None]).to(torch.float8_e4m3fn), s


@pytest.mark.parametrize("M,N,K", [(512, 512, 1024), (512, 512, 8192), (100, 2000, 65536),
                                   (8, 4096, 4096), (32, 512, 65536), (300, 4000, 5120)])
def test_outputs_beside_the_rounded_exact_one(w8, M, N, K):
    """An output lies beside the rounded exact one where the sum's error, normal with
    2^-16 of the outputs' root mean square, carries it over a border between two bf16
    values: |error| / step of the outputs, with E|error| = 0.8 of that.  Twice as many
    may; a sum that was rounded as much at each of 64 steps would give five times."""
    print(f"[case] {M} x {N} x {K}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N + K)
    (xq, sx), (wq, sw) = normal_codes(g, M, K), normal_codes(g, N, K)
    y = w8.token_gemm("FP8_Dynamic", xq, sx, wq, sw)
    exact = (xq.double() * sx.double()[:, None]) @ (wq.double() * sw.double()[:, None]).t()
    _, e = torch.frexp(exact)
    step = torch.ldexp(torch.ones_like(exact), e - 8)  # |exact| in [2^(e-1), 2^e)
    rms = exact.square().mean().sqrt()
    share = (0.8 * 2.0 ** -16 * rms / step).clamp(max=1).mean().item()
    beside = (y != exact.to(torch.bfloat16)).double().mean().item()
    assert beside <= 2 * share, f"{beside} of the outputs, {share} by the instruction's rounding"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,topk,D,I", [(32, 8, 4, 2048, 768), (32, 4, 2, 1024, 4096),
                                          (24, 2, 2, 2048, 2048)])
def test_layer_within_a_rounding_and_its_codes(w8, fmt, T, E, topk, D, I):
    """The outputs' rounding is 2^-8 / 3^(1/2) of a value at most, 0.0023, in the root
    mean square.  A hidden value's error of d carries its code over a border with
    probability 2 d / step and changes it by a step, so codes add the root of 2 d step:
    d is 2^-15 of a value (two halves, each 2^-16 of the halves' root mean square), the
    step 2^-3 of it at most: 0.0028.  Both together stay below 2^-8 = 0.0039."""
    c = Layer(fmt, T, E, topk, *sized(fmt, D, I))
    y, _ = c.expected()
    got = w8.moe_layer(*c.args(w8)).double().cpu().numpy()
    off = np.linalg.norm(got - y) / np.linalg.norm(y)
    assert off <= 2.0 ** -8, off
