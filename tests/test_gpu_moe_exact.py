"""W8A8_INT8 through the MoE layer: a product's sum is exact however it is split,
so a token's outputs are the same bits whoever else is in the call."""
import numpy as np
import pytest
import torch

from tests.block_cases import DEV, on_device
from tests.token_cases import codes, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


@pytest.mark.parametrize("E,topk,D,I,coded", [
    (1, 1, 4096, 4096, True),    # the second projection in four parts, codes of the hidden values apart
    (2, 1, 2048, 2048, False),   # in two parts, by the tiles
    (4, 2, 2048, 1024, False)])  # whole
def test_a_token_whoever_else_is_there(w8, E, topk, D, I, coded):
    """A part that is rounded before the others are added shows in about one output
    of 25000 (where the fp32 value lies next to a bf16 border): half a million are
    compared."""
    g = np.random.default_rng([E, D, I])
    w1, w2 = (on_device(codes(g, "W8A8_INT8", *s)).view(torch.int8) for s in ((E, 2 * I, D), (E, D, I)))
    s1 = on_device((g.uniform(0.5, 2, (E, 2 * I)) / (73 * 73 * D ** 0.5)).astype(np.float32))
    s2 = on_device(scales(g, (E, D)))
    T = 32 if coded else 12
    for seed in range(-(-(1 << 19) // (T * D))):
        xq = on_device(codes(g, "W8A8_INT8", T, D)).view(torch.int8)
        sx = on_device(g.uniform(0.5, 2, T).astype(np.float32))
        experts = on_device(np.stack([g.permutation(E)[:topk] for _ in range(T)]).astype(np.int32))
        weights = on_device(g.uniform(0.05, 1, (T, topk)).astype(np.float32))
        one = [xq, sx, experts, weights]
        together = w8.moe_layer("W8A8_INT8", *one, w1, s1, w2, s2)
        alone = torch.cat([w8.moe_layer("W8A8_INT8", *(a[t:t + 1] for a in one), w1, s1, w2, s2)
                           for t in range(T)])
        assert torch.isfinite(together).all()
        differ = (together != alone).sum().item()
        assert differ == 0, f"{differ} of {T * D} outputs, call {seed}"
