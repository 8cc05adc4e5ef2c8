"""Tensors of the right number of elements in another order, which the MoE
operators refuse, without a GPU: device tensors stand in as shapes and strides
only."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

F32, I32, BF16 = torch.float32, torch.int32, torch.bfloat16
T, E, K, D, I = 8, 4, 2, 256, 384


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


@pytest.fixture
def fake():
    """torch factories give tensors without memory on a device that need not exist."""
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        with FakeTensorMode():
            yield lambda *shape, dtype=torch.int8: torch.empty(*shape, dtype=dtype, device="cuda:0")


@pytest.mark.parametrize("shape", [(K, T), (T * K,), (T, K, 1), (1, T, K)])
def test_weights_of_the_choices_in_another_order(w8, fake, shape):
    """[topk, T] holds as many weights as [T, topk], of other choices."""
    weights, choices = fake(*shape, dtype=F32), fake(T, K, dtype=I32)
    with pytest.raises(ValueError, match=r"weights must be \[8, 2\]"):
        w8.moe_combine(fake(T * K, D, dtype=BF16), weights, choices)
    with pytest.raises(ValueError, match=r"weights must be \[8, 2\]"):
        w8.moe_layer("W8A8_INT8", fake(T, D), fake(T, dtype=F32), choices, weights,
                     fake(E, 2 * I, D), fake(E, 2 * I, dtype=F32), fake(E, D, I),
                     fake(E, D, dtype=F32))
