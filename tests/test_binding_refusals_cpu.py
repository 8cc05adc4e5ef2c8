"""Arguments that the Python binding refuses before the library sees them,
without a GPU: device tensors stand in as shapes and strides only (their data
pointers are null, which the library would refuse in turn, with another
error)."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


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
            yield lambda *shape, dtype=torch.uint8: torch.empty(*shape, dtype=dtype, device="cuda:0")


M, N, K, E = 48, 256, 512, 3
F32, I32 = torch.float32, torch.int32


@pytest.mark.parametrize("one_row", [lambda t: t[..., :1, :].expand(*t.shape),
                                     lambda t: t.as_strided(t.shape, t.stride()[:-2] + (16, 1))])
def test_weight_rows_that_share_memory(w8, fake, one_row):
    """A row stride of 0 is the library's sign for packed weights: it would read
    N x K bytes from a buffer that holds one row."""
    xq, sx = fake(M, K), fake(M, K // 128, dtype=F32)
    sw, sws = fake(N // 128, K // 128, dtype=F32), fake(E, N // 128, K // 128, dtype=F32)
    wq, experts = one_row(fake(N, K)), one_row(fake(E, N, K))
    off, rows = fake(E + 1, dtype=I32), fake(M, dtype=I32)
    with pytest.raises(ValueError, match="row stride"):
        w8.block_gemm(xq, sx, wq, sw)
    with pytest.raises(ValueError, match="row stride"):
        w8.grouped_gemm(xq, sx, off, experts, sws)
    with pytest.raises(ValueError, match="row stride"):
        w8.gemm_w8a8("Block_FP8", xq[:8], sx[:8], wq, sw)
    with pytest.raises(ValueError, match="row stride"):
        w8.linear("Block_FP8", fake(8, K, dtype=torch.bfloat16), wq, sw, fused=True)
    with pytest.raises(ValueError, match="row stride"):
        w8.moe_gemm("Block_FP8", xq[:8], sx[:8], off, rows, experts, sws)
    with pytest.raises(ValueError, match="row stride"):
        w8.moe_linear("Block_FP8", fake(8, K, dtype=torch.bfloat16), off, rows, experts, sws)


def test_a_single_weight_row_may_have_any_stride(w8):
    assert w8._weight_stride(0, 1, 512) == 512
    assert w8._weight_stride(7, 1, 512) == 512
    assert w8._weight_stride(528, 1, 512) == 528
    assert w8._weight_stride(528, 9, 512) == 528
