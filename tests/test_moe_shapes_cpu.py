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


def test_scales_of_blocks_in_another_order(w8, fake, monkeypatch):
    """Block_FP8's scales as they lie behind a transposed or permuted tensor: as many
    elements, of other blocks.  Flat ones are taken as they lie."""
    G, H = D // 128, I // 128
    a = dict(xq=fake(T, D), sx=fake(T, G, dtype=F32), experts=fake(T, K, dtype=I32),
             weights=fake(T, K, dtype=F32), w1=fake(E, 2 * I, D), s1=fake(E, 2 * H, G, dtype=F32),
             w2=fake(E, D, I), s2=fake(E, G, H, dtype=F32))
    for name, what, shape in (("sx", "sx", (G, T)), ("s1", "scales of w1", (E, G, 2 * H)),
                              ("s1", "scales of w1", (2 * H, E, G)), ("s2", "scales of w2", (E, H, G))):
        with pytest.raises(ValueError, match=what + " must be"):
            w8.moe_layer("Block_FP8", **{**a, name: fake(*shape, dtype=F32)})
    monkeypatch.setattr(w8.moe, "_current_device", lambda: 0)
    # (past these checks: pointers without memory are what the library refuses)
    for s in ({}, dict(sx=fake(T * G, dtype=F32), s1=fake(E * 2 * H * G, dtype=F32))):
        with pytest.raises(w8.W8Error, match="null device pointer"):
            w8.moe_layer("Block_FP8", **{**a, **s}, y=fake(T, D, dtype=BF16),
                         workspace=w8.Workspace("cuda:0"), stream=0)


def test_a_single_expert_may_have_any_stride(w8):
    """No address holds it.  (The call ends at the workspace that it does not have.)"""
    p = 0x1000

    def status(E, **kw):
        a = dict(fmt=1, E=E, T=T, topk=1, D=D, I=I, xq=p, ldq=D, sx=p, experts=p, weights=p, w1=p,
                 ldw1=D, w1_stride=2 * I * D, s1=p, s1_stride=2 * I, w2=p, ldw2=I, w2_stride=D * I,
                 s2=p, s2_stride=D, base=None, ldb=0, y=p, ldy=D, ws=None, ws_bytes=0, stream=None)
        assert set(kw) <= set(a)
        return w8._lib.w8_moe_layer(*{**a, **kw}.values())

    invalid, workspace = 1, 3
    for kw in (dict(w1_stride=1), dict(w2_stride=0), dict(w1_stride=-7, s1_stride=0),
               dict(w2_stride=8, s2_stride=1), dict(ldw1=0, w1_stride=1)):
        assert status(1, **kw) == workspace
        assert status(2, **kw) == invalid
