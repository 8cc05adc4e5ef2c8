"""Argument checks of the token-scaled operators for any token count and of the
MoE operators around the grouped products, without a GPU: every refusal happens
before the device is touched, and calls with nothing to do return at once."""
import ctypes
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FP8, INT8, BLOCK = 0, 1, 2
P = 0x1000  # a well-aligned address that no refused call reads
BIG = 1 << 40


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


@pytest.fixture(scope="module")
def lib(w8):
    return w8._lib


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


def null(d):
    return {k: (None if v == P else v) for k, v in d.items()}


QUANT = dict(fmt=INT8, M=4, K=256, x=P, ldx=256, gate=P, ldg=256, reciprocal=0, xq=P, ldq=256, sx=P,
             stream=None)
GEMM = dict(fmt=INT8, M=48, N=512, K=5120, xq=P, ldq=5120, sx=P, wq=P, ldw=5120, sw=P, y=P,
            ldy=512, ws=P, ws_bytes=BIG, stream=None)
ROUTE = dict(T=100, E=64, topk=8, logits=P, ldl=64, fp32=1, renormalize=1, scale=1.0, experts=P,
             weights=P, offsets=P, rows=P, slots=P, ws=P, ws_bytes=BIG, stream=None)
COMBINE = dict(T=10, topk=8, D=100, y=P, ldy=100, n_rows=80, weights=P, slots=P, base=P, ldb=100,
               out=P, ldo=100, stream=None)
LAYER = dict(fmt=BLOCK, E=4, T=8, topk=2, D=256, I=128, xq=P, ldq=256, sx=P, experts=P, weights=P,
             w1=P, ldw1=256, w1_stride=256 * 256, s1=P, s1_stride=4, w2=P, ldw2=128,
             w2_stride=256 * 128, s2=P, s2_stride=2, base=P, ldb=256, y=P, ldy=256, ws=P, ws_bytes=BIG,
             stream=None)


@pytest.mark.parametrize("bad", [
    dict(fmt=BLOCK), dict(fmt=3), dict(fmt=-1), dict(M=-1), dict(M=1 << 22), dict(K=0),
    dict(K=132), dict(K=(1 << 22) + 8), dict(reciprocal=2), dict(x=None), dict(xq=None), dict(sx=None), dict(x=P + 8),
    dict(ldx=248), dict(ldx=260), dict(gate=P + 2), dict(ldg=128), dict(ldg=257), dict(xq=P + 4),
    dict(ldq=248), dict(ldq=260), dict(sx=P + 2)])
def test_quantize_refuses(lib, bad):
    assert call(lib.w8_token_quantize, QUANT, **bad) == INVALID
    assert lib.w8_last_error()


@pytest.mark.parametrize("bad", [
    dict(fmt=BLOCK), dict(fmt=7), dict(M=-1), dict(M=1 << 22), dict(N=0), dict(N=(1 << 24) + 1),
    dict(K=8), dict(K=5112), dict(K=(1 << 17), ldq=1 << 17, ldw=1 << 17),
    dict(fmt=FP8, K=(1 << 22) + 16), dict(xq=None), dict(sx=None), dict(wq=None), dict(sw=None),
    dict(y=None), dict(xq=P + 8), dict(wq=P + 8), dict(ldq=5104), dict(ldq=5128), dict(ldw=5104),
    dict(ldw=5128), dict(ldw=-2), dict(ldy=511), dict(sx=P + 2), dict(sw=P + 1), dict(y=P + 1),
    dict(ldw=0, K=5104), dict(ldq=(1 << 23) + 16), dict(ldw=(1 << 23) + 16), dict(ws=P + 8)])
def test_gemm_refuses(lib, bad):
    assert call(lib.w8_token_gemm, GEMM, **bad) == INVALID
    assert lib.w8_last_error()


def test_gemm_workspace_and_plan(lib, w8):
    need = w8.token_gemm_workspace_size("W8A8_INT8", 48, 512, 5120)
    assert need > 0
    assert call(lib.w8_token_gemm, GEMM, ws_bytes=need - 1) == WORKSPACE
    assert call(lib.w8_token_gemm, GEMM, ws=None) == WORKSPACE
    assert str(need).encode() in lib.w8_last_error()
    n = ctypes.c_size_t(7)
    size = lib.w8_token_gemm_workspace_size
    for args in ((BLOCK, 48, 512, 1024, 0), (INT8, -1, 512, 1024, 0), (INT8, 48, 512, 1000, 0),
                 (INT8, 48, 512, 1024, 2), (INT8, 48, 512, 1 << 17, 0)):
        assert size(*args, ctypes.byref(n)) == INVALID
    assert size(INT8, 48, 512, 1024, 0, None) == INVALID and n.value == 7
    assert size(INT8, 0, 512, 1024, 0, ctypes.byref(n)) == OK and n.value == 0
    for fmt in ("W8A8_INT8", "FP8_Dynamic"):
        assert w8.token_gemm_workspace_size(fmt, 8192, 8192, 8192) == 0
        assert w8.token_gemm_plan(fmt, 8192, 8192, 8192)["tile_m"] == 256
        p = w8.token_gemm_plan(fmt, 48, 512, 5120)
        assert p["split_k"] > 1 and p["workgroups"] > 0
        assert w8.token_gemm_plan(fmt, 1, 512, 1024)["tile_m"] == 0  # the small-M GEMM
    with pytest.raises(w8.W8Error, match="128"):
        w8.token_gemm_plan("FP8_Dynamic", 48, 512, 1040, packed=True)
    with pytest.raises(w8.W8Error, match="Block_FP8"):
        w8.token_gemm_plan("Block_FP8", 48, 512, 1024)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 22), dict(E=0), dict(E=1025, ldl=1025), dict(topk=0), dict(topk=33),
    dict(E=4, topk=5), dict(logits=None), dict(experts=None), dict(weights=None), dict(ldl=63),
    dict(fp32=2), dict(renormalize=2), dict(rows=None), dict(slots=None), dict(offsets=None),
    dict(offsets=None, rows=None), dict(logits=P + 2), dict(fp32=0, logits=P + 1),
    dict(experts=P + 2), dict(weights=P + 2), dict(offsets=P + 2), dict(rows=P + 2),
    dict(slots=P + 2), dict(ws=P + 8)])
def test_route_refuses(lib, bad):
    assert call(lib.w8_moe_route, ROUTE, **bad) == INVALID
    assert lib.w8_last_error()


def test_route_workspace(lib, w8):
    assert w8.moe_route_workspace_size(32, 128, 8) == 0  # 256 entries: one launch
    need = w8.moe_route_workspace_size(100, 64, 8)
    assert need > 0
    assert call(lib.w8_moe_route, ROUTE, ws_bytes=need - 1) == WORKSPACE
    assert call(lib.w8_moe_route, ROUTE, ws=None) == WORKSPACE
    assert w8.moe_route_workspace_size(0, 64, 8) == 0
    # several rounds of choices in one workgroup take two launches
    assert w8.moe_route_workspace_size(16, 1000, 8) == 0
    assert w8.moe_route_workspace_size(42, 1000, 6) > 0
    assert w8.moe_route_workspace_size(85, 256, 3) == w8.moe_route_workspace_size(256, 8, 1) == 0
    # the counts of at most 1024 workgroups, past the counter region
    assert w8.moe_route_workspace_size((1 << 22) - 1, 1024, 32) <= (2 << 20) + 1024 * 1024 * 4
    with pytest.raises(w8.W8Error, match="topk"):
        w8.moe_route_workspace_size(4, 8, 9)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=1 << 22), dict(topk=0), dict(topk=33), dict(D=0), dict(D=(1 << 20) + 1),
    dict(n_rows=-1), dict(y=None), dict(weights=None), dict(slots=None), dict(out=None),
    dict(ldy=99), dict(ldb=99), dict(ldo=99), dict(y=P + 1), dict(base=P + 1), dict(out=P + 1),
    dict(weights=P + 2), dict(slots=P + 2),
    dict(T=(1 << 22) - 1, D=1 << 20, ldy=1 << 20, ldb=1 << 20, ldo=1 << 20)])
def test_combine_refuses(lib, bad):
    assert call(lib.w8_moe_combine, COMBINE, **bad) == INVALID
    assert lib.w8_last_error()


@pytest.mark.parametrize("bad", [
    dict(fmt=3), dict(fmt=-1), dict(E=0), dict(E=1025), dict(T=-1), dict(topk=0), dict(topk=33),
    dict(D=0), dict(D=272, ldq=272), dict(I=144), dict(D=65536 + 128, ldq=65536 + 128), dict(I=65664),
    dict(fmt=INT8, D=264, ldq=272), dict(fmt=FP8, I=136), dict(xq=None), dict(sx=None),
    dict(experts=None), dict(weights=None), dict(w1=None), dict(s1=None), dict(w2=None),
    dict(s2=None), dict(y=None), dict(xq=P + 8), dict(ldq=240), dict(ldq=264), dict(ldy=255),
    dict(ldb=255), dict(base=P + 1),
    dict(sx=P + 2), dict(experts=P + 2), dict(weights=P + 1), dict(y=P + 1), dict(w1=P + 8),
    dict(w2=P + 8), dict(s1=P + 2), dict(s2=P + 2), dict(ldw1=240), dict(ldw1=264), dict(ldw1=-2),
    dict(ldw2=112), dict(ldw2=136), dict(w1_stride=256 * 256 - 16), dict(w1_stride=256 * 256 + 8),
    dict(w2_stride=256 * 128 - 16), dict(s1_stride=3), dict(s2_stride=1),
    dict(ldw1=0, w1_stride=256 * 256 - 16), dict(ws=P + 8)])
def test_layer_refuses(lib, bad):
    assert call(lib.w8_moe_layer, LAYER, **bad) == INVALID
    assert lib.w8_last_error()


def test_layer_window_and_workspace(lib, w8):
    assert call(lib.w8_moe_layer, LAYER, T=33) == UNSUPPORTED
    with pytest.raises(w8.UnsupportedShape):
        w8.moe_layer_workspace_size(33, 2, 256, 128)
    need = w8.moe_layer_workspace_size(8, 2, 256, 128)
    assert call(lib.w8_moe_layer, LAYER, ws_bytes=need - 1) == WORKSPACE
    assert call(lib.w8_moe_layer, LAYER, ws=None) == WORKSPACE
    assert w8.moe_layer_workspace_size(0, 2, 256, 128) == 0


def test_nothing_to_do(lib):
    """No tokens: fine without any buffer."""
    assert call(lib.w8_token_quantize, null(QUANT), M=0) == OK
    assert call(lib.w8_token_gemm, null(GEMM), M=0) == OK
    assert call(lib.w8_moe_route, null(ROUTE), T=0) == OK
    assert call(lib.w8_moe_combine, null(COMBINE), T=0, n_rows=0) == OK
    assert call(lib.w8_moe_layer, null(LAYER), T=0) == OK
    assert lib.w8_last_error() == b""


# ------------------------------------------------------------------ binding --
@pytest.fixture
def fake():
    """torch factories give tensors without memory on a device that need not exist."""
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        with FakeTensorMode():
            yield lambda *shape, dtype=torch.int8, device="cuda:0": torch.empty(
                *shape, dtype=dtype, device=device)


F32, I32, BF16 = torch.float32, torch.int32, torch.bfloat16


def test_binding_refuses_host_tensors(w8):
    x, q, s = torch.zeros(4, 256, dtype=BF16), torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4)
    i = torch.zeros(4, 2, dtype=I32)
    for f in (lambda: w8.token_quantize("W8A8_INT8", x), lambda: w8.token_gemm("W8A8_INT8", q, s, q, s),
              lambda: w8.moe_route(x, 2), lambda: w8.moe_combine(x, torch.zeros(4, 2), i),
              lambda: w8.moe_layer("W8A8_INT8", q, s, i, torch.zeros(4, 2), q[None], s, q[None], s)):
        with pytest.raises(TypeError, match="HIP"):
            f()


def test_binding_refuses_shapes_types_and_devices(w8, fake):
    T, E, k, D, I = 8, 4, 2, 256, 128
    xq, sx = fake(T, D), fake(T, dtype=F32)
    experts, weights = fake(T, k, dtype=I32), fake(T, k, dtype=F32)
    w1, s1, w2, s2 = fake(E, 2 * I, D), fake(E, 2 * I, dtype=F32), fake(E, D, I), fake(E, D, dtype=F32)

    def layer(**kw):
        a = dict(xq=xq, sx=sx, experts=experts, weights=weights, w1=w1, s1=s1, w2=w2, s2=s2)
        return w8.moe_layer("W8A8_INT8", **{**a, **kw})

    with pytest.raises(ValueError, match="experts"):
        layer(experts=fake(T + 1, k, dtype=I32))
    with pytest.raises(TypeError, match="int32"):
        layer(experts=fake(T, k, dtype=torch.int64))
    with pytest.raises(ValueError, match="weights"):
        layer(weights=fake(T, k + 1, dtype=F32))
    with pytest.raises(ValueError, match="scales of w1"):
        layer(s1=fake(E, 2 * I + 1, dtype=F32))
    with pytest.raises(ValueError, match="2 I"):
        layer(w1=fake(E, I, D), s1=fake(E, I, dtype=F32))
    with pytest.raises(ValueError, match="row stride"):
        layer(w2=fake(E, 1, I).expand(E, D, I))
    with pytest.raises(ValueError, match="unit inner"):
        layer(w2=fake(E, I, D).transpose(1, 2))
    with pytest.raises(ValueError, match="y must be"):
        layer(y=fake(T, D + 1, dtype=BF16))
    with pytest.raises(ValueError, match="base must be"):
        layer(base=fake(T + 1, D, dtype=BF16))
    with pytest.raises(ValueError, match="must be on"):
        layer(s2=fake(E, D, dtype=F32, device="cuda:1"))
    with pytest.raises(ValueError, match="must be on"):
        w8.token_gemm("W8A8_INT8", xq, sx, w2[0].t().contiguous(), fake(I, dtype=F32, device="cuda:1"))
    with pytest.raises(ValueError, match="row stride"):
        w8.token_gemm("W8A8_INT8", xq, sx, fake(1, D).expand(64, D), fake(64, dtype=F32))
    with pytest.raises(ValueError, match="K mismatch"):
        w8.token_gemm("W8A8_INT8", xq, sx, fake(64, 128), fake(64, dtype=F32))
    with pytest.raises(ValueError, match="sx"):
        w8.token_gemm("W8A8_INT8", xq, fake(T, 2, dtype=F32), fake(64, D), fake(64, dtype=F32))
    with pytest.raises(TypeError, match="bfloat16"):
        w8.token_quantize("W8A8_INT8", fake(T, D, dtype=F32))
    with pytest.raises(ValueError, match="gate"):
        w8.token_quantize("W8A8_INT8", fake(T, D, dtype=BF16), gate=fake(T, D + 8, dtype=BF16))
    with pytest.raises(TypeError, match="logits"):
        w8.moe_route(fake(T, E, dtype=torch.float16), k)
    for topk in (0, -1):
        with pytest.raises(w8.W8Error, match="topk"):
            w8.moe_route(fake(T, E, dtype=F32), topk)
    with pytest.raises(ValueError, match="slots"):
        w8.moe_combine(fake(16, D, dtype=BF16), weights, fake(T * k, dtype=I32))
    with pytest.raises(ValueError, match="base"):
        w8.moe_combine(fake(16, D, dtype=BF16), weights, experts, base=fake(T, D + 1, dtype=BF16))
