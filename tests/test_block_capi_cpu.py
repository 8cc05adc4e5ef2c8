"""Argument checks of the Block_FP8 operators for any token count, without a
GPU: every refusal happens before the device is touched, and calls with
nothing to do return at once."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 0x1000  # a well-aligned address that no refused call reads


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


QUANT = dict(M=4, K=256, x=P, ldx=256, gate=P, ldg=256, xq=P, ldq=256, sx=P, stream=None)
NORM = dict(M=4, D=100, y=P, ldy=100, residual=P, ldr=100, fp32=0, post=P, gate=P, ldg=100,
            scale=1.0, weight=P, eps=1e-6, h=P, ldh=100, z=P, ldz=100, zq=P, ldq=112, sz=P,
            stream=None)
GEMM = dict(M=48, N=512, K=1024, xq=P, ldq=1024, sx=P, wq=P, ldw=1024, sw=P, y=P, ldy=512,
            ws=P, ws_bytes=1 << 40, stream=None)
GROUPED = dict(E=4, T=64, N=512, K=1024, xq=P, ldq=1024, sx=P, offsets=P, rows=P, n_rows=100,
               wq=P, ldw=1024, w_stride=512 * 1024, sw=P, sw_stride=32, y=P, ldy=512, stream=None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(M=1 << 22), dict(K=0), dict(K=-8), dict(K=132), dict(K=(1 << 22) + 8),
    dict(x=None), dict(xq=None), dict(sx=None), dict(x=P + 8), dict(ldx=248), dict(ldx=260),
    dict(gate=P + 2), dict(ldg=128), dict(ldg=257), dict(xq=P + 4), dict(ldq=248),
    dict(ldq=260), dict(sx=P + 2)])
def test_quantize_refuses(lib, bad):
    assert call(lib.w8_block_quantize, QUANT, **bad) == INVALID
    assert lib.w8_last_error()


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(M=1 << 22), dict(D=0), dict(fp32=2), dict(eps=-1.0), dict(eps=float("nan")),
    dict(y=None), dict(residual=None), dict(weight=None), dict(h=None), dict(z=None, zq=None),
    dict(sz=None), dict(ldy=99), dict(ldr=99), dict(ldh=99), dict(ldg=99), dict(ldz=99),
    dict(ldq=99), dict(y=P + 1), dict(residual=P + 1), dict(fp32=1, residual=P + 2),
    dict(fp32=1, h=P + 2), dict(weight=P + 1), dict(post=P + 1), dict(gate=P + 1),
    dict(z=P + 1), dict(sz=P + 2)])
def test_norm_refuses(lib, bad):
    assert call(lib.w8_residual_norm, NORM, **bad) == INVALID
    assert lib.w8_last_error()


def test_norm_row_length_limit(lib):
    wide = dict(ldy=40000, ldr=40000, ldg=40000, ldh=40000, ldz=40000, ldq=40000)
    assert call(lib.w8_residual_norm, NORM, D=32769, **wide) == UNSUPPORTED


GEMM_BAD = [
    dict(N=0), dict(N=(1 << 24) + 1), dict(K=8), dict(K=1032), dict(K=(1 << 22) + 16),
    dict(xq=None), dict(sx=None), dict(wq=None), dict(sw=None), dict(y=None), dict(xq=P + 8),
    dict(wq=P + 8), dict(ldq=1008), dict(ldq=1032), dict(ldw=1008), dict(ldw=1032),
    dict(ldw=-2), dict(ldy=511), dict(sx=P + 2), dict(sw=P + 1), dict(y=P + 1),
    dict(ldw=0, K=1008)]


@pytest.mark.parametrize("bad", GEMM_BAD + [dict(M=-1), dict(M=1 << 22), dict(ws=P + 8)])
def test_gemm_refuses(lib, bad):
    assert call(lib.w8_block_gemm, GEMM, **bad) == INVALID
    assert lib.w8_last_error()


@pytest.mark.parametrize("bad", GEMM_BAD + [
    dict(n_rows=-1), dict(n_rows=1 << 22), dict(E=0), dict(E=65537), dict(T=-1), dict(T=0),
    dict(offsets=None), dict(rows=None), dict(offsets=P + 2), dict(rows=P + 1),
    dict(w_stride=512 * 1024 - 16), dict(w_stride=512 * 1024 + 8), dict(sw_stride=31),
    dict(ldw=0, w_stride=512 * 1024 - 16)])
def test_grouped_refuses(lib, bad):
    assert call(lib.w8_grouped_gemm, GROUPED, **bad) == INVALID
    assert lib.w8_last_error()


def test_workspace(lib, w8):
    need = w8.block_gemm_workspace_size(48, 512, 1024)
    assert need > 0
    assert call(lib.w8_block_gemm, GEMM, ws_bytes=need - 1) == WORKSPACE
    assert call(lib.w8_block_gemm, GEMM, ws=None) == WORKSPACE
    assert str(need).encode() in lib.w8_last_error()
    n = ctypes.c_size_t(7)
    size = lib.w8_block_gemm_workspace_size
    for args in ((-1, 512, 1024, 0), (48, 0, 1024, 0), (48, 512, 1000, 0), (48, 512, 1024, 2)):
        assert size(*args, ctypes.byref(n)) == INVALID
    assert size(48, 512, 1024, 0, None) == INVALID and n.value == 7
    assert size(0, 512, 1024, 0, ctypes.byref(n)) == OK and n.value == 0
    # large products fill the GPU without splitting K
    assert w8.block_gemm_workspace_size(8192, 8192, 8192) == 0


def test_nothing_to_do(lib):
    """No rows: fine without any buffer."""
    null = lambda d, *keep: {k: (None if v == P else v) for k, v in d.items()}
    assert call(lib.w8_block_quantize, null(QUANT), M=0) == OK
    assert call(lib.w8_residual_norm, null(NORM), M=0) == OK
    assert call(lib.w8_block_gemm, null(GEMM), M=0) == OK
    assert call(lib.w8_grouped_gemm, null(GROUPED), n_rows=0, T=0) == OK
    assert lib.w8_last_error() == b""


def test_binding_refuses_host_tensors(w8):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q = torch.zeros(4, 256, dtype=torch.uint8)
    s = torch.zeros(4, 2)
    with pytest.raises(TypeError, match="HIP"):
        w8.block_quantize(x)
    with pytest.raises(TypeError, match="HIP"):
        w8.residual_norm(x, x, x[0])
    with pytest.raises(TypeError, match="HIP"):
        w8.block_gemm(q, s, q, s)
    with pytest.raises(TypeError, match="HIP"):
        w8.grouped_gemm(q, s, torch.zeros(2, dtype=torch.int32), q[None], s[None])


def test_strides_and_groups_limits(lib):
    """Beyond what the kernels' 32-bit offsets address."""
    for kw in (dict(ldq=(1 << 23) + 16), dict(ldw=(1 << 23) + 16)):
        assert call(lib.w8_block_gemm, GEMM, **kw) == INVALID
        assert call(lib.w8_grouped_gemm, GROUPED, w_stride=1 << 40, **kw) == INVALID
        assert b"2^23" in lib.w8_last_error()
    long = dict(M=1 << 17, K=1 << 21, ldx=1 << 21, ldg=1 << 21, ldq=1 << 21)
    assert call(lib.w8_block_quantize, QUANT, **long) == INVALID
    assert b"2^31" in lib.w8_last_error()
