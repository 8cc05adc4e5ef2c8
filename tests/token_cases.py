"""Inputs and references for the tests of the token-scaled operators (W8A8_INT8,
FP8_Dynamic) for any token count, from the formulas, on the CPU and with none of
the library's code."""
import numpy as np
import torch

from tests.block_cases import E4M3, draw_codes

QMAX = {"W8A8_INT8": 127.0, "FP8_Dynamic": 448.0}
FORMATS = list(QMAX)


def codes(g, fmt, *shape):
    """Codes as bytes: any int8 (-128 too), or finite E4M3FN as a quantizer leaves them."""
    if fmt == "W8A8_INT8":
        return g.integers(-128, 128, shape).astype(np.int8).view(np.uint8)
    return draw_codes(g, *shape)


def values(fmt, q):
    """The values of codes in 64 bits."""
    return q.view(np.int8).astype(np.float64) if fmt == "W8A8_INT8" else E4M3[q]


def scales(g, n):
    return (2.0 ** g.uniform(-12, -6, n)).astype(np.float32)


def bf16_bits(v):
    """fp32 rounded to bf16 (nearest, ties to even), as bits."""
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16).view(
        torch.int16).numpy().view(np.uint16)


def int8_product(xq, sx, wq, sw):
    """The W8A8_INT8 GEMM's bits: exact sums (below 2^53 in float64), their fp32
    value times sx, times sw, each rounded, then bf16."""
    acc = values("W8A8_INT8", xq) @ values("W8A8_INT8", wq).T
    return bf16_bits(acc.astype(np.float32) * sx[:, None] * sw[None, :])


def assert_product(fmt, got_bits, xq, sx, wq, sw, what=""):
    """W8A8_INT8: bit for bit.  FP8_Dynamic: a bf16 rounding (2^-8 of the value,
    half a step), and sums within 2^-14 of the sum of |products| (the bound that
    the fp8 matrix instructions are held to in the Block_FP8 tests), which covers
    the fp32 sums over the steps and the two scale products (2^-24 each)."""
    if fmt == "W8A8_INT8":
        want = int8_product(xq, sx, wq, sw)
        bad = got_bits != want
    else:
        x, w = values(fmt, xq) * sx[:, None], values(fmt, wq) * sw[:, None]
        x, w = x.astype(np.float64), w.astype(np.float64)
        Y, S = x @ w.T, np.abs(x) @ np.abs(w).T
        got = (got_bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        bad = ~(np.abs(got - Y) <= 2.0 ** -8 * 1.01 * np.abs(Y) + 2.0 ** -14 * 1.01 * S + 1e-38)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, at {np.argwhere(bad)[:4].tolist()}"


def bits_of(y):
    return y.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def quantized(fmt, v):
    """(codes as bytes, scales) of fp32 rows, in fp32 as the definition has it:
    s = amax / Qmax, codes of x / s to the nearest, ties to even."""
    v = np.ascontiguousarray(v, dtype=np.float32)
    amax = np.abs(v).max(axis=1)
    s = np.where(amax == 0, np.float32(1), (amax / np.float32(QMAX[fmt])).astype(np.float32))
    t = (v / s[:, None]).clip(-QMAX[fmt], QMAX[fmt])
    if fmt == "W8A8_INT8":
        return np.rint(t).astype(np.int8).view(np.uint8), s
    return torch.from_numpy(t).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), s


def assert_codes(fmt, q, s, v, dv, what=""):
    """Codes (bytes) and scales of 64-bit rows v whose computed counterparts are
    within dv: the scale within its row's largest change and two roundings
    (2^-23 of it), each code's value within half a step of v / s plus what dv
    and the scale move, and a rounding of the quotient (2^-22 of it)."""
    top = QMAX[fmt]
    amax = np.abs(v).max(axis=1)
    S = np.where(amax > 0, amax / top, 1.0)
    ds = dv.max(axis=1) / top + 2.0 ** -23 * S
    assert (np.abs(s.astype(np.float64) - S) <= ds).all(), f"{what}: scales"
    t = v / S[:, None]
    dt = (dv + np.abs(t) * ds[:, None]) / S[:, None] + 2.0 ** -22 * np.abs(t)
    step = 1.0
    if fmt != "W8A8_INT8":
        _, e = np.frexp(np.abs(t) + dt)
        step = 2.0 ** np.maximum(e - 4, -9).astype(np.float64)
    bad = ~(np.abs(values(fmt, q) - t) <= step / 2 + dt)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, at {np.argwhere(bad)[:4].tolist()}"
