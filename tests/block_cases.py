"""Inputs and 64-bit references for the tests of the Block_FP8 operators for
any token count.  The references follow the formulas in numpy/torch float64 on
the CPU and use none of the library's code; codes fed to the GEMMs are drawn
directly (any finite E4M3FN code), so both sides start from the same bytes."""
import numpy as np
import torch

GROUP = 128
DEV = torch.device("cuda:0")


def groups(n):
    return -(-n // GROUP)


def e4m3_table():
    """Value of each E4M3FN code (NaN codes 0x7f and 0xff)."""
    v = np.empty(256)
    for c in range(256):
        sign, e, f = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        mag = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (e == 15 and f == 7) else sign * mag
    return v


E4M3 = e4m3_table()


def draw_codes(g, *shape):
    """Finite codes with normally distributed values, as a quantizer leaves them."""
    grid = np.sort(E4M3[np.isfinite(E4M3)])
    codes = np.argsort(E4M3)[:len(grid)].astype(np.uint8)
    x = np.clip(g.standard_normal(shape) * 100, -448, 448)
    return codes[np.clip(np.searchsorted(grid, x), 0, len(grid) - 1)]


def draw_scales(g, *shape):
    return (2.0 ** g.uniform(-12, -6, shape)).astype(np.float32)


def dequant_rows(q, s):
    K = q.shape[-1]
    return E4M3[q] * np.repeat(s.astype(np.float64), GROUP, axis=-1)[..., :K]


def dequant_blocks(q, s):
    N, K = q.shape[-2:]
    w = np.repeat(s.astype(np.float64), GROUP, axis=-2)[..., :N, :]
    return E4M3[q] * np.repeat(w, GROUP, axis=-1)[..., :K]


def assert_product(y, x, w, what=""):
    """y (bf16 [M, N]) against x . w^T in 64 bits.  The bound: bf16 rounds by
    at most 2^-8 of the value; the fp8 matrix instruction's sums are within
    2^-14 of the sum of |products| (the bound the small-M GEMM's accumulators
    are held to), which covers the fp32 sum over the groups (2^-24 per group,
    at most 2^6 groups here)."""
    Y, S = x @ w.T, np.abs(x) @ np.abs(w).T
    got = y.float().cpu().numpy().astype(np.float64)
    assert got.shape == Y.shape
    bad = ~(np.abs(got - Y) <= 2.0 ** -8 * 1.01 * np.abs(Y) + 2.0 ** -14 * 1.01 * S + 1e-38)
    assert not bad.any(), (f"{what}: {bad.sum()} of {Y.size} outside the bound, first at "
                           f"{np.argwhere(bad)[:4].tolist()}")


def assert_codes(q, s, v, dv, what=""):
    """Codes q and scales s of 64-bit values v whose computed counterparts are
    within dv (absolute): the scale within its group's largest relative
    change, and each code's value within half a step of v / s (the distance of
    a correct rounding) plus what dv moves."""
    M, K = v.shape
    G = groups(K)
    pad = ((0, 0), (0, G * GROUP - K))
    vp = np.pad(v, pad).reshape(M, G, GROUP)
    dp = np.pad(dv, pad).reshape(M, G, GROUP)
    amax = np.abs(vp).max(axis=2)
    S = np.where(amax > 0, amax / 448, 1.0)
    got_s = s.cpu().numpy().astype(np.float64)
    assert got_s.shape == (M, G)
    ds = dp.max(axis=2) / 448 + 2.0 ** -23 * S
    assert (np.abs(got_s - S) <= ds).all(), f"{what}: scales off by {np.abs(got_s - S).max()}"
    got = np.pad(E4M3[q.view(torch.uint8).cpu().numpy()], pad).reshape(M, G, GROUP)
    t = vp / S[:, :, None]
    dt = (dp + np.abs(t) * ds[:, :, None]) / S[:, :, None] + 2.0 ** -22 * np.abs(t)
    _, e = np.frexp(np.abs(t) + dt)
    step = 2.0 ** np.maximum(e - 4, -9).astype(np.float64)
    bad = ~(np.abs(got - t) <= step / 2 + dt)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} codes off, first at "
                           f"{np.argwhere(bad)[:4].tolist()}")


def bf16(a):
    """(device bf16 tensor, its values in 64 bits) of a numpy array."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


def on_device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def codes_on_device(q):
    return on_device(q).view(torch.float8_e4m3fn)


def rms(v, eps):
    return v / np.sqrt((v * v).mean(axis=-1, keepdims=True) + eps)
