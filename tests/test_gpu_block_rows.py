"""The residual norm and the gated 1 x 128 quantizer on the GPU against their
formulas in 64 bits."""
import numpy as np
import pytest
import torch

from tests.block_cases import (DEV, E4M3, assert_codes, bf16, dequant_rows, groups, on_device,
                               rms)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


# ----------------------------------------------------------------- quantize --
def silu(g):
    return g / (1 + np.exp(-g))


@pytest.mark.parametrize("M,K", [(1, 8), (1, 128), (3, 136), (33, 768), (5, 2048), (300, 1040),
                                 (1, 16384), (2000, 264)])
@pytest.mark.parametrize("gated", [False, True])
def test_quantize(w8, M, K, gated):
    g = np.random.default_rng([M, K, gated])
    both, v = bf16(g.standard_normal((M, 2 * K)) * 3)
    gate, x = both[:, :K], both[:, K:]
    q, s = w8.block_quantize(x, gate=gate if gated else None)
    want = silu(v[:, :K]) * v[:, K:] if gated else v[:, K:]
    # the gated product: exponential, reciprocal and two products, each within
    # 2^-22 of its result
    assert_codes(q, s, want, np.abs(want) * (2.0 ** -20 if gated else 0.0))


def test_quantize_matches_small_m_quantizer(w8):
    """Ungated codes and scales are quantize_act's, bit for bit."""
    g = np.random.default_rng(5)
    x, _ = bf16(g.standard_normal((32, 1024)) * 2.0 ** g.integers(-60, 60, (32, 1)))
    x[3, 128:256] = 0
    q, s = w8.block_quantize(x)
    q0, s0 = w8.quantize_act("Block_FP8", x)
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)


def test_gate_extremes(w8):
    """Gates far out on both sides: silu(g) = g above, 0 below."""
    gates = np.array([-1e30, -200, -104, -89, -88, -87, -60, -1e-30, 0, 1e-30, 30, 88, 89, 200,
                      1e4, 1e6])
    gate, gv = bf16(np.tile(gates, 8)[None, :])
    x, xv = bf16(np.full((1, 128), 0.5))
    q, s = w8.block_quantize(x, gate=gate)
    with np.errstate(over="ignore"):
        want = silu(gv) * xv
    assert_codes(q, s, want, np.abs(want) * 2.0 ** -20 + 1e-37)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_groups_stay_nonfinite(w8, bad):
    x = torch.ones(2, 384, dtype=torch.bfloat16, device=DEV)
    x[1, 200] = bad
    q, s = w8.block_quantize(x)
    ok = torch.isfinite(s)
    assert ok.tolist() == [[True] * 3, [True, False, True]]
    v = dequant_rows(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy())
    assert not np.isfinite(v[1, 200])
    np.testing.assert_allclose(v[1, :128], 1.0, rtol=1e-6)


def test_quantize_edges(w8):
    q, s = w8.block_quantize(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0, 1)
    z = torch.zeros(2, 256, dtype=torch.bfloat16, device=DEV)
    q, s = w8.block_quantize(z)
    assert (q.view(torch.uint8) == 0).all() and (s == 1).all()
    # written through a wider buffer: the columns beside stay
    buf = torch.full((5, 272), 0x55, dtype=torch.uint8, device=DEV)
    x, v = bf16(np.random.default_rng(0).standard_normal((5, 256)))
    out = buf.view(torch.float8_e4m3fn)[:, :256]
    _, s = w8.block_quantize(x, xq=out)
    assert_codes(out, s, v, 0 * v)
    assert (buf[:, 256:] == 0x55).all()


# --------------------------------------------------------------------- norm --
def norm_case(M, D, rdtype, post, gate, seed=0, spread=1.0):
    g = np.random.default_rng([seed, M, D])
    y, yv = bf16(g.standard_normal((M, D)) * spread)
    r = (4 * g.standard_normal((M, D))).astype(np.float32)
    if rdtype == "bf16":
        r, rv = bf16(r)
    else:
        r, rv = on_device(r), r.astype(np.float64)
    w, wv = bf16(1 + 0.1 * g.standard_normal(D))
    pw, pv = bf16(1 + 0.1 * g.standard_normal(D))
    gt, gv = bf16(g.standard_normal(D if gate == "channel" else (M, D)))
    kw = dict(post_weight=pw if post else None, gate=None if gate == "none" else gt)
    b = rms(yv, 1e-6) * pv if post else yv
    if gate != "none":
        b = b * gv
    h = rv + 0.7 * b
    z = rms(h, 1e-6) * wv
    # fp32 rounding before the last one: a few 2^-24 of each term of h (the
    # branch's has up to five factors, the root's with a sum of D terms in
    # chunks below 2^7 long), moved into z by its factor w / rms
    dh = 2.0 ** -20 * (np.abs(rv) + np.abs(0.7 * b))
    dz = 2.0 ** -19 * np.abs(z) + dh * np.abs(z / np.where(h == 0, 1, h)) \
        + dh * np.abs(wv) / np.sqrt((h * h).mean(axis=-1, keepdims=True) + 1e-6)
    return y, r, w, kw, h, z, dh, dz


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.abs(got - want).max()}"


SIZES = [(1, 1), (3, 7), (1, 64), (5, 129), (33, 512), (2, 513), (4, 1000), (7, 2048), (3, 2056),
         (1, 4096), (2, 5120), (9, 7168), (1, 8192), (2, 8199), (1, 16384), (2, 20000),
         (1, 32768), (1030, 256)]


@pytest.mark.parametrize("M,D", SIZES)
@pytest.mark.parametrize("rdtype,post,gate", [("bf16", False, "none"), ("fp32", True, "token"),
                                              ("bf16", True, "channel")])
def test_residual_norm(w8, M, D, rdtype, post, gate):
    print(f"[case] M={M} D={D} {rdtype} {post} {gate}", flush=True)
    y, r, w, kw, h, z, dh, dz = norm_case(M, D, rdtype, post, gate)
    r0 = r.clone()
    gh, gz = w8.residual_norm(y, r, w, scale=0.7, eps=1e-6, **kw)
    rh = 2.0 ** -8 if rdtype == "bf16" else 2.0 ** -24
    near(gh, h, dh + rh * 1.01 * np.abs(h) + 1e-38, "h")
    near(gz, z, dz + 2.0 ** -8 * 1.01 * np.abs(z) + 1e-38, "z")
    assert torch.equal(r, r0) and gh.dtype == r.dtype
    gh2, zq, sz = w8.residual_norm(y, r, w, scale=0.7, eps=1e-6, quantize=True, **kw)
    assert torch.equal(gh2, gh)
    assert_codes(zq, sz, z, dz, "codes")
    gh3, zq3, sz3, gz3 = w8.residual_norm(y, r, w, scale=0.7, eps=1e-6, quantize=True,
                                          with_z=True, **kw)
    assert torch.equal(gh3, gh) and torch.equal(gz3, gz) and torch.equal(sz3, sz)
    assert torch.equal(zq3.view(torch.uint8), zq.view(torch.uint8))


@pytest.mark.parametrize("M,D", [(3, 8), (5, 9), (2, 15), (600, 2057), (530, 5003), (3, 9001),
                                 (2, 20007)])
@pytest.mark.parametrize("rdtype,post,gate", [("bf16", False, "none"), ("fp32", True, "token")])
def test_residual_norm_short_last_chunk(w8, M, D, rdtype, post, gate):
    test_residual_norm(w8, M, D, rdtype, post, gate)


@pytest.mark.parametrize("D", [520, 1003, 2051])
def test_in_place_without_post_norm(w8, D):
    """No barrier stands between a row's loads and the stores of h over them."""
    y, r, w, kw, h, z, dh, dz = norm_case(700, D, "fp32", False, "none")
    gh, gz = w8.residual_norm(y, r, w, scale=0.7, eps=1e-6, h=r, **kw)
    assert gh is r
    near(gh, h, dh + 2.0 ** -24 * 1.01 * np.abs(h) + 1e-38, "h")
    near(gz, z, dz + 2.0 ** -8 * 1.01 * np.abs(z) + 1e-38, "z")


def test_in_place_and_strides(w8):
    """h written over the residual, rows inside wider buffers whose other
    columns stay, odd strides."""
    M, D = 6, 1000
    y, r, w, kw, h, z, dh, dz = norm_case(M, D, "bf16", True, "token")

    def wide(t, left, right):
        buf = torch.full((M, left + D + right), 3.0, dtype=t.dtype, device=DEV)
        buf[:, left:left + D] = t
        return buf, buf[:, left:left + D]

    _, yv = wide(y, 1, 2)
    rbuf, rv = wide(r, 3, 4)
    zbuf, zv = wide(torch.zeros_like(y), 5, 0)
    kw["gate"] = wide(kw["gate"], 7, 1)[1]
    gh, gz = w8.residual_norm(yv, rv, w, scale=0.7, eps=1e-6, h=rv, out=zv, **kw)
    near(gh, h, dh + 2.0 ** -8 * 1.01 * np.abs(h), "h")
    near(gz, z, dz + 2.0 ** -8 * 1.01 * np.abs(z), "z")
    assert (rbuf[:, :3] == 3).all() and (rbuf[:, 3 + D:] == 3).all() and (zbuf[:, :5] == 3).all()


def test_norm_zero_rows_and_zero_values(w8):
    D = 256
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    e = torch.empty(0, D, dtype=torch.bfloat16, device=DEV)
    h, z = w8.residual_norm(e, e, w)
    assert h.shape == z.shape == (0, D)
    o = torch.zeros(3, D, dtype=torch.bfloat16, device=DEV)
    h, zq, sz = w8.residual_norm(o, o, w, post_weight=w, quantize=True)
    assert (h == 0).all() and (zq.view(torch.uint8) == 0).all() and (sz == 1).all()


def test_norm_nan_stays_in_its_row(w8):
    y, r, w, kw, h, z, dh, dz = norm_case(5, 600, "fp32", False, "none")
    y[2, 17] = float("nan")
    gh, gz = w8.residual_norm(y, r, w, scale=0.7)
    assert torch.isnan(gz[2]).all() and torch.isnan(gh[2, 17])
    keep = [0, 1, 3, 4]
    near(gz[keep], z[keep], dz[keep] + 2.0 ** -8 * 1.01 * np.abs(z[keep]), "z")


def test_rows_past_32_bit_offsets(w8):
    """Rows whose elements and codes lie more than 2^32 bytes from the first:
    the same results as on their own."""
    M, K = 70000, 65536
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn(3, K, device=DEV).bfloat16()
    q, s = w8.block_quantize(x)
    q0, s0 = w8.block_quantize(x[-3:].contiguous())
    assert torch.equal(q[-3:].view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s[-3:], s0)
    del q, s
    x = x.view(-1, 16384)
    w = torch.ones(16384, dtype=torch.bfloat16, device=DEV)
    h, z = w8.residual_norm(x, x, w)
    h0, z0 = w8.residual_norm(x[-12:].contiguous(), x[-12:].contiguous(), w)
    assert torch.equal(h[-12:], h0) and torch.equal(z[-12:], z0)
