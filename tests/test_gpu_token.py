"""The token-scaled quantizer and tiled GEMM on the GPU: W8A8_INT8 products and
ungated codes bit for bit, the rest against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from tests.block_cases import DEV, bf16, on_device
from tests.token_cases import (FORMATS, QMAX, assert_codes, assert_product, bits_of, codes,
                               quantized, scales, values)
from tests.token_plans import SHAPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


def typed(fmt, q):
    return q.view(torch.int8 if fmt == "W8A8_INT8" else torch.float8_e4m3fn)


def code_bytes(q):
    return q.contiguous().view(torch.uint8).cpu().numpy()


# ----------------------------------------------------------------- quantize --
SIZES = [(1, 8), (1, 128), (3, 136), (5, 512), (6, 520), (33, 768), (5, 2048), (300, 1040),
         (1, 7168), (2, 8192), (3, 8200), (1, 16384), (2, 32768), (2, 40008), (1, 100000),
         (4100, 264), (1050, 2056), (1024, 4104), (1, 16392), (3, 20480)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", SIZES)
def test_quantize(w8, fmt, M, K):
    """Ungated: the definition in fp32, bit for bit."""
    print(f"[case] {fmt} M={M} K={K}", flush=True)
    g = np.random.default_rng([M, K])
    x, v = bf16(g.standard_normal((M, K)) * 2.0 ** g.integers(-40, 40, (M, 1)))
    q, s = w8.token_quantize(fmt, x)
    want, want_s = quantized(fmt, v)
    assert q.dtype == typed(fmt, q).dtype and s.shape == (M,)
    np.testing.assert_array_equal(s.cpu().numpy(), want_s)
    np.testing.assert_array_equal(code_bytes(q), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", SIZES)
def test_quantize_gated(w8, fmt, M, K):
    print(f"[case] {fmt} M={M} K={K}", flush=True)
    g = np.random.default_rng([M, K, 1])
    both, v = bf16(g.standard_normal((M, 2 * K)) * 3)
    q, s = w8.token_quantize(fmt, both[:, K:], gate=both[:, :K])
    want = v[:, :K] / (1 + np.exp(-v[:, :K])) * v[:, K:]
    # the gated product: exponential, reciprocal and two products, each within
    # 2^-22 of its result
    assert_codes(fmt, code_bytes(q), s.cpu().numpy(), want, np.abs(want) * 2.0 ** -20)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_matches_small_m_quantizer(w8, fmt):
    g = np.random.default_rng(5)
    x, _ = bf16(g.standard_normal((32, 1040)) * 2.0 ** g.integers(-120, 60, (32, 1)))
    x[3] = 0
    q, s = w8.token_quantize(fmt, x)
    q0, s0 = w8.quantize_act(fmt, x)
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 264), (50, 1040), (700, 2048), (3, 40008)])
def test_reciprocal_scales_are_torchs(w8, fmt, M, K):
    """Codes and scales as torch computes them on the GPU, bit for bit."""
    x = torch.randn(M, K, generator=torch.Generator("cuda").manual_seed(M), device=DEV).bfloat16()
    x[0] = 0
    q, s = w8.token_quantize(fmt, x, reciprocal=True)
    amax = x.float().abs().amax(dim=1)
    want_s = torch.where(amax == 0, torch.ones_like(amax), amax / QMAX[fmt])
    t = (x.float() / want_s[:, None]).clamp(-QMAX[fmt], QMAX[fmt])
    want = t.round().to(torch.int8) if fmt == "W8A8_INT8" else t.to(torch.float8_e4m3fn)
    assert torch.equal(s, want_s)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("K,at", [(384, 200), (2048, 2047), (40000, 39999)])
def test_nonfinite_rows_stay_nonfinite(w8, fmt, bad, K, at):
    x = torch.ones(3, K, dtype=torch.bfloat16, device=DEV)
    x[1, at] = bad
    q, s = w8.token_quantize(fmt, x)
    assert torch.isfinite(s).tolist() == [True, False, True]
    with np.errstate(invalid="ignore"):
        v = values(fmt, code_bytes(q)) * s.cpu().numpy().astype(np.float64)[:, None]
    assert not np.isfinite(v[1, at])
    np.testing.assert_allclose(v[[0, 2]], 1.0, rtol=1e-6)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_edges(w8, fmt):
    q, s = w8.token_quantize(fmt, torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0,)
    q, s = w8.token_quantize(fmt, torch.zeros(2, 256, dtype=torch.bfloat16, device=DEV))
    assert (q.view(torch.uint8) == 0).all() and (s == 1).all()
    # rows that the GEMMs take, on whole lines where they are long
    for K, ld in ((8, 16), (504, 512), (496, 496), (512, 512), (520, 640), (7248, 7296)):
        x, v = bf16(np.random.default_rng(K).standard_normal((3, K)))
        q, s = w8.token_quantize(fmt, x)
        assert q.stride() == (ld, 1)
        np.testing.assert_array_equal(code_bytes(q), quantized(fmt, v)[0])
        q, s = w8.token_quantize(fmt, x, stream=torch.cuda.current_stream())
        assert q.stride() == (ld, 1)
    # from a wider buffer into a wider buffer: the columns beside stay
    for K in (256, 1040, 9000):
        both, v = bf16(np.random.default_rng(0).standard_normal((5, K + 24)))
        buf = torch.full((7, K + 16), 0x55, dtype=torch.uint8, device=DEV)
        out = typed(fmt, buf)[1:6, :K]
        _, s = w8.token_quantize(fmt, both[:, 16:16 + K], xq=out)
        want, _ = quantized(fmt, v[:, 16:16 + K])
        np.testing.assert_array_equal(buf[1:6, :K].cpu().numpy(), want)
        assert (buf[:, K:] == 0x55).all() and (buf[0] == 0x55).all() and (buf[6] == 0x55).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_gate_extremes(w8, fmt):
    """Gates far out on both sides: silu(g) = g above, 0 below."""
    gates = np.array([-1e30, -200, -104, -89, -88, -87, -60, -1e-30, 0, 1e-30, 30, 88, 89, 200,
                      1e4, 1e6])
    gate, gv = bf16(np.tile(gates, (16, 1)) * (np.arange(16) == np.arange(16)[:, None]))
    x, xv = bf16(np.full((16, 16), 0.5))
    q, s = w8.token_quantize(fmt, x, gate=gate)
    with np.errstate(over="ignore"):
        want = gv / (1 + np.exp(-gv)) * xv
    # The product is fp32: below 2^-150, half its smallest number, it is 0, and a
    # row of zeros has the scale 1.  (-200 exp(-200) / 2 = 2^-282)
    want[np.abs(want) < 2.0 ** -150] = 0
    assert_codes(fmt, code_bytes(q), s.cpu().numpy(), want, np.abs(want) * 2.0 ** -20 + 1e-37)


# --------------------------------------------------------------------- GEMM --
class Gemm:
    def __init__(self, fmt, M, N, K):
        print(f"[case] {fmt} M={M} N={N} K={K}", flush=True)
        g = np.random.default_rng([M, N, K])
        self.fmt = fmt
        self.host = (codes(g, fmt, M, K), scales(g, M), codes(g, fmt, N, K), scales(g, N))
        self.dev = [on_device(c) for c in self.host]
        self.dev[0], self.dev[2] = typed(fmt, self.dev[0]), typed(fmt, self.dev[2])

    def check(self, y, rows=None):
        """All rows, or of many the ones at the tiles' borders and some others."""
        xq, sx, wq, sw = self.host
        M = len(xq)
        if rows is None:
            rows = np.arange(M) if M <= 700 else np.unique(np.r_[
                np.arange(0, M, 64), np.arange(63, M, 64), M - 1,
                np.random.default_rng(1).integers(0, M, 200)])
        assert_product(self.fmt, bits_of(y[torch.from_numpy(rows).to(DEV)]), xq[rows], sx[rows], wq,
                       sw)


def tile(p):
    return p["tile_m"], p["tile_n"]



@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", SHAPES)
def test_gemm(w8, fmt, shape):
    M, N, K, packed = shape
    p = w8.token_gemm_plan(fmt, M, N, K, packed=packed)
    assert (tile(p), p["split_k"], p["parts"]) == SHAPES[shape]
    c = Gemm(fmt, M, N, K)
    if packed:
        c.dev[2] = w8.pack_weight(fmt, c.dev[2])
    buf = torch.full((M + 2, N + 5), 7.0, dtype=torch.bfloat16, device=DEV)
    y = w8.token_gemm(fmt, *c.dev, y=buf[1:1 + M, 1:1 + N])
    c.check(y)
    assert (buf[:, 0] == 7).all() and (buf[:, 1 + N:] == 7).all()
    assert (buf[0] == 7).all() and (buf[M + 1] == 7).all()
    assert torch.equal(w8.token_gemm(fmt, *c.dev), y)


def test_every_tile_and_split_gives_the_same_int8_bits(w8):
    """Exact sums: whichever kernel runs, the first rows are the same."""
    c = Gemm("W8A8_INT8", 4000, 4200, 4128)
    xq, sx, wq, sw = c.dev
    first = w8.token_gemm("W8A8_INT8", *c.dev)[:20]
    c.check(first, np.arange(20))
    plans = set()
    for M in (20, 33, 48, 70, 100, 150, 300, 500, 700, 930, 1000, 1500, 2500, 3300):
        p = w8.token_gemm_plan("W8A8_INT8", M, 4200, 4128)
        plans.add((tile(p), p["split_k"], p["parts"]))
        assert torch.equal(w8.token_gemm("W8A8_INT8", xq[:M], sx[:M], wq, sw)[:20], first), p
    assert len(plans) >= 6, plans


def test_int8_extremes(w8):
    """The largest sums that int32 holds: codes of -128 over the longest K."""
    K = 131056
    x = torch.full((40, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((64, K), -128, dtype=torch.int8, device=DEV)
    x[1::2] = 127
    s = torch.ones(64, device=DEV)
    y = w8.token_gemm("W8A8_INT8", x, s[:40], w, s)
    want = torch.tensor([128.0 * 128 * K, -127.0 * 128 * K]).to(torch.bfloat16)
    assert torch.equal(y.cpu(), want.repeat(20)[:, None].expand(40, 64))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [5, 40, 300])
def test_nonfinite_scales_stay_in_their_rows(w8, fmt, M):
    """A token whose scale is not finite (a row with a NaN or an infinity)."""
    c = Gemm(fmt, M, 256, 512)
    want = w8.token_gemm(fmt, *c.dev)
    sx = c.dev[1].clone()
    sx[2], sx[3] = float("nan"), float("inf")
    y = w8.token_gemm(fmt, c.dev[0], sx, *c.dev[2:])
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[3]).any()
    keep = [m for m in range(M) if m not in (2, 3)]
    assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("fmt", FORMATS)
def test_strided_operands(w8, fmt):
    """Row strides beyond K on both sides, and no rows at all."""
    c = Gemm(fmt, 200, 300, 272)
    wide_x = torch.full((200, 320), 0x7F, dtype=torch.uint8, device=DEV)
    wide_w = torch.full((300, 288), 0x7F, dtype=torch.uint8, device=DEV)
    wide_x[:, 16:288] = c.dev[0].view(torch.uint8)
    wide_w[:, :272] = c.dev[2].view(torch.uint8)
    x, w = typed(fmt, wide_x)[:, 16:288], typed(fmt, wide_w)[:, :272]
    assert torch.equal(w8.token_gemm(fmt, x, c.dev[1], w, c.dev[3]), w8.token_gemm(fmt, *c.dev))
    assert w8.token_gemm(fmt, x[:0], c.dev[1][:0], w, c.dev[3]).shape == (0, 300)


@pytest.mark.parametrize("fmt", FORMATS)
def test_capture_streams_and_overlap(w8, fmt):
    """Split calls replayed from a graph, on two streams at once without a
    workspace, and afterwards: the same bits."""
    c = Gemm(fmt, 48, 512, 7168)
    assert w8.token_gemm_workspace_size(fmt, 48, 512, 7168) > 0
    alone = w8.token_gemm(fmt, *c.dev, workspace=w8.Workspace(DEV, 64 << 20))
    c.check(alone)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [w8.token_gemm(fmt, *c.dev, y=torch.empty_like(alone), stream=st)
           for _ in range(10) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(y, alone) for y in got)
    y, ws = torch.empty_like(alone), w8.Workspace(DEV, 64 << 20)
    x = torch.randn(48, 7168, device=DEV).bfloat16()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w8.token_gemm(fmt, *c.dev, y=y, workspace=ws)
        q, s = w8.token_quantize(fmt, x)
    eager = w8.token_quantize(fmt, x)
    for _ in range(4):
        y.fill_(float("nan"))
        s.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, alone) and torch.equal(w8.token_gemm(fmt, *c.dev), alone)
        assert torch.equal(s, eager[1]) and torch.equal(q.view(torch.uint8),
                                                        eager[0].view(torch.uint8))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 5, 40, 700])
def test_feed_forward(w8, fmt, T):
    """The operators as a dense layer uses them: codes of the tokens, gate and up
    projection, codes of silu(gate) * up, down projection."""
    D, I = 512, 1360
    g = np.random.default_rng([T, D])
    x, xv = bf16(g.standard_normal((T, D)))
    w1, s1, w2, s2 = (codes(g, fmt, 2 * I, D), scales(g, 2 * I) * np.float32(0.02),
                      codes(g, fmt, D, I), scales(g, D))
    d = [on_device(a) for a in (w1, s1, w2, s2)]
    xq, sx = w8.token_quantize(fmt, x)
    both = w8.token_gemm(fmt, xq, sx, typed(fmt, d[0]), d[1])
    aq, sa = w8.token_quantize(fmt, both[:, I:], gate=both[:, :I])
    y = w8.token_gemm(fmt, aq, sa, typed(fmt, d[2]), d[3])
    # each step against the one before as the library left it
    q0, s0 = quantized(fmt, xv)
    np.testing.assert_array_equal(code_bytes(xq), q0)
    assert_product(fmt, bits_of(both), q0, s0, w1, s1, "gate and up")
    b = both.double().cpu().numpy()
    v = b[:, :I] / (1 + np.exp(-b[:, :I])) * b[:, I:]
    assert_codes(fmt, code_bytes(aq), sa.cpu().numpy(), v, np.abs(v) * 2.0 ** -20, "gated codes")
    assert_product(fmt, bits_of(y), code_bytes(aq), sa.cpu().numpy(), w2, s2, "down")
