"""The Block_FP8 GEMM for any M and the grouped GEMM on the GPU, against the
product of the dequantized codes in 64 bits: sizes around the kernels' tiles,
ragged K groups, strides, both weight layouts, split K, ragged and empty
experts, repeated and clamped rows."""
import numpy as np
import pytest
import torch

from tests.block_cases import (DEV, assert_product, codes_on_device, dequant_blocks,
                               dequant_rows, draw_codes, draw_scales, groups, on_device)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


class Gemm:
    def __init__(self, M, N, K, seed=0):
        print(f"[case] M={M} N={N} K={K}", flush=True)
        g = np.random.default_rng([seed, M, N, K])
        self.M, self.N, self.K = M, N, K
        self.xq, self.sx = draw_codes(g, M, K), draw_scales(g, M, groups(K))
        self.wq, self.sw = draw_codes(g, N, K), draw_scales(g, groups(N), groups(K))
        self.x, self.w = dequant_rows(self.xq, self.sx), dequant_blocks(self.wq, self.sw)
        self.dev = [codes_on_device(self.xq), on_device(self.sx), codes_on_device(self.wq),
                    on_device(self.sw)]


SHAPES = [
    (1, 1, 16), (1, 128, 128), (2, 17, 48), (7, 130, 272), (16, 256, 1024), (17, 129, 1040),
    (31, 896, 1024), (33, 512, 640), (48, 300, 2048), (64, 257, 144), (65, 640, 896),
    (127, 128, 7168), (128, 129, 128), (129, 1000, 384), (200, 5, 2064), (255, 255, 1536),
    (256, 256, 256), (257, 513, 400), (700, 384, 128), (1000, 1100, 272),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(w8, M, N, K):
    c = Gemm(M, N, K)
    assert_product(w8.block_gemm(*c.dev), c.x, c.w, "row-major")
    if K % 128 == 0:
        wp = w8.pack_weight("Block_FP8", c.dev[2])
        assert_product(w8.block_gemm(c.dev[0], c.dev[1], wp, c.dev[3]), c.x, c.w, "packed")


@pytest.mark.parametrize("M,N,K", [(3900, 3200, 640), (8200, 1600, 272), (5000, 3600, 1040),
                                   (5000, 4500, 1040)])
def test_product_many_tiles(w8, M, N, K):
    """Enough tiles to run several per compute unit, with last rounds that run
    in halves and quarters of a tile; checked on sampled rows."""
    c = Gemm(M, N, K)
    y = w8.block_gemm(*c.dev)
    rows = np.unique(np.r_[0, M - 1, np.random.default_rng(1).integers(0, M, 300)])
    assert_product(y[torch.from_numpy(rows).to(DEV)], c.x[rows], c.w)


@pytest.mark.parametrize("M,N,K", [(1, 256, 256), (40, 130, 512), (300, 257, 272)])
def test_strides(w8, M, N, K):
    """Padded rows of every operand, and an output whose rows start unaligned;
    what lies between the rows is left alone."""
    c = Gemm(M, N, K)
    xq = codes_on_device(np.pad(c.xq, ((0, 0), (0, 48)), constant_values=0x7F))[:, :K]
    wq = codes_on_device(np.pad(c.wq, ((0, 0), (0, 16)), constant_values=0x7F))[:, :K]
    for pad, first in ((3, 1), (4, 4)):
        buf = torch.full((M, N + first + pad), 7.0, dtype=torch.bfloat16, device=DEV)
        y = w8.block_gemm(xq, c.dev[1], wq, c.dev[3], y=buf[:, first:first + N])
        assert_product(y, c.x, c.w)
        assert (buf[:, :first] == 7).all() and (buf[:, first + N:] == 7).all()


def test_zero_rows(w8):
    c = Gemm(1, 64, 128)
    y = w8.block_gemm(c.dev[0][:0], c.dev[1][:0], c.dev[2], c.dev[3])
    assert y.shape == (0, 64)


def test_deterministic_and_shared_workspace(w8):
    """Split-K shapes repeat bit for bit, on one workspace shared with the
    small-M GEMM, and with one of their own on another stream."""
    ws = w8.Workspace(DEV)
    cases = [Gemm(48, 512, 7168), Gemm(100, 256, 2048)]
    small = Gemm(8, 512, 7168)
    first = [w8.block_gemm(*c.dev, workspace=ws) for c in cases]
    s0 = w8.gemm_w8a8("Block_FP8", *small.dev, workspace=ws)
    assert w8.block_gemm_workspace_size(48, 512, 7168) > 0
    for _ in range(3):
        for c, y in zip(cases, first):
            assert torch.equal(w8.block_gemm(*c.dev, workspace=ws), y)
        assert torch.equal(w8.gemm_w8a8("Block_FP8", *small.dev, workspace=ws), s0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = [w8.block_gemm(*c.dev, workspace=w8.Workspace(DEV, 64 << 20), stream=st)
             for c in cases]
    st.synchronize()
    for c, y, o in zip(cases, first, other):
        assert torch.equal(o, y)
        assert_product(y, c.x, c.w)


def test_nan_scale_reaches_its_row_only(w8):
    c = Gemm(70, 200, 512)
    c.dev[1][33, 2] = float("nan")
    y = w8.block_gemm(*c.dev)
    assert torch.isnan(y[33]).all()
    keep = [i for i in range(70) if i != 33]
    assert_product(y[keep], c.x[keep], c.w)


def test_graph_capture(w8):
    c = Gemm(48, 512, 2048)
    ws = w8.Workspace(DEV, max(256, w8.block_gemm_workspace_size(48, 512, 2048)))
    eager = w8.block_gemm(*c.dev, workspace=ws)
    y = torch.empty_like(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w8.block_gemm(*c.dev, y=y, workspace=ws)
    for _ in range(4):
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
        assert torch.equal(w8.block_gemm(*c.dev, workspace=ws), eager)


# ------------------------------------------------------------------ grouped --
class Grouped:
    def __init__(self, counts, N, K, T=None, seed=0):
        print(f"[case] counts={counts} N={N} K={K} T={T}", flush=True)
        E, n = len(counts), sum(counts)
        g = np.random.default_rng([seed, E, n, N, K])
        self.E, self.n = E, n
        self.offsets = np.r_[0, np.cumsum(counts)].astype(np.int32)
        self.rows = None if T is None else g.integers(0, T, n).astype(np.int32)
        xr = n if T is None else T
        self.xq, self.sx = draw_codes(g, xr, K), draw_scales(g, xr, groups(K))
        self.wq, self.sw = draw_codes(g, E, N, K), draw_scales(g, E, groups(N), groups(K))
        self.x, self.w = dequant_rows(self.xq, self.sx), dequant_blocks(self.wq, self.sw)
        self.dev = [codes_on_device(self.xq), on_device(self.sx), on_device(self.offsets),
                    codes_on_device(self.wq), on_device(self.sw)]
        self.drows = None if T is None else on_device(self.rows)

    def check(self, y):
        for e in range(self.E):
            lo, hi = self.offsets[e], self.offsets[e + 1]
            if lo < hi:
                at = np.arange(lo, hi) if self.rows is None else self.rows[lo:hi]
                assert_product(y[int(lo):int(hi)], self.x[at], self.w[e], f"expert {e}")


COUNTS = [
    ([1], 16, 16, None), ([5, 0, 3], 130, 272, 4), ([0, 0, 1, 0], 64, 128, 9),
    ([16, 17, 15, 1, 0, 33], 256, 512, None), ([32] * 8, 300, 384, 40),
    ([0, 200, 1, 0, 64, 65, 0], 257, 640, 100), ([129, 0, 500], 384, 400, None),
    ([300, 5, 128, 0, 270], 130, 256, 700), ([1000], 256, 128, 3),
    ([2] * 70 + [0] * 60 + [9] * 3, 128, 128, 50), ([700, 900, 0, 513], 512, 272, 1000),
]


@pytest.mark.parametrize("counts,N,K,T", COUNTS)
def test_grouped(w8, counts, N, K, T):
    c = Grouped(counts, N, K, T)
    c.check(w8.grouped_gemm(*c.dev, rows=c.drows))
    if K % 128 == 0:
        experts = w8.pack_experts("Block_FP8", c.dev[3])
        xq, sx, off, _, sw = c.dev
        c.check(w8.grouped_gemm(xq, sx, off, experts, sw, rows=c.drows))


@pytest.mark.parametrize("counts,N,K", [
    ([1100, 1030, 1279, 991], 1280, 144),         # one round, all of it in halves
    ([3400, 3329, 3300, 3571], 1280, 128),        # a full round and a rest in quarters
    ([2600, 2000, 2305, 1, 0, 2561], 1800, 272),  # a full round and a rest in halves
    ([600, 0, 0, 0, 0, 0, 0, 0], 2560, 256)])     # one round, all of it in quarters
def test_grouped_last_round_in_pieces(w8, counts, N, K):
    c = Grouped(counts, N, K, 600)
    c.check(w8.grouped_gemm(*c.dev, rows=c.drows))


def test_grouped_equals_dense_per_expert(w8):
    """Bit for bit: with four groups K is not split, and every tile shape adds
    the groups in the same order."""
    c = Grouped([300, 0, 270], 384, 512)
    y = w8.grouped_gemm(*c.dev)
    xq, sx, _, wq, sw = c.dev
    for e in (0, 2):
        lo, hi = int(c.offsets[e]), int(c.offsets[e + 1])
        assert torch.equal(y[lo:hi], w8.block_gemm(xq[lo:hi], sx[lo:hi], wq[e], sw[e]))


def test_grouped_no_entries(w8):
    c = Grouped([3, 2], 64, 128, T=4)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    y = w8.grouped_gemm(c.dev[0], c.dev[1], off, c.dev[3], c.dev[4],
                        rows=torch.empty(0, dtype=torch.int32, device=DEV))
    assert y.shape == (0, 64)


def test_grouped_bad_routing_stays_inside(w8):
    """Offsets and rows outside the arrays are clamped: nothing outside y's
    rows is written, and well-routed entries are right."""
    c = Grouped([40, 24], 130, 256, T=20)
    off = c.dev[2].clone()
    off[2] = 1 << 20          # past the end: clamped to n_rows
    rows = c.drows.clone()
    rows[0], rows[1] = -5, 1 << 30
    buf = torch.full((c.n + 8, 130), 7.0, dtype=torch.bfloat16, device=DEV)
    w8.grouped_gemm(c.dev[0], c.dev[1], off, c.dev[3], c.dev[4], rows=rows, y=buf[4:4 + c.n])
    assert (buf[:4] == 7).all() and (buf[4 + c.n:] == 7).all()
    c.rows = c.rows.copy()
    c.rows[0], c.rows[1] = 0, 19
    c.check(buf[4:4 + c.n])


def test_grouped_strided_experts(w8):
    """Experts inside a larger buffer with padded rows."""
    c = Grouped([9, 70], 96, 272, T=30)
    buf = np.full((2, 100, 304), 0x7F, dtype=np.uint8)
    buf[:, :96, :272] = c.wq
    wq = codes_on_device(buf)[:, :96, :272]
    c.check(w8.grouped_gemm(c.dev[0], c.dev[1], c.dev[2], wq, c.dev[4], rows=c.drows))


# ------------------------------------------------------- past 32-bit offsets --
def test_output_past_32_bit_offsets(w8):
    """An output of more than 2^32 bytes: its last rows and columns."""
    M, N, K = 66000, 33000, 128
    c = Gemm(16, N, K)
    x, s = c.dev[0].view(torch.uint8).repeat(M // 16, 1), c.dev[1].repeat(M // 16, 1)
    y = w8.block_gemm(x, s, c.dev[2], c.dev[3])
    assert y.shape == (M, N)
    assert_product(y[-16:], c.x, c.w)
    assert_product(y[32768:32784], c.x, c.w)


def test_weights_and_tokens_past_32_bit_offsets(w8):
    """Weight rows and gathered token rows more than 2^32 bytes from the first."""
    K, far = 8192, 540000
    c = Gemm(300, 256, K)
    big = torch.zeros(far, K, dtype=torch.uint8, device=DEV)
    scales = torch.ones(far, K // 128, device=DEV)
    big[-300:], scales[-300:] = c.dev[0].view(torch.uint8), c.dev[1]
    rows = torch.arange(far - 300, far, dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    y = w8.grouped_gemm(big, scales, offsets, c.dev[2][None], c.dev[3][None], rows=rows)
    assert_product(y, c.x, c.w, "tokens")
    del scales
    # the same codes as weights, the last 256 rows of 540000
    big[-256:] = c.dev[2].view(torch.uint8)
    sw = torch.ones(far // 128 + 1, K // 128, device=DEV)
    sw[-3:] = c.dev[3][0]  # (the last rows start inside a scale block)
    y = w8.block_gemm(c.dev[0][:40], c.dev[1][:40], big, sw)
    w = dequant_blocks(c.wq, np.repeat(c.sw[:1], 2, axis=0))
    assert_product(y[:, -256:], c.x[:40], w, "weights")
