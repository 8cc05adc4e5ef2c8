"""Every kernel of the Block_FP8 GEMMs on the GPU, by the shapes that the
library's plan gives it (block_plans.py), against the product of the
dequantized codes in 64 bits."""
import numpy as np
import pytest
import torch

from tests.block_cases import (DEV, GROUP, assert_product, codes_on_device, dequant_blocks,
                               dequant_rows, draw_codes, draw_scales, groups, on_device)
from tests.block_plans import DENSE, EVERY_TILE, GROUPED, LARGE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


def draw_weights(g, N, K):
    """Codes [N, K]: rows of a prime number of different ones, in turn."""
    return draw_codes(g, min(N, 509), K)[np.arange(N) % 509]


class Gemm:
    def __init__(self, M, N, K):
        print(f"[case] M={M} N={N} K={K}", flush=True)
        g = np.random.default_rng([M, N, K])
        self.xq, self.sx = draw_codes(g, M, K), draw_scales(g, M, groups(K))
        self.wq, self.sw = draw_weights(g, N, K), draw_scales(g, groups(N), groups(K))
        self.dev = [codes_on_device(self.xq), on_device(self.sx), codes_on_device(self.wq),
                    on_device(self.sw)]

    def check(self, y, rows=None):
        """All rows, or of many the ones at the tiles' borders and some others."""
        M = len(self.xq)
        if rows is None:
            rows = np.arange(M) if M <= 700 else np.unique(np.r_[
                np.arange(0, M, 64), np.arange(63, M, 64), M - 1,
                np.random.default_rng(1).integers(0, M, 200)])
        assert_product(y[torch.from_numpy(rows).to(DEV)],
                       dequant_rows(self.xq[rows], self.sx[rows]),
                       dequant_blocks(self.wq, self.sw))


def tile(p):
    return p["tile_m"], p["tile_n"]


@pytest.mark.parametrize("shape", DENSE)
def test_dense(w8, shape):
    M, N, K, packed = shape
    p = w8.block_gemm_plan(M, N, K, packed=packed)
    assert (tile(p), p["split_k"], p["parts"]) == DENSE[shape]
    c = Gemm(M, N, K)
    if packed:
        c.dev[2] = w8.pack_weight("Block_FP8", c.dev[2])
    buf = torch.full((M, N + 5), 7.0, dtype=torch.bfloat16, device=DEV)
    y = w8.block_gemm(*c.dev, y=buf[:, 1:1 + N])
    c.check(y)
    assert (buf[:, 0] == 7).all() and (buf[:, 1 + N:] == 7).all()
    again = w8.block_gemm(*c.dev)
    assert torch.equal(again, y)


@pytest.mark.parametrize("K", [272, 384])
def test_every_tile_adds_the_groups_in_the_same_order(w8, K):
    """Bit for bit: the first rows of each product, K not split."""
    M = max(EVERY_TILE)
    c = Gemm(M, 4200, K)
    xq, sx, wq, sw = c.dev
    first = w8.block_gemm(xq[:40], sx[:40], wq, sw)
    c.check(first, np.arange(40))
    for rows, (t, parts) in EVERY_TILE.items():
        p = w8.block_gemm_plan(rows, 4200, K)
        assert (tile(p), p["split_k"], p["parts"]) == (t, 1, parts)
        assert torch.equal(w8.block_gemm(xq[:rows], sx[:rows], wq, sw)[:40], first), t


@pytest.mark.parametrize("counts,N,K,T,t", GROUPED)
def test_grouped(w8, counts, N, K, T, t):
    E, n = len(counts), sum(counts)
    assert tile(w8.grouped_gemm_plan(E, T or n, N, K, n_rows=n)) == t
    print(f"[case] counts={counts} N={N} K={K} T={T}", flush=True)
    g = np.random.default_rng([E, n, N, K])
    off = np.r_[0, np.cumsum(counts)].astype(np.int32)
    rows = None if T is None else g.integers(0, T, n).astype(np.int32)
    xq, sx = draw_codes(g, T or n, K), draw_scales(g, T or n, groups(K))
    wq = np.stack([draw_weights(g, N, K) for _ in counts])
    sw = draw_scales(g, E, groups(N), groups(K))
    x = dequant_rows(xq, sx)
    dev = [codes_on_device(xq), on_device(sx), on_device(off)]
    drows = None if rows is None else on_device(rows)

    def check(experts):
        y = w8.grouped_gemm(*dev, experts, on_device(sw), rows=drows)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            at = np.arange(lo, hi)
            if hi - lo > 700:
                at = np.unique(np.r_[at[::64], at[63::64], at[-1], g.choice(at, 200)])
            assert_product(y[torch.from_numpy(at).to(DEV)], x[at if rows is None else rows[at]],
                           dequant_blocks(wq[e], sw[e]), f"expert {e}")

    codes = codes_on_device(wq)
    check(codes)
    if K % GROUP == 0:
        check(w8.pack_experts("Block_FP8", codes))


# ------------------------------------------------------- past 32-bit offsets --
def strided(codes, stride):
    """The codes as rows `stride` bytes apart (what lies between is never read)."""
    buf = torch.empty(len(codes), stride, dtype=torch.uint8, device=DEV)
    buf[:, :codes.shape[1]] = on_device(codes)
    return buf.view(torch.float8_e4m3fn)[:, :codes.shape[1]]


def test_rows_at_the_longest_stride(w8):
    """2^23 bytes between rows of both operands in the largest tile: offsets
    inside a tile near 2^31, bases past 2^34."""
    M, N, K = 2568, 3090, 64
    assert tile(w8.block_gemm_plan(M, N, K)) == LARGE
    c = Gemm(M, N, K)
    c.dev[0], c.dev[2] = strided(c.xq, 1 << 23), strided(c.wq, 1 << 23)
    c.check(w8.block_gemm(*c.dev))


@pytest.mark.parametrize("T,t", [(4095, LARGE), (4096, (128, 128))])
def test_gathered_rows_around_4_gib(w8, T, t):
    """Up to 2^32 bytes from the first row to the last the largest tile
    addresses gathered rows by 32-bit offsets, beyond another tile by pointers."""
    stride, n, N, K = 1 << 20, 4200, 2100, 256
    assert tile(w8.grouped_gemm_plan(1, T, N, K, n_rows=n, ldq=stride)) == t
    c = Gemm(T, N, K)
    rows = np.random.default_rng(2).permutation(np.r_[np.arange(T), np.full(n - T, T - 1)])
    off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    y = w8.grouped_gemm(strided(c.xq, stride), c.dev[1], off, c.dev[2][None], c.dev[3][None],
                        rows=on_device(rows.astype(np.int32)))
    at = np.unique(np.r_[np.arange(0, n, 37), np.argsort(rows)[-300:]])
    assert_product(y[torch.from_numpy(at).to(DEV)], dequant_rows(c.xq[rows[at]], c.sx[rows[at]]),
                   dequant_blocks(c.wq, c.sw))
