"""The MoE operators and the token-scaled quantizer on the CPU, behind their C-ABI:
every launch's every workgroup, with each buffer against a page that cannot be
touched, so that a load outside it fails even where its value is not used.  What
the lanes of a wavefront leave for each other in LDS is read only where the
kernels say so, whichever workgroup runs first."""
import os

import numpy as np
import pytest
import torch

from tests.kernel_host import moe as host
from tests.test_gpu_moe_layer import FORMATS, Layer, sized
from tests.test_gpu_route import check as check_route
from tests.test_gpu_route import route as exact_route
from tests.token_cases import assert_codes, bf16_bits, quantized

pytestmark = pytest.mark.skipif(not os.path.exists(host.CLANG), reason="no clang")


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return host.build(str(tmp_path_factory.mktemp("moe")))


def as_bf16(bits):
    return torch.from_numpy(bits.astype(np.int16)).view(torch.bfloat16)


def values(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def run(lib, c, **kw):
    y, wrong = host.layer(lib, c.fmt, c.xq, c.sx, c.experts, c.weights, c.w1, c.s1, c.w2, c.s2,
                          pack=host.pack, **kw)
    assert wrong is None, wrong
    return y


# -------------------------------------------------------------------- layer --
SIZES = [  # T, E, topk, D, I (Block_FP8: rounded up to whole 128s)
    # few entries: a wave each, several, chunks of I, of one token and of several
    (1, 1, 1, 16, 16), (1, 128, 8, 80, 48), (1, 8, 8, 16, 3360), (2, 4, 1, 48, 2064), (1, 2, 2, 32, 8208),
    (4, 60, 2, 144, 336), (8, 1000, 1, 32, 32),
    # the experts' slots: entries, or the experts that have tokens
    (5, 64, 3, 80, 144), (9, 3, 2, 144, 272), (17, 2, 1, 64, 400), (32, 40, 4, 80, 32),
    # the first projection by whole waves
    (5, 64, 3, 144, 848),
    # hidden codes made in chunks, in parts of I, apart
    (6, 1, 1, 64, 7200), (9, 1, 1, 80, 2064), (9, 1, 1, 64, 4112), (20, 2, 2, 64, 800), (31, 1, 1, 48, 4208)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,topk,D,I", SIZES)
def test_layer(lib, fmt, T, E, topk, D, I):
    c = Layer(fmt, T, min(E, 100) if fmt == "Block_FP8" else E, topk, *sized(fmt, D, I))
    c.check(as_bf16(run(lib, c)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,topk,D,I", [(1, 4, 2, 48, 144), (9, 3, 2, 144, 272), (9, 1, 1, 64, 4112),
                                          (20, 2, 1, 64, 1232)])
def test_orders_and_beginnings(lib, fmt, T, E, topk, D, I):
    """The last workgroup first, and buffers that begin behind a page's end: the same bits."""
    c = Layer(fmt, T, E, topk, *sized(fmt, D, I))
    y = run(lib, c)
    assert (run(lib, c, descending=True) == y).all()
    assert (run(lib, c, at_end=False) == y).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("packed", [(True, False), (False, True)])
@pytest.mark.parametrize("T,D,I", [(1, 80, 144), (9, 144, 272), (20, 80, 912)])
def test_packed_weights(lib, fmt, packed, T, D, I):
    c = Layer(fmt, T, 3, 2, *sized(fmt, D, I))
    assert (run(lib, c, packed=packed) == run(lib, c)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("experts", [[[2, -1, 2], [9, 9, 9]], [[-1, -5, 1 << 30]],
                                     [[0, 1, 0], [-1, -1, -1], [2, 2, 2], [1, 0, 3], [3, 3, 2]] * 2])
def test_choices_left_out_and_repeated(lib, fmt, experts):
    c = Layer(fmt, len(experts), 3, 3, *sized(fmt, 80, 144), experts=experts)
    c.check(as_bf16(run(lib, c)))
    base = bf16_bits(np.random.default_rng(1).standard_normal((c.T, c.D)))
    got = values(run(lib, c, base=base)).astype(np.float64)
    y, room = c.expected()
    want = y + values(base)
    assert (np.abs(got - want) <= room + 1.01 * 2.0 ** -8 * np.abs(want)).all()


# ------------------------------------------------------------------ routing --
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,topk,ld", [
    (1, 1, 1, 1), (3, 5, 5, 5), (8, 128, 8, 128), (17, 130, 3, 131), (16, 200, 4, 200),
    (9, 300, 6, 304), (2, 1024, 32, 1024), (42, 1000, 6, 1001), (300, 16, 2, 16), (130, 60, 4, 64),
    (700, 9, 1, 9)])
def test_route(lib, dtype, T, E, topk, ld):
    g = np.random.default_rng([T, E, topk])
    l = (g.standard_normal((T, E)) * 2).astype(np.float32)
    l[T // 2, : E // 2] = -np.inf
    l[T // 3, E // 3:] = np.nan
    logits = l
    if dtype == "bf16":
        logits = bf16_bits(l)
        l = values(logits)
    for renorm, descending, at_end in ((True, False, True), (False, True, False)):
        got, wrong = host.route(lib, logits, topk, renorm, 1.5, ld=ld, descending=descending,
                                at_end=at_end)
        assert wrong is None, wrong
        check_route([torch.from_numpy(v) for v in got], exact_route(l, topk, renorm, 1.5))
    pair, wrong = host.route(lib, logits, topk, ld=ld, lists=False)
    assert wrong is None and (pair[0] == got[0]).all()


# -------------------------------------------------- combination, quantizer --
@pytest.mark.parametrize("T,topk,D,n", [(1, 1, 1, 1), (3, 2, 7, 4), (5, 9, 8, 11), (2, 8, 129, 16),
                                        (9, 3, 2056, 20), (1, 32, 4100, 3), (4, 2, 100, 0)])
@pytest.mark.parametrize("base", [False, True])
def test_combine(lib, T, topk, D, n, base):
    g = np.random.default_rng([T, topk, D])
    y, b = bf16_bits(g.standard_normal((n, D))), bf16_bits(g.standard_normal((T, D)))
    w = g.uniform(0, 1, (T, topk)).astype(np.float32)
    slots = g.integers(-3, n + 3, (T, topk))
    on = (slots >= 0) & (slots < n)
    rows = np.concatenate([values(y), np.zeros((1, D), np.float32)])[np.where(on, slots, n)]
    each = rows.astype(np.float64) * w[:, :, None]
    want, size = each.sum(axis=1), np.abs(each).sum(axis=1)
    if base:
        want, size = want + values(b), size + np.abs(values(b))
    for kw in (dict(), dict(at_end=False), dict(in_place=True)):
        if not base and kw.get("in_place"):
            continue
        got, wrong = host.combine(lib, y, w, slots, b if base else None, **kw)
        assert wrong is None, wrong
        # fp32 sums of topk + 1 terms, each within 2^-24 of what it reaches, and the rounding
        room = 2.0 ** -8 * np.abs(want) + (topk + 2) * 2.0 ** -23 * size
        assert (np.abs(values(got) - want) <= room).all()


@pytest.mark.parametrize("fmt", ["W8A8_INT8", "FP8_Dynamic"])
@pytest.mark.parametrize("M,K", [(1, 8), (5, 136), (6, 512), (3, 520), (1, 8200), (2, 24584)])
def test_quantize(lib, fmt, M, K):
    g = np.random.default_rng([M, K])
    x, gate = (bf16_bits(g.standard_normal((M, K)) * 3) for _ in range(2))
    for at_end in (True, False):
        q, s, wrong = host.quantize(lib, fmt, x, at_end=at_end)
        assert wrong is None, wrong
        want, want_s = quantized(fmt, values(x))
        np.testing.assert_array_equal(s, want_s)
        np.testing.assert_array_equal(q, want)
        q, s, wrong = host.quantize(lib, fmt, x, gate, at_end=at_end)
        assert wrong is None, wrong
        v = values(gate).astype(np.float64)
        v = v / (1 + np.exp(-v)) * values(x)
        assert_codes(fmt, q, s, v, np.abs(v) * 2.0 ** -20)


# ------------------------------------------------------------- the harness --
def test_an_access_outside_is_seen(lib):
    """A row stride that reaches past the last row, in front of the first."""
    x = bf16_bits(np.ones((4, 256)))
    for at_end, offset in ((True, 8), (False, -8)):
        b = host.Buffers(lib, at_end)
        p = b.put("x", x).value + 2 * offset
        q, s = b.put("xq", np.zeros((4, 256), np.uint8)), b.put("sx", np.zeros(4, np.float32))
        rc = lib.emu_quantize(0, 1, 4, 256, host.ctypes.c_void_p(p), host._i64(256), None,
                              host._i64(0), 0, q, host._i64(256), s)
        assert rc == 3 and "access at x" in lib.emu_text().decode()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,I", [(1, 144), (9, 272), (32, 800)])
def test_every_array_of_the_layer_is_read_to_its_end(lib, fmt, T, I):
    """An array that is an element short is one that a kernel reads past."""
    D, I = sized(fmt, 80, I)
    c = Layer(fmt, T, 2, 2, D, I, experts=[[0, 1]] * T)
    base = bf16_bits(np.ones((T, D)))
    for name in ("xq", "sx", "experts", "weights", "w1", "s1", "w2", "s2", "base"):
        _, wrong = host.layer(lib, fmt, c.xq, c.sx, c.experts, c.weights, c.w1, c.s1, c.w2, c.s2,
                              base=base, short=name)
        assert wrong and f"access at {name} " in wrong, (name, wrong)


def test_a_refusal_is_a_refusal(lib):
    c = Layer("W8A8_INT8", 2, 2, 1, 32, 32)
    y, wrong = host.layer(lib, c.fmt, c.xq, c.sx, c.experts, c.weights, c.w1, c.s1, c.w2, c.s2, pad=8)
    assert "ldq % 16" in wrong and (y == host.GUARD * 257).all()
