"""The MoE layer of a few tokens on the GPU, against the formulas in 64 bits with
every rounding that the definition has, and against the separate operators."""
import numpy as np
import pytest
import torch

from tests.block_cases import (DEV, E4M3, GROUP, dequant_blocks, dequant_rows, draw_codes,
                               draw_scales, groups, on_device)
from tests.token_cases import QMAX, codes, scales, values

pytestmark = pytest.mark.gpu

FORMATS = ["W8A8_INT8", "FP8_Dynamic", "Block_FP8"]


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


class Layer:
    """T tokens over E experts; experts: [T, topk] ids (default: drawn without
    repetition)."""

    def __init__(self, fmt, T, E, topk, D, I, experts=None, seed=0):
        print(f"[case] {fmt} T={T} E={E} topk={topk} D={D} I={I}", flush=True)
        g = np.random.default_rng([seed, T, E, topk, D, I])
        self.fmt, self.T, self.E, self.topk, self.D, self.I = fmt, T, E, topk, D, I
        if experts is None:
            experts = np.stack([g.permutation(E)[:topk] for _ in range(T)])
        self.experts = np.asarray(experts, dtype=np.int32).reshape(T, topk)
        self.weights = g.uniform(0.05, 1, (T, topk)).astype(np.float32)
        draw = draw_codes if fmt != "W8A8_INT8" else lambda g, *s: codes(g, fmt, *s)
        self.xq, self.w1, self.w2 = draw(g, T, D), draw(g, E, 2 * I, D), draw(g, E, D, I)
        # scales that leave the gate and up values of order 1
        one = 1 / (80 * 80 * D ** 0.5)
        if fmt == "Block_FP8":
            self.sx = g.uniform(0.5, 2, (T, groups(D))).astype(np.float32)
            self.s1 = (one * g.uniform(0.5, 2, (E, groups(2 * I), groups(D)))).astype(np.float32)
            self.s2 = draw_scales(g, E, groups(D), groups(I))
        else:
            self.sx = g.uniform(0.5, 2, T).astype(np.float32)
            self.s1 = (one * g.uniform(0.5, 2, (E, 2 * I))).astype(np.float32)
            self.s2 = scales(g, (E, D))

    def args(self, w8, packed=(False, False)):
        t = torch.int8 if self.fmt == "W8A8_INT8" else torch.float8_e4m3fn
        w = [on_device(a).view(t) for a in (self.w1, self.w2)]
        w = [w8.pack_experts(self.fmt, a) if p else a for a, p in zip(w, packed)]
        return (self.fmt, on_device(self.xq).view(t), on_device(self.sx), on_device(self.experts),
                on_device(self.weights), w[0], on_device(self.s1), w[1], on_device(self.s2))

    def _rows(self, q, s):
        return dequant_rows(q, s) if self.fmt == "Block_FP8" else \
            values(self.fmt, q) * s.astype(np.float64)[:, None]

    def _weights(self, q, s):
        return dequant_blocks(q, s) if self.fmt == "Block_FP8" else \
            values(self.fmt, q) * s.astype(np.float64)[:, None]

    def _codes(self, v, dv):
        """(dequantized codes of v, how far each may be from what a computed v
        within dv gives): a value whose quotient is within reach of a rounding's
        border may go to either side of it, and the scale moves with its group's
        largest value."""
        top = QMAX.get(self.fmt, 448.0)
        width = GROUP if self.fmt == "Block_FP8" else v.shape[1]
        p, dp = v.reshape(len(v), -1, width), dv.reshape(len(v), -1, width)
        amax = np.abs(p).max(axis=2, keepdims=True)
        s = np.where(amax > 0, amax / top, 1.0)
        ds = dp.max(axis=2, keepdims=True) / top + 2.0 ** -23 * s
        t = p / s
        dt = (dp + np.abs(t) * ds) / s + 2.0 ** -22 * np.abs(t)

        def code(u):
            if self.fmt == "W8A8_INT8":
                return np.clip(np.rint(u), -top, top)
            _, e = np.frexp(u)
            step = 2.0 ** np.maximum(e - 4, -9).astype(np.float64)
            return np.clip(np.round(u / step) * step, -top, top)

        q, lo, hi = code(t), code(t - dt), code(t + dt)
        dq = np.maximum(np.abs(hi - q), np.abs(q - lo)) * s + np.abs(q) * ds
        return (q * s).reshape(v.shape), dq.reshape(v.shape)

    def expected(self):
        """(y in 64 bits, a bound of the computed value's distance)."""
        x = self._rows(self.xq, self.sx)
        y, room = np.zeros((self.T, self.D)), np.zeros((self.T, self.D))
        # the matrix instructions' sums: int8 exact, fp8 within 2^-14 of the sum
        # of |products| (the bound of the GEMMs' tests); then two scale products
        unit = 2.0 ** -22 if self.fmt == "W8A8_INT8" else 2.0 ** -14 * 1.01
        for e in np.unique(self.experts[(self.experts >= 0) & (self.experts < self.E)]):
            t = np.flatnonzero((self.experts == e).any(axis=1))
            w1, w2 = self._weights(self.w1[e], self.s1[e]), self._weights(self.w2[e], self.s2[e])
            a = x[t] @ w1.T
            da = unit * (np.abs(x[t]) @ np.abs(w1).T if unit > 2.0 ** -20 else np.abs(a))
            g, u, dg, du = a[:, :self.I], a[:, self.I:], da[:, :self.I], da[:, self.I:]
            silu = g / (1 + np.exp(-g))
            v = silu * u
            # |silu'| <= 1.1; the gated product within 2^-20 of its value
            dv = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(v)
            q, dq = self._codes(v, dv)
            p = q @ w2.T
            dp = dq @ np.abs(w2).T + unit * (np.abs(q) @ np.abs(w2).T + dq @ np.abs(w2).T)
            wt = np.where(self.experts[t] == e, self.weights[t], 0).astype(np.float64).sum(axis=1)
            y[t] += wt[:, None] * p
            room[t] += wt[:, None] * (dp + 2.0 ** -19 * np.abs(p))
        return y, room + 1.01 * 2.0 ** -8 * np.abs(y) + 1e-38

    def check(self, got, what=""):
        y, room = self.expected()
        got = got.double().cpu().numpy()
        bad = ~(np.abs(got - y) <= room)
        assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size}, at {np.argwhere(bad)[:4].tolist()}, "
                               f"worst {np.abs(got - y).max()} of {np.abs(y).max()}")
        # and the bound itself is tight enough to say something
        assert np.linalg.norm(got - y) <= 2.0 ** -6 * np.linalg.norm(y) + 1e-30


SIZES = [  # T, E, topk, D, I (Block_FP8: rounded up to whole 128s)
    (1, 1, 1, 16, 16), (1, 8, 2, 128, 128), (1, 128, 8, 256, 128), (2, 5, 3, 272, 144),
    (3, 4, 4, 80, 336), (5, 16, 2, 1040, 48), (8, 128, 8, 256, 128), (16, 4, 2, 528, 256),
    (17, 2, 1, 64, 400), (31, 3, 2, 144, 1680), (32, 2, 2, 256, 272), (32, 64, 8, 128, 64),
    (32, 1000, 32, 32, 32), (4, 8, 2, 2048, 768), (32, 1, 1, 256, 2064), (2, 3, 2, 64, 8192),
    (8, 3, 2, 64, 7200), (16, 2, 1, 144, 3472), (5, 9, 9, 64, 16), (1, 40, 16, 64, 3600),
    (1, 8, 1, 272, 9008), (1, 2, 2, 1024, 4096), (2, 64, 8, 144, 1552), (4, 64, 3, 64, 528),
    (1, 5, 5, 80, 50000), (4, 2, 2, 272, 2064), (8, 3, 1, 64, 128), (2, 4, 4, 144, 4208),
    # the second projection in parts, the first by whole waves
    (1, 8, 8, 144, 3360), (6, 4, 2, 80, 4112), (5, 3, 3, 64, 2064), (32, 2, 1, 64, 8208),
    (8, 60, 6, 128, 512), (20, 64, 8, 144, 336), (3, 2, 2, 64, 9008),
    # the hidden codes by a launch of their own; by the tiles, in chunks
    (32, 2, 2, 64, 400), (20, 2, 1, 80, 2064), (6, 1, 1, 64, 2064), (32, 40, 1, 64, 3968)]


def sized(fmt, D, I):
    return (D, I) if fmt != "Block_FP8" else (groups(D) * GROUP, groups(I) * GROUP)


def workspace_of_nan(w8, c):
    """NaN behind the counters (the smallest layer's are followed by four arrays of
    256 bytes), so that what is read without having been written shows."""
    ws = w8.Workspace(DEV, w8.moe_layer_workspace_size(c.T, c.topk, c.D, c.I))
    ws.buf[w8.moe_layer_workspace_size(1, 1, 16, 16) - 4 * 256:].fill_(255)
    return ws


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,topk,D,I", SIZES)
def test_layer(w8, fmt, T, E, topk, D, I):
    if fmt == "Block_FP8" and E > 200:
        E = 40
    c = Layer(fmt, T, E, topk, *sized(fmt, D, I))
    args = c.args(w8)
    buf = torch.full((T + 2, c.D + 5), 7.0, dtype=torch.bfloat16, device=DEV)
    y = w8.moe_layer(*args, y=buf[1:1 + T, 1:1 + c.D])
    c.check(y)
    assert (buf[:, 0] == 7).all() and (buf[:, 1 + c.D:] == 7).all()
    assert (buf[0] == 7).all() and (buf[T + 1] == 7).all()
    ws = workspace_of_nan(w8, c)
    for _ in range(2):
        assert torch.equal(w8.moe_layer(*args), y)
        assert torch.equal(w8.moe_layer(*args, workspace=ws), y)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("packed", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T,D,I", [(3, 256, 128), (20, 272, 400), (20, 144, 2752), (5, 80, 4112)])
def test_packed_weights(w8, fmt, packed, T, D, I):
    """Either layout of either weight: the same bits."""
    c = Layer(fmt, T, 6, 2, *sized(fmt, D, I))
    assert torch.equal(w8.moe_layer(*c.args(w8, packed)), w8.moe_layer(*c.args(w8)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_choices_left_out_and_repeated(w8, fmt):
    """Tokens without an expert, experts beyond the range, the same expert twice
    or only, all tokens on one expert."""
    E = 6
    experts = [[0, 3, 5], [-1, -1, -1], [2, 2, 2], [-1, 4, -7], [6, 1, 1 << 30], [5, 0, 5],
               [-(1 << 31), 2, 2], [3, 3, 3]]
    c = Layer(fmt, 8, E, 3, 256, 128, experts=experts)
    y = w8.moe_layer(*c.args(w8))
    c.check(y)
    assert (y[1] == 0).all()
    c = Layer(fmt, 9, E, 3, 256, 128, experts=np.full((9, 3), -1))
    y = w8.moe_layer(*c.args(w8), y=torch.full((9, 256), 5.0, dtype=torch.bfloat16, device=DEV))
    assert (y == 0).all()
    c = Layer(fmt, 32, E, 1, 256, 128, experts=np.full((32, 1), 4))
    c.check(w8.moe_layer(*c.args(w8)))
    # with the hidden codes made once
    experts = [[0, 3, 0], [-1, -1, -1], [2, 2, 2], [-1, 4, -7], [6, 1, 1 << 30], [5, 0, 5]] * 5
    c = Layer(fmt, 30, E, 3, 128, 1152, experts=experts)
    c.check(w8.moe_layer(*c.args(w8), workspace=workspace_of_nan(w8, c)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("E,I,experts", [
    (4, 128, [[2, 2]]), (8, 128, [[3, 1, 3, -1, 1]]), (64, 256, [[7, 9, 7], [9, 7, 9]]),
    (3, 4224, [[1, 0, 1]]), (50, 128, [[5, 5, 5, 5], [5, 6, 5, 6], [9, 9, 50, 9]]),
    (64, 128, [[8, 8, 3, 3], [3, 8, 8, 3], [1, 2, 2, 1], [2, 2, 2, 2], [0, 0, 1, 0]]),
    (4, 1664, [[1, 1, 0], [2, 0, 2], [0, 0, 0], [3, 1, 3], [1, 0, 1], [2, 2, 2], [0, 1, -1],
               [9, 1, 1], [1, 0, 2], [3, 2, 3]])])
def test_an_expert_twice_among_few(w8, fmt, E, I, experts):
    c = Layer(fmt, len(experts), E, len(experts[0]), 256, I, experts=experts)
    c.check(w8.moe_layer(*c.args(w8), workspace=workspace_of_nan(w8, c)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [1, 7, 20])
def test_base(w8, fmt, T):
    """Added before the one rounding, in place too; a token without an expert
    keeps it."""
    c = Layer(fmt, T, 5, 2, 256, 128)
    c.experts[T // 2] = -1
    a = c.args(w8)
    y, room = c.expected()
    g = np.random.default_rng(T)
    buf = torch.from_numpy(g.standard_normal((T, 259)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    base = buf[:, 1:257]
    want = y + base.double().cpu().numpy()
    got = w8.moe_layer(*a, base=base)
    # (the bound holds a rounding of y; here it is the sum that is rounded)
    room = room + 1.01 * 2.0 ** -8 * np.abs(want)
    assert (np.abs(got.double().cpu().numpy() - want) <= room).all()
    assert torch.equal(got[T // 2], base[T // 2])
    before = buf.clone()
    assert w8.moe_layer(*a, base=base, y=base) is base
    assert torch.equal(base, got) and torch.equal(buf[:, 0], before[:, 0])
    assert torch.equal(buf[:, 257:], before[:, 257:])
    c = Layer(fmt, T, 5, 2, 256, 128, experts=np.full((T, 2), -1))
    assert torch.equal(w8.moe_layer(*c.args(w8), base=before[:, 1:257]), before[:, 1:257])


@pytest.mark.parametrize("fmt", FORMATS)
def test_experts_without_tokens_are_not_read(w8, fmt):
    """Their codes and scales may hold anything."""
    c = Layer(fmt, 4, 8, 2, 256, 128, experts=[[1, 6], [6, 1], [1, -1], [6, 6]])
    a = list(c.args(w8))
    want = w8.moe_layer(*a)
    for i in (6, 8):
        a[i] = a[i].clone()
        a[i][[0, 2, 3, 4, 5, 7]] = float("nan")
    assert torch.equal(w8.moe_layer(*a), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_token_that_is_not_finite_stays_alone(w8, fmt, bad):
    c = Layer(fmt, 7, 4, 2, 256, 128)
    a = list(c.args(w8))
    want = w8.moe_layer(*a)
    a[2] = a[2].clone()
    a[2].view(7, -1)[3] = bad
    got = w8.moe_layer(*a)
    assert not torch.isfinite(got[3]).any()
    keep = [0, 1, 2, 4, 5, 6]
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("fmt", FORMATS)
def test_each_token_as_if_alone(w8, fmt):
    """A token's outputs depend on the others of the call by the order of sums at
    most (a call of few entries splits them): not at all where sums are exact."""
    for D, I in ((256, 256), (144, 1040), (64, 4096)):
        c = Layer(fmt, 32, 5, 2, *sized(fmt, D, I))
        a = c.args(w8)
        all_ = w8.moe_layer(*a)
        y, room = c.expected()
        for t in (0, 7, 31):
            one = w8.moe_layer(fmt, *(x[t:t + 1] for x in a[1:5]), *a[5:])
            if fmt == "W8A8_INT8":
                assert torch.equal(one[0], all_[t])
            assert (np.abs(one[0].double().cpu().numpy() - y[t]) <= room[t]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_strided_tokens_and_experts(w8, fmt):
    """Codes in wider rows, experts some way apart, no tokens."""
    c = Layer(fmt, 5, 4, 2, 256, 128)
    a = list(c.args(w8))
    want = w8.moe_layer(*a)
    t = a[1].dtype
    x = torch.full((5, 304), 0x7F, dtype=torch.uint8, device=DEV)
    x[:, 32:288] = a[1].view(torch.uint8)
    w1 = torch.full((4, 300, 288), 0x7F, dtype=torch.uint8, device=DEV)
    w1[:, 8:264, 16:272] = a[5].view(torch.uint8)
    w2 = torch.full((8, 256, 160), 0x7F, dtype=torch.uint8, device=DEV)
    w2[::2, :, :128] = a[7].view(torch.uint8)
    a[1], a[5], a[7] = x.view(t)[:, 32:288], w1.view(t)[:, 8:264, 16:272], w2.view(t)[::2, :, :128]
    assert torch.equal(w8.moe_layer(*a), want)
    none = w8.moe_layer(fmt, a[1][:0], a[2][:0], a[3][:0], a[4][:0], *a[5:])
    assert none.shape == (0, 256)


@pytest.mark.parametrize("fmt", FORMATS)
def test_workspace_shared_with_the_other_operators(w8, fmt):
    """One workspace for the layer and for products that split K, in turn."""
    c = Layer(fmt, 8, 8, 2, 256, 128)
    a, ws = c.args(w8), w8.Workspace(DEV, 64 << 20)
    want = w8.moe_layer(*a)
    g = np.random.default_rng(0)
    x, w = (on_device(codes(g, "W8A8_INT8", n, 7168)).view(torch.int8) for n in (48, 512))
    s = torch.ones(512, device=DEV)
    product = w8.token_gemm("W8A8_INT8", x, s[:48], w, s)
    assert w8.token_gemm_workspace_size("W8A8_INT8", 48, 512, 7168) > 0
    few = w8.gemm_w8a8("W8A8_INT8", x[:8], s[:8], w, s)
    for _ in range(4):
        assert torch.equal(w8.moe_layer(*a, workspace=ws), want)
        assert torch.equal(w8.token_gemm("W8A8_INT8", x, s[:48], w, s, workspace=ws), product)
        assert torch.equal(w8.gemm_w8a8("W8A8_INT8", x[:8], s[:8], w, s, workspace=ws), few)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,topk,D,I", [(8, 16, 4, 512, 256), (6, 4, 2, 128, 4224),
                                          (2, 16, 4, 256, 384), (24, 16, 2, 128, 4096),
                                          (24, 4, 2, 128, 1152)])
def test_capture_streams_and_overlap(w8, fmt, T, E, topk, D, I):
    c = Layer(fmt, T, E, topk, D, I)
    a = c.args(w8)
    want = w8.moe_layer(*a)
    c.check(want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [w8.moe_layer(*a, y=torch.empty_like(want), stream=st) for _ in range(10) for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
    y, ws = torch.empty_like(want), w8.Workspace(DEV, w8.moe_layer_workspace_size(T, topk, D, I))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w8.moe_layer(*a, y=y, workspace=ws)
    other = a[3].roll(1, 0)
    moved = w8.moe_layer(*a[:3], other, *a[4:])
    first = a[3].clone()
    for i in range(4):  # the choices are read when the graph runs
        a[3].copy_(other if i % 2 else first)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, moved if i % 2 else want)
        assert torch.equal(w8.moe_layer(*a), moved if i % 2 else want)


@pytest.mark.parametrize("T", [1, 9, 32])
def test_the_layer_and_its_parts(w8, T):
    """Router to output, as a layer of a decoding step runs them: moe_route and
    moe_layer, against moe_route, the grouped products, the gated quantizer and
    moe_combine."""
    fmt, E, topk, D, I = "Block_FP8", 16, 4, 512, 256
    c = Layer(fmt, T, E, topk, D, I)
    a = c.args(w8)
    logits = torch.from_numpy(np.random.default_rng(T).standard_normal((T, E)).astype(np.float32)).to(DEV)
    experts, weights, offsets, rows, slots = w8.moe_route(logits, topk)
    c.experts, c.weights = experts.cpu().numpy(), weights.cpu().numpy()
    y = w8.moe_layer(fmt, a[1], a[2], experts, weights, *a[5:])
    c.check(y)
    both = w8.grouped_gemm(a[1], a[2], offsets, a[5], a[6], rows=rows)
    q, s = w8.block_quantize(both[:, I:], gate=both[:, :I])
    parts = w8.moe_combine(w8.grouped_gemm(q, s, offsets, a[7], a[8]), weights, slots)
    # the parts round the halves and the outputs to bf16 on the way: codes may
    # differ by a step (2^-4 of a value at most) where such a rounding (2^-8)
    # crosses a border (one in 2^4 of them), 2^-6 of the norm, and the outputs'
    # own roundings
    assert torch.linalg.norm((y - parts).double()) <= 2.0 ** -5 * torch.linalg.norm(y.double())
