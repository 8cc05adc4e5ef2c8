"""MoE routing and combination on the GPU: whole numbers exactly, weights and
sums against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

from tests.block_cases import DEV, bf16, on_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import bit_quantized_gemm_token_amd as mod
    return mod


def route(logits, topk, renormalize=True, scale=1.0):
    """(experts, weights, offsets, rows, slots) by the definition, in 64 bits."""
    l = logits.astype(np.float64)
    T, E = l.shape
    l = np.where(np.isnan(l), -np.inf, l)
    order = np.argsort(-l, axis=1, kind="stable")[:, :topk]
    v = np.take_along_axis(l, order, axis=1)
    off = np.isneginf(v)
    top = v[:, :1]

    def over_top(a):
        with np.errstate(invalid="ignore", over="ignore"):
            return np.where(a == top, 1.0, np.exp(a - np.where(np.isneginf(top), 0, top)))

    p = np.where(off, 0, over_top(v))
    total = p.sum(axis=1, keepdims=True) if renormalize else \
        np.where(np.isneginf(l), 0, over_top(l)).sum(axis=1, keepdims=True)
    weights = np.where(off, 0, scale * p / np.where(total == 0, 1, total))
    experts = np.where(off, -1, order).astype(np.int32)
    e = experts.reshape(-1)
    kept = np.flatnonzero(e >= 0)
    at = kept[np.argsort(e[kept], kind="stable")]
    rows = np.zeros(T * topk, np.int32)
    rows[:len(at)] = at // topk
    slots = np.full(T * topk, -1, np.int32)
    slots[at] = np.arange(len(at))
    offsets = np.r_[0, np.cumsum(np.bincount(e[kept], minlength=E))].astype(np.int32)
    return experts, weights, offsets, rows, slots.reshape(T, topk)


def check(got, want, what=""):
    for name, a, b in zip(("experts", "weights", "offsets", "rows", "slots"), got, want):
        a = a.cpu().numpy()
        assert a.shape == b.shape, f"{what} {name}"
        if name == "weights":
            # the exponential and its argument's rounding (|l - l_max| below 2^7
            # here, each within 2^-24: 2^-16 would be far off; sums of up to 2^10
            # terms, a quotient and a product, 2^-24 each)
            np.testing.assert_allclose(a, b, rtol=2.0 ** -13, atol=1e-37, err_msg=what)
            big = b > 1e-4
            np.testing.assert_allclose(a[big], b[big], rtol=2.0 ** -19, err_msg=what)
        else:
            np.testing.assert_array_equal(a, b, err_msg=f"{what} {name}")


def logits_of(g, T, E, dtype, spread=2.0):
    l = (g.standard_normal((T, E)) * spread).astype(np.float32)
    if dtype == "bf16":
        return bf16(l)[0], bf16(l)[1].astype(np.float32)
    return on_device(l), l


@pytest.mark.parametrize("T,E,topk", [
    (1, 1, 1), (1, 8, 2), (1, 128, 8), (3, 5, 5), (8, 128, 8), (32, 128, 8), (33, 128, 8),
    (64, 60, 4), (65, 60, 4), (100, 64, 6), (42, 64, 6), (43, 64, 6), (257, 16, 1), (16, 1024, 32),
    (8, 1000, 32), (9, 1000, 31), (300, 200, 7), (1000, 129, 8), (5000, 128, 8), (3000, 256, 2),
    (20000, 8, 2), (40, 1024, 1), (16, 256, 8), (17, 256, 8), (32, 250, 8), (200, 256, 1),
    (24, 300, 8), (42, 1000, 6), (128, 300, 2), (239, 256, 6), (2100, 200, 1)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route(w8, T, E, topk, dtype):
    print(f"[case] T={T} E={E} topk={topk} {dtype}", flush=True)
    d, l = logits_of(np.random.default_rng([T, E, topk]), T, E, dtype)
    got = w8.moe_route(d, topk)
    check(got, route(l, topk))
    pair = w8.moe_route(d, topk, lists=False)
    assert len(pair) == 2 and torch.equal(pair[0], got[0]) and torch.equal(pair[1], got[1])
    check(w8.moe_route(d, topk, renormalize=False, scale=2.5), route(l, topk, False, 2.5))


@pytest.mark.parametrize("E,topk", [(128, 8), (256, 6), (300, 5)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [20, 700])
def test_masks_ties_and_nonfinite_logits(w8, E, topk, dtype, T):
    g = np.random.default_rng([E, topk])
    l = g.integers(-2, 3, (T, E)).astype(np.float32)  # many ties
    l[l == 0] *= g.choice([-1.0, 1.0], (l == 0).sum())  # zeros of both signs
    l[0] = -np.inf                       # nothing left
    l[1] = np.nan
    l[2] = -np.inf
    l[2, [7, 100]] = 3.0                 # fewer than topk
    l[3, ::2] = np.nan
    l[4] = np.finfo(np.float32).min      # the type's lowest value is a logit like any
    l[5, [9, 3]] = np.inf                # +inf: all the weight, shared
    l[6] = -np.inf
    l[6, E - 1] = np.inf
    l[7, 5:] = -np.inf
    l[8] = 0.0
    if dtype == "bf16":
        l[4] = torch.finfo(torch.bfloat16).min
        d = torch.from_numpy(l).to(torch.bfloat16).to(DEV)
        l = d.float().cpu().numpy()
    else:
        d = on_device(l)
    for renorm in (True, False):
        check(w8.moe_route(d, topk, renormalize=renorm), route(l, topk, renorm))


def test_all_tokens_to_one_expert_and_none(w8):
    for T in (10, 3000):
        l = np.full((T, 64), -np.inf, np.float32)
        check(w8.moe_route(on_device(l), 4), route(l, 4))
        l[:, 63] = 1.0
        check(w8.moe_route(on_device(l), 4), route(l, 4))
        l[:, :4] = 2.0
        check(w8.moe_route(on_device(l), 4), route(l, 4))


def test_no_tokens(w8):
    e, w, off, rows, slots = w8.moe_route(torch.empty(0, 64, device=DEV), 4)
    assert e.shape == w.shape == slots.shape == (0, 4) and rows.shape == (0,)
    assert off.tolist() == [0] * 65
    assert w8.moe_route(torch.empty(0, 64, device=DEV), 4, lists=False)[0].shape == (0, 4)


def test_strided_logits(w8):
    wide, l = logits_of(np.random.default_rng(3), 300, 131, "bf16")
    check(w8.moe_route(wide[:, 1:130], 8), route(l[:, 1:130], 8))


def test_more_tokens_than_workgroups_of_one_pass(w8):
    """More than 1024 workgroups' worth of entries: several passes each."""
    T, E, topk = 2048 * 16 + 5, 16, 16  # 8 tokens a pass
    g = np.random.default_rng(1)
    d, l = logits_of(g, T, E, "fp32")
    l[5::7] = -np.inf
    d = on_device(l)
    check(w8.moe_route(d, topk), route(l, topk))


def test_lists_are_what_the_grouped_product_takes(w8):
    """Together with the grouped product and the combination: a token's outputs
    are the weighted sum of its experts' products."""
    from tests.block_cases import (codes_on_device, dequant_blocks, dequant_rows, draw_codes,
                                   draw_scales, groups)
    T, E, topk, N, K = 70, 12, 3, 264, 384
    g = np.random.default_rng(7)
    d, l = logits_of(g, T, E, "fp32")
    l[:, 4] = -np.inf
    l[9] = -np.inf
    experts, weights, offsets, rows, slots = w8.moe_route(on_device(l), topk)
    xq, sx = draw_codes(g, T, K), draw_scales(g, T, groups(K))
    wq, sw = draw_codes(g, E, N, K), draw_scales(g, E, groups(N), groups(K))
    y = w8.grouped_gemm(codes_on_device(xq), on_device(sx), offsets, codes_on_device(wq),
                        on_device(sw), rows=rows)
    base, bv = bf16(g.standard_normal((T, N)))
    out = w8.moe_combine(y, weights, slots, base=base).double().cpu().numpy()
    x, w = dequant_rows(xq, sx), dequant_blocks(wq, sw)
    want, room = bv.copy(), np.abs(bv)
    e, wt = experts.cpu().numpy(), weights.double().cpu().numpy()
    for t in range(T):
        for j in range(topk):
            if e[t, j] >= 0:
                p = x[t] @ w[e[t, j]].T
                want[t] += wt[t, j] * p
                room[t] += np.abs(wt[t, j]) * (np.abs(p) + 2.0 ** -5 * (np.abs(x[t]) @ np.abs(w[e[t, j]]).T))
    # bf16 of each product (2^-8 of it) and of the sum, and the products' sums
    # (2^-14 of the sum of |products|, 2^-9 of the 2^-5 above)
    assert (np.abs(out - want) <= 1.01 * 2.0 ** -8 * (room + np.abs(want)) + 1e-38).all()
    assert np.array_equal(out[9], bv[9])  # no expert: the base alone


# ------------------------------------------------------------------ combine --
def combine(y, w, slots, base):
    """(the sum in 64 bits, the sum of the absolute terms)."""
    on = (slots >= 0) & (slots < len(y))
    at = np.where(on, slots, 0)
    terms = np.where(on[:, :, None], y[at] * w[:, :, None].astype(np.float64), 0) if len(y) else \
        np.zeros(slots.shape + (y.shape[1],))
    b = 0 if base is None else base
    return terms.sum(axis=1) + b, np.abs(terms).sum(axis=1) + np.abs(b)


@pytest.mark.parametrize("T,topk,D", [
    (1, 1, 1), (1, 8, 2048), (3, 2, 7), (5, 8, 64), (33, 6, 129), (2, 32, 100), (7, 9, 2056),
    (4, 8, 4097), (333, 8, 512), (1000, 4, 72), (3, 17, 8199), (3000, 2, 8)])
@pytest.mark.parametrize("with_base", [False, True])
def test_combine(w8, T, topk, D, with_base):
    print(f"[case] T={T} topk={topk} D={D}", flush=True)
    g = np.random.default_rng([T, topk, D])
    n = max(1, T * topk - 2)
    y, yv = bf16(g.standard_normal((n, D)))
    w = g.standard_normal((T, topk)).astype(np.float32)
    slots = g.integers(-2, n + 2, (T, topk)).astype(np.int32)  # both ends beyond the rows
    slots[0] = -1
    base, bv = bf16(g.standard_normal((T, D))) if with_base else (None, None)
    buf = torch.full((T + 2, D + 3), 7.0, dtype=torch.bfloat16, device=DEV)
    out = w8.moe_combine(y, on_device(w), on_device(slots), base=base, out=buf[1:1 + T, 1:1 + D])
    want, room = combine(yv, w, slots, bv)
    # a rounding to bf16, and fp32 sums of at most 33 terms
    bad = ~(np.abs(out.double().cpu().numpy() - want)
            <= 1.01 * 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * room + 1e-38)
    assert not bad.any(), np.argwhere(bad)[:4].tolist()
    assert (buf[:, 0] == 7).all() and (buf[:, 1 + D:] == 7).all()
    assert (buf[0] == 7).all() and (buf[T + 1] == 7).all()
    if with_base:  # in place
        assert torch.equal(w8.moe_combine(y, on_device(w), on_device(slots), base=base, out=base), out)


def test_combine_leaves_out_what_it_does_not_name(w8):
    """Rows that no slot names may hold anything, row 0 too."""
    y = torch.full((6, 40), float("nan"), dtype=torch.bfloat16, device=DEV)
    y[3], y[4] = 2.0, float("inf")
    slots = torch.tensor([[-1, 3], [3, 6], [1 << 30, -(1 << 31)], [4, 3]], dtype=torch.int32, device=DEV)
    w = torch.full((4, 2), 0.5, device=DEV)
    out = w8.moe_combine(y, w, slots).float().cpu()
    assert (out[:2] == 1).all() and (out[2] == 0).all() and torch.isinf(out[3]).all()
    none = w8.moe_combine(y[:0], w, slots, base=torch.ones(4, 40, dtype=torch.bfloat16, device=DEV))
    assert (none == 1).all()
    assert w8.moe_combine(y, w[:0], slots[:0]).shape == (0, 40)


def test_capture_and_streams(w8):
    T, E, topk, D = 500, 64, 6, 264
    g = np.random.default_rng(2)
    d, l = logits_of(g, T, E, "fp32")
    y, _ = bf16(g.standard_normal((T * topk, D)))
    want = w8.moe_route(d, topk)
    out = w8.moe_combine(y, want[1], want[4])
    check(want, route(l, topk))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for st in streams:
            r = w8.moe_route(d, topk, stream=st)
            got.append((r, w8.moe_combine(y, r[1], r[4], stream=st)))
    torch.cuda.synchronize()
    for r, o in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want)) and torch.equal(o, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = w8.moe_route(d, topk)
        o = w8.moe_combine(y, r[1], r[4])
    for _ in range(4):
        for t in (*r, o):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, want)) and torch.equal(o, out)
        assert torch.equal(w8.moe_route(d, topk)[3], want[3])
