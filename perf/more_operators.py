"""Token-scaled products of any size and the mixture-of-experts layer of a few tokens: cases,
inputs, plain forms and exact results.

Five operators that stand beside the small-M GEMM, the grouped GEMM and the Block_FP8
quantizer:

  gemm      Y[M, N] = dequant(Xq) . dequant(Wq)^T for any M, one scale per token and one per
            output channel (W8A8_INT8 and FP8_Dynamic)
  quantize  the codes and scales that product takes, of x or of silu(gate) * x
  route     top-k of the router's logits: experts and weights of each token, and the lists per
            expert that the grouped products take
  combine   each token's sum of its experts' outputs, weighted
  layer     the experts of a few tokens as a whole: gate and up projections, silu(gate) * up,
            its codes, down projection, weighted sum

A case is a dict of plain values; prepare() makes its inputs on the GPU and run() is one call,
in the library's kernels where `own` is true and in elementary torch operations in fp32
otherwise.
"""
import math

import torch

own = False

GROUP = 128
QMAX = {"W8A8_INT8": 127.0, "FP8_Dynamic": 448.0, "Block_FP8": 448.0}
E4M3 = torch.float8_e4m3fn


# -------------------------------------------------------------------- cases --
def listed():
    return [
        # a batch of drafted or batched tokens just past the small-M window
        dict(name="gemm_batch48", op="gemm", fmt="W8A8_INT8", M=48, N=4608, K=7168),
        # ragged in all three sizes
        dict(name="gemm_ragged", op="gemm", fmt="FP8_Dynamic", M=333, N=897, K=1040),
        # a full prefill chunk through the deepest projection
        dict(name="gemm_prefill", op="gemm", fmt="W8A8_INT8", M=8192, N=5120, K=8192),
        # the activations of that batch in front of its projection
        dict(name="quantize_batch48", op="quantize", fmt="W8A8_INT8", M=48, K=7168, gated=False),
        # the gated activation of a prefill chunk in front of the deepest projection
        dict(name="quantize_prefill", op="quantize", fmt="FP8_Dynamic", M=8192, K=8192, gated=True),
        # the router of a few decoding sequences
        dict(name="route_decode", op="route", T=8, E=128, topk=8, logits="fp32", masked=0.0),
        # the router of a prefill chunk; its bf16 logits hold many ties
        dict(name="route_prefill", op="route", T=8192, E=128, topk=8, logits="bf16", masked=0.0),
        # the experts' outputs of a mid-sized batch, some experts on another device
        dict(name="combine_ragged", op="combine", T=333, topk=8, D=2048, base=True, dropped=0.25),
        # the experts' outputs of a prefill chunk
        dict(name="combine_prefill", op="combine", T=4096, topk=8, D=2048, base=False, dropped=0.0),
        # one decoding sequence through a layer of 128 experts
        dict(name="layer_one_token", op="layer", fmt="Block_FP8", T=1, E=128, topk=8, D=2048,
             I=768, dropped=0.0),
        # a few decoding sequences
        dict(name="layer_batch8", op="layer", fmt="W8A8_INT8", T=8, E=128, topk=8, D=2048, I=768,
             dropped=0.0),
        # the most tokens of the decode window; nearly every expert is reached
        dict(name="layer_batch32", op="layer", fmt="FP8_Dynamic", T=32, E=128, topk=8, D=2048,
             I=768, dropped=0.0),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemm", "quantize", "route", "combine", "layer"))
    if op == "gemm":
        while True:
            M, N = _log_between(rng, 1, 8192), _log_between(rng, 256, 8192)
            K = 16 * _log_between(rng, 16, 512)
            if rng.random() < 0.5:  # half the layers are whole 128s wide
                N, K = -(-N // 128) * 128, -(-K // 128) * 128
            if M * N * K <= 8192 * 5120 * 8192:
                return dict(op=op, fmt=rng.choice(("W8A8_INT8", "FP8_Dynamic")), M=M, N=N, K=K)
    if op == "quantize":
        while True:
            M, K = _log_between(rng, 1, 32768), 8 * _log_between(rng, 16, 2048)
            if M * K <= 8192 * 8192:
                return dict(op=op, fmt=rng.choice(("W8A8_INT8", "FP8_Dynamic")), M=M, K=K,
                            gated=rng.random() < 0.5)
    if op == "route":
        E = rng.choice((8, 16, 60, 64, 128, 256))
        while True:
            T = _log_between(rng, 1, 16384)
            if T * E <= 8192 * 128:
                return dict(op=op, T=T, E=E, topk=rng.choice((1, 2, 4, 6, 8)),
                            logits=rng.choice(("fp32", "bf16")), masked=rng.choice((0.0, 0.5)))
    if op == "combine":
        topk = rng.choice((1, 2, 4, 6, 8))
        while True:
            T, D = _log_between(rng, 1, 8192), _log_between(rng, 64, 8192)
            if rng.random() < 0.7:
                D = -(-D // 128) * 128
            if T * topk * D <= 4096 * 8 * 2048:
                return dict(op=op, T=T, topk=topk, D=D, base=rng.random() < 0.5,
                            dropped=rng.choice((0.0, 0.25)))
    fmt = rng.choice(("W8A8_INT8", "FP8_Dynamic", "Block_FP8"))
    unit = 128 if fmt == "Block_FP8" else 16
    E, topk = rng.choice((8, 16, 60, 64, 128)), rng.choice((1, 2, 4, 6, 8))
    while True:
        T = _log_between(rng, 1, 32)
        D, I = (unit * max(1, round(_log_between(rng, 256, 4096) / unit)),
                unit * max(1, round(_log_between(rng, 128, 4096) / unit)))
        if E * D * I <= 128 * 2048 * 768:
            return dict(op=op, fmt=fmt, T=T, E=E, topk=topk, D=D, I=I,
                        dropped=rng.choice((0.0, 0.25)))


# ------------------------------------------------------------------- inputs --
def _groups(n):
    return -(-n // GROUP)


def _round_codes(t, fmt):
    t = t.clamp(-QMAX[fmt], QMAX[fmt])
    return torch.round(t).to(torch.int8) if fmt == "W8A8_INT8" else t.to(E4M3)


def _scale(amax, fmt):
    return torch.where(amax == 0, torch.ones_like(amax), amax / QMAX[fmt])


def _codes_rows(v, fmt):
    """Codes and fp32 scales of fp32 v [rows, K]: one scale a row, Block_FP8 one per 1 x 128."""
    if fmt != "Block_FP8":
        s = _scale(v.abs().amax(dim=-1), fmt)
        return _round_codes(v / s[..., None], fmt), s
    rows, K = v.shape
    p = v.view(rows, K // GROUP, GROUP)
    s = _scale(p.abs().amax(dim=2), fmt)
    return _round_codes(p / s[:, :, None], fmt).view(rows, K), s


def _codes_weights(w, fmt):
    """Codes and scales of fp32 w [..., N, K]: one scale an output channel, Block_FP8 one per
    128 x 128."""
    if fmt != "Block_FP8":
        s = w.abs().amax(dim=-1) / QMAX[fmt]
        return _round_codes(w / s[..., None], fmt), s
    N, K = w.shape[-2:]
    p = w.view(*w.shape[:-2], N // GROUP, GROUP, K // GROUP, GROUP)
    s = p.abs().amax(dim=(-3, -1)) / QMAX[fmt]
    return _round_codes(p / s[..., :, None, :, None], fmt).view(w.shape), s.contiguous()


def _choices(T, E, topk, g):
    """Logits of T tokens over experts of unequal popularity."""
    pop = 0.5 * torch.randn(E, generator=g, device="cuda")
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    return pop - torch.log(-torch.log(u))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s, op = dict(case), case["op"]
    if op == "gemm":
        s["xq"], s["sx"] = _codes_rows(randn(case["M"], case["K"]), case["fmt"])
        s["wq"], s["sw"] = _codes_weights(0.02 * randn(case["N"], case["K"]), case["fmt"])
    elif op == "quantize":
        M, K = case["M"], case["K"]
        if case["gated"]:  # the two halves of one projection's output
            both = randn(M, 2 * K).to(torch.bfloat16)
            s["gate"], s["x"] = both[:, :K], both[:, K:]
        else:
            s["gate"], s["x"] = None, randn(M, K).to(torch.bfloat16)
    elif op == "route":
        T, E = case["T"], case["E"]
        logits = _choices(T, E, case["topk"], g)
        if case["masked"]:  # experts out of use: some for every token, some tokens without any
            logits[:, rand(E) < case["masked"]] = -math.inf
            logits[rand(T) < 0.1] = -math.inf
        s["scores"] = logits.to(torch.bfloat16 if case["logits"] == "bf16" else torch.float32)
    elif op == "combine":
        T, topk, D = case["T"], case["topk"], case["D"]
        n = T * topk
        s["y"] = randn(n, D).to(torch.bfloat16)
        s["weights"] = torch.softmax(randn(T, topk), dim=1)
        place = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        s["slots"] = torch.where(rand(n) < case["dropped"], -1, place).to(torch.int32).view(T, topk)
        s["added"] = randn(T, D).to(torch.bfloat16) if case["base"] else None
    else:
        T, E, topk, D, I, fmt = (case[k] for k in ("T", "E", "topk", "D", "I", "fmt"))
        s["xq"], s["sx"] = _codes_rows(randn(T, D), fmt)
        s["w1"], s["s1"] = _codes_weights(randn(E, 2 * I, D) / D ** 0.5, fmt)
        s["w2"], s["s2"] = _codes_weights(randn(E, D, I) / I ** 0.5, fmt)
        top = _choices(T, E, topk, g).topk(topk, dim=1)
        s["weights"] = torch.softmax(top.values, dim=1)
        s["experts"] = torch.where(rand(T, topk) < case["dropped"], -1, top.indices).to(torch.int32)
    return s


# -------------------------------------------------------------- plain forms --
def _silu_times(g, u):
    return g / (1 + torch.exp(-g)) * u


def _wide_rows(q, s):
    if s.dim() == q.dim():  # Block_FP8
        s = s.repeat_interleave(GROUP, dim=-1)
        return q.float() * s
    return q.float() * s[..., None]


def _wide_weights(q, s):
    if s.dim() == q.dim():  # Block_FP8
        return q.float() * s.repeat_interleave(GROUP, dim=-2).repeat_interleave(GROUP, dim=-1)
    return q.float() * s[..., None]


def _of(q, at):
    """Rows `at` of codes (torch indexes no 8-bit floats)."""
    return q.view(torch.uint8)[at].view(q.dtype)


def _plain_gemm(s):
    return (_wide_rows(s["xq"], s["sx"]) @ _wide_weights(s["wq"], s["sw"]).t()).to(torch.bfloat16)


def _plain_quantize(s):
    x = s["x"].float()
    return _codes_rows(x if s["gate"] is None else _silu_times(s["gate"].float(), x), s["fmt"])


def _plain_route(s):
    l, E, topk = s["scores"].float(), s["E"], s["topk"]
    v, i = l.sort(dim=1, descending=True, stable=True)  # (ties: the lowest index first)
    v, i = v[:, :topk], i[:, :topk]
    off = torch.isneginf(v)
    p = torch.where(off, 0, torch.exp(v - v[:, :1]))
    weights = torch.where(off, 0, p / p.sum(dim=1, keepdim=True))
    experts = torch.where(off, -1, i).to(torch.int32)
    e = torch.where(off, E, i).reshape(-1)
    order = e.argsort(stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=e.device)
    offsets[1:] = torch.bincount(e, minlength=E + 1)[:E].cumsum(0)
    at = torch.arange(len(e), device=e.device)
    rows = torch.where(at < offsets[E], order // topk, 0).to(torch.int32)
    slots = torch.empty_like(order).scatter_(0, order, at)
    slots = torch.where(e < E, slots, -1).to(torch.int32).view(-1, topk)
    return experts, weights, offsets, rows, slots


def _plain_combine(s):
    at = s["slots"].long()
    w = torch.where(at >= 0, s["weights"], 0)
    out = (s["y"][at.clamp(min=0)].float() * w[:, :, None]).sum(dim=1)
    if s["added"] is not None:
        out = out + s["added"].float()
    return out.to(torch.bfloat16)


def _plain_layer(s):
    T, E, topk, D, I = (s[k] for k in ("T", "E", "topk", "D", "I"))
    e = s["experts"].long().reshape(-1)
    w = torch.where(e >= 0, s["weights"].reshape(-1), 0)
    e = e.clamp(min=0)
    token = torch.arange(T, device=e.device).repeat_interleave(topk)
    x = _wide_rows(s["xq"], s["sx"])
    few = T * topk <= E  # the chosen experts' weights, or with more entries all experts'
    if few:
        w1, w2 = _wide_weights(_of(s["w1"], e), s["s1"][e]), _wide_weights(_of(s["w2"], e), s["s2"][e])
        a = torch.bmm(x[token][:, None], w1.transpose(1, 2))[:, 0]
    else:
        w1, w2 = _wide_weights(s["w1"], s["s1"]), _wide_weights(s["w2"], s["s2"])
        a = torch.matmul(x, w1.transpose(1, 2))[e, token]
    v = _wide_rows(*_codes_rows(_silu_times(a[:, :I], a[:, I:]), s["fmt"]))
    if few:
        o = torch.bmm(v[:, None], w2.transpose(1, 2))[:, 0]
    else:
        at = torch.zeros(E, T, I, device=v.device)
        at[e, token] = v
        o = torch.bmm(at, w2.transpose(1, 2))[e, token]
    return (o * w[:, None]).view(T, topk, D).sum(dim=1).to(torch.bfloat16)


# --------------------------------------------------------------------- runs --
def _own(s):
    import bit_quantized_gemm_token_amd as w8
    op = s["op"]
    if op == "gemm":
        return w8.token_gemm(s["fmt"], s["xq"], s["sx"], s["wq"], s["sw"])
    if op == "quantize":
        # (torch divides by a constant through its reciprocal on the GPU; whole numbers are equal
        # only with scales that are rounded the same way)
        return w8.token_quantize(s["fmt"], s["x"], gate=s["gate"], reciprocal=True)
    if op == "route":
        return w8.moe_route(s["scores"], s["topk"])
    if op == "combine":
        return w8.moe_combine(s["y"], s["weights"], s["slots"], base=s["added"])
    return w8.moe_layer(s["fmt"], s["xq"], s["sx"], s["experts"], s["weights"], s["w1"], s["s1"],
                        s["w2"], s["s2"])


def run(state):
    if own:
        out = _own(state)
    else:
        out = {"gemm": _plain_gemm, "quantize": _plain_quantize, "route": _plain_route,
               "combine": _plain_combine, "layer": _plain_layer}[state["op"]](state)
    if state["op"] == "quantize" and state["gated"] and state["fmt"] == "W8A8_INT8":
        # rounded from a computed product, where a value next to a border may go either way:
        # as the numbers that the codes stand for
        out = out[0].to(torch.bfloat16), out[1]
    return out


# --------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 2 * M * N + 4 * (M + N), "flops": 2 * M * N * K}
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (3 + 2 * case["gated"]) + 4 * M,
                "flops": M * K * (3 + 5 * case["gated"])}
    if op == "route":
        T, E, n = case["T"], case["E"], case["T"] * case["topk"]
        return {"bytes": T * E * (4 if case["logits"] == "fp32" else 2) + 16 * n + 4 * (E + 1),
                "flops": 4 * T * E}
    if op == "combine":
        T, D, n = case["T"], case["D"], case["T"] * case["topk"]
        read = n * (1 - case["dropped"])
        return {"bytes": 2 * D * (read + T * (1 + case["base"])) + 8 * n, "flops": 2 * read * D}
    T, E, topk, D, I = (case[k] for k in ("T", "E", "topk", "D", "I"))
    kept = 1 - case["dropped"]
    reached = E * (1 - (1 - topk * kept / E) ** T)  # experts that any token chose, as expected
    per, act = 3 * I * D, T * D
    if case["fmt"] == "Block_FP8":
        per, act = per + 4 * per // GROUP ** 2, act + 4 * act // GROUP
    else:
        per, act = per + 4 * (2 * I + D), act + 4 * T
    return {"bytes": reached * per + act + 8 * T * topk + 2 * T * D,
            "flops": 6 * T * topk * kept * I * D}


# -------------------------------------------------------------------- exact --
def _exact_codes(v, fmt):
    """Codes (as their values) and scales of 64-bit rows by the definition: the nearest whole
    number, or the nearest E4M3FN value (ties to even): a grid of 2^-9 below 2^-6 and of three
    fraction bits above."""
    top = QMAX[fmt]
    M, K = v.shape
    p = v.reshape(M, -1, GROUP) if fmt == "Block_FP8" else v.reshape(M, 1, K)
    amax = p.abs().max(dim=2).values
    s = torch.where(amax > 0, amax / top, torch.ones_like(amax))
    t = p / s.unsqueeze(2)
    if fmt == "W8A8_INT8":
        q = torch.round(t)
    else:
        _, e = torch.frexp(t)  # |t| in [2^(e-1), 2^e)
        step = torch.ldexp(torch.ones_like(t), (e - 4).clamp(min=-9))
        q = torch.round(t / step) * step
    q = q.clamp(-top, top)
    return q.reshape(M, K), (s if fmt == "Block_FP8" else s[:, 0])


def _exact_rows(q, s):
    each = s.double().reshape(q.shape[0], -1)
    return q.double() * each[:, torch.arange(q.shape[1], device=q.device) * each.shape[1] // q.shape[1]]


def _exact_weights(q, s):
    N, K = q.shape
    if s.dim() == 1:
        return q.double() * s.double()[:, None]
    ng, kg = (torch.arange(n, device=q.device) // GROUP for n in (N, K))
    return q.double() * s.double()[ng][:, kg]


def _exact_silu(g):
    return g * torch.sigmoid(g)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        return torch.mm(_exact_rows(s["xq"], s["sx"]),
                        _exact_weights(s["wq"], s["sw"]).T.contiguous())
    if op == "quantize":
        x = s["x"].double()
        if s["gate"] is not None:
            x = x * _exact_silu(s["gate"].double())
        return _exact_codes(x, case["fmt"])
    if op == "route":
        # by counting: an expert's place is the number of those in front of it
        l, topk = s["scores"].double(), case["topk"]
        weights = torch.zeros(case["T"], topk, dtype=torch.float64, device=l.device)
        left = l.clone()
        for j in range(topk):
            weights[:, j], at = left.max(dim=1)
            left.scatter_(1, at[:, None], -math.inf)
        weights = torch.nan_to_num(torch.softmax(weights, dim=1), nan=0.0)
        return None, weights, None, None, None
    if op == "combine":
        out = torch.zeros(case["T"], case["D"], dtype=torch.float64, device="cuda")
        if s["added"] is not None:
            out += s["added"].double()
        for j in range(case["topk"]):
            at = s["slots"][:, j].long()
            t = (at >= 0).nonzero()[:, 0]
            out[t] += s["weights"][t, j].double()[:, None] * s["y"][at[t]].double()
        return out
    x, I = _exact_rows(s["xq"], s["sx"]), case["I"]
    out = torch.zeros(case["T"], case["D"], dtype=torch.float64, device="cuda")
    for e in sorted(set(s["experts"].flatten().tolist()) - {-1}):
        t, j = (s["experts"] == e).nonzero(as_tuple=True)
        a = torch.mm(x[t], _exact_weights(s["w1"][e], s["s1"][e]).T.contiguous())
        v = _exact_rows(*_exact_codes(_exact_silu(a[:, :I]) * a[:, I:], case["fmt"]))
        y = torch.mm(v, _exact_weights(s["w2"][e], s["s2"][e]).T.contiguous())
        out.index_add_(0, t, y * s["weights"][t, j].double()[:, None])
    return out
