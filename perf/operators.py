"""The Block_FP8 operators for any number of tokens: cases, inputs, plain forms and exact results.

Four operators that make up a Block_FP8 layer outside the small-M window
(activations in E4M3FN with one scale per 1 x 128 group, weights with one
scale per 128 x 128 block):

  norm      h = residual + scale * gate * N(y), z = N(h): the residual stream's
            update between two blocks, z in bfloat16 or as codes and scales
  quantize  codes and scales of x, or of silu(gate) * x
  gemm      Y[M, N] = dequant(Xq) . dequant(Wq)^T
  grouped   the same product per expert, over ragged lists of token rows

A case is a dict of plain values; prepare() makes its inputs on the GPU and
run() is one call, in the library's kernels where `own` is true and in
elementary torch operations in fp32 otherwise.
"""
import math

import torch

own = False

GROUP = 128
QMAX = 448.0
E4M3 = torch.float8_e4m3fn


# -------------------------------------------------------------------- cases --
def listed():
    return [
        # one token through a projection: a decoding step outside any batch
        dict(name="gemm_one_token", op="gemm", M=1, N=4608, K=7168),
        # just past the small-M window: a batch of drafted or batched tokens
        dict(name="gemm_batch48", op="gemm", M=48, N=4608, K=7168),
        # ragged in all three sizes, K ending inside a group
        dict(name="gemm_ragged", op="gemm", M=333, N=897, K=1040),
        # one long prompt into a wide projection of short depth
        dict(name="gemm_prompt", op="gemm", M=4096, N=5120, K=2048),
        # a full prefill chunk through the deepest projection
        dict(name="gemm_prefill", op="gemm", M=8192, N=5120, K=8192),
        # experts' gate/up projection of a few decoding sequences
        dict(name="grouped_decode", op="grouped", T=8, E=128, topk=8, N=1536, K=2048, gather=True),
        # experts' down projection of a mid-sized batch; rows already in expert order
        dict(name="grouped_down", op="grouped", T=512, E=128, topk=8, N=2048, K=768, gather=False),
        # experts' gate/up projection of a prefill chunk
        dict(name="grouped_prefill", op="grouped", T=4096, E=128, topk=8, N=1536, K=2048, gather=True),
        # between two blocks for one decoding sequence, straight to codes
        dict(name="norm_one_token", op="norm", M=1, D=7168, residual="bf16", post=False,
             gate="none", out="codes"),
        # between two blocks of a prefill chunk: normed and gated branch, fp32 residual stream
        dict(name="norm_prefill", op="norm", M=8192, D=5120, residual="fp32", post=True,
             gate="token", out="bf16"),
        # gated activation of a few sequences
        dict(name="quantize_decode", op="quantize", M=33, K=2048, gated=True),
        # gated activation of the experts' gate/up outputs of a prefill chunk
        dict(name="quantize_prefill", op="quantize", M=32768, K=768, gated=True),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemm", "grouped", "norm", "quantize"))
    if op == "gemm":
        while True:
            M, N = _log_between(rng, 1, 8192), _log_between(rng, 256, 8192)
            K = 16 * _log_between(rng, 16, 512)
            if rng.random() < 0.5:  # half the layers are whole groups wide
                N, K = -(-N // 128) * 128, -(-K // 128) * 128
            if M * N * K <= 8192 * 5120 * 8192 and 3072 not in (M, N, K):
                return dict(op=op, M=M, N=N, K=K)
    if op == "grouped":
        E = rng.choice((8, 16, 60, 64, 128))
        topk = rng.choice((1, 2, 4, 8))
        while True:
            T = _log_between(rng, 1, 4096)
            N, K = _log_between(rng, 256, 2048), 16 * _log_between(rng, 16, 128)
            if rng.random() < 0.5:
                N, K = -(-N // 128) * 128, -(-K // 128) * 128
            if T * topk == 3072:
                continue
            if T * topk * N * K <= 4096 * 8 * 1536 * 2048 and E * N * K <= 128 * 1536 * 2048:
                return dict(op=op, T=T, E=E, topk=topk, N=N, K=K, gather=rng.random() < 0.6)
    if op == "norm":
        while True:
            M, D = _log_between(rng, 1, 16384), _log_between(rng, 64, 16384)
            if rng.random() < 0.7:
                D = -(-D // 128) * 128
            if M * D <= 8192 * 5120 and 3072 not in (M, D):
                return dict(op=op, M=M, D=D, residual=rng.choice(("bf16", "fp32")),
                            post=rng.random() < 0.5, gate=rng.choice(("none", "channel", "token")),
                            out=rng.choice(("bf16", "codes")))
    while True:
        M, K = _log_between(rng, 1, 32768), 8 * _log_between(rng, 16, 1024)
        if rng.random() < 0.7:
            K = -(-K // 128) * 128
        if M * K <= 32768 * 768 and 3072 not in (M, K, 2 * K):
            return dict(op=op, M=M, K=K, gated=rng.random() < 0.6)


# ------------------------------------------------------------------- inputs --
def _groups(n):
    return -(-n // GROUP)


def _codes_1x128(x):
    """E4M3FN codes and fp32 scales [rows, ceil(K / 128)] of fp32 x [rows, K]."""
    rows, K = x.shape
    G = _groups(K)
    xp = torch.nn.functional.pad(x, (0, G * GROUP - K)).view(rows, G, GROUP)
    amax = xp.abs().amax(dim=2)
    s = torch.where(amax == 0, torch.ones_like(amax), amax / QMAX)
    q = (xp / s[:, :, None]).clamp(-QMAX, QMAX).to(E4M3)
    return q.view(torch.uint8).view(rows, G * GROUP)[:, :K].contiguous().view(E4M3), s


def _codes_blocks(w):
    """E4M3FN codes and fp32 scales [..., ceil(N / 128), ceil(K / 128)] of fp32 w [..., N, K]."""
    N, K = w.shape[-2:]
    NB, KB = _groups(N), _groups(K)
    wp = torch.nn.functional.pad(w, (0, KB * GROUP - K, 0, NB * GROUP - N))
    wp = wp.view(*w.shape[:-2], NB, GROUP, KB, GROUP)
    s = wp.abs().amax(dim=(-3, -1)) / QMAX
    q = (wp / s[..., :, None, :, None]).clamp(-QMAX, QMAX).to(E4M3)
    q = q.view(torch.uint8).view(*w.shape[:-2], NB * GROUP, KB * GROUP)[..., :N, :K]
    return q.contiguous().view(E4M3), s.contiguous()


def _routing(T, E, topk, g):
    """Top-k routing of T tokens over experts of unequal popularity: offsets
    int32 [E + 1], token rows int32 [T * topk] grouped by expert, largest count."""
    pop = 0.5 * torch.randn(E, generator=g, device="cuda")
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    experts = (pop - torch.log(-torch.log(u))).topk(topk, dim=1).indices.reshape(-1)
    order = experts.argsort(stable=True)
    counts = torch.bincount(experts, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, (order // topk).to(torch.int32), int(counts.max())


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    op = case["op"]
    s = dict(case)
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["xq"], s["sx"] = _codes_1x128(randn(M, K))
        s["wq"], s["sw"] = _codes_blocks(0.02 * randn(N, K))
    elif op == "grouped":
        T, E, N, K = case["T"], case["E"], case["N"], case["K"]
        s["offsets"], s["rows"], s["cap"] = _routing(T, E, case["topk"], g)
        if not case["gather"]:
            s["rows"] = None
        s["xq"], s["sx"] = _codes_1x128(randn(T if case["gather"] else T * case["topk"], K))
        s["wq"], s["sw"] = _codes_blocks(0.02 * randn(E, N, K))
    elif op == "norm":
        M, D = case["M"], case["D"]
        s["y"] = randn(M, D).to(torch.bfloat16)
        s["residual"] = 4 * randn(M, D)
        if case["residual"] == "bf16":
            s["residual"] = s["residual"].to(torch.bfloat16)
        s["weight"] = (1 + 0.1 * randn(D)).to(torch.bfloat16)
        s["post_weight"] = (1 + 0.1 * randn(D)).to(torch.bfloat16) if case["post"] else None
        s["gate"] = {"none": lambda: None,
                     "channel": lambda: randn(D).to(torch.bfloat16),
                     "token": lambda: randn(M, D).to(torch.bfloat16)}[case["gate"]]()
        s["scale"], s["eps"] = 0.7, 1e-6
    else:
        M, K = case["M"], case["K"]
        if case["gated"]:  # the two halves of one projection's output
            both = randn(M, 2 * K).to(torch.bfloat16)
            s["gate"], s["x"] = both[:, :K], both[:, K:]
        else:
            s["gate"], s["x"] = None, randn(M, K).to(torch.bfloat16)
    return s


# -------------------------------------------------------------- plain forms --
def _wide_x(q, s):
    K = q.shape[1]
    return q.float() * s.repeat_interleave(GROUP, dim=1)[:, :K]


def _wide_w(q, s):
    N, K = q.shape[-2:]
    wide = s.repeat_interleave(GROUP, dim=-2)[..., :N, :].repeat_interleave(GROUP, dim=-1)
    return q.float() * wide[..., :K]


def _plain_gemm(s):
    return (_wide_x(s["xq"], s["sx"]) @ _wide_w(s["wq"], s["sw"]).t()).to(torch.bfloat16)


def _plain_grouped(s):
    off = s["offsets"].long()
    n = s["T"] * s["topk"]
    entries = torch.arange(n, device=off.device)
    expert = torch.searchsorted(off[1:].contiguous(), entries, right=True)
    place = entries - off[expert]
    # every expert's rows, padded to the longest list
    slot = (off[:-1, None] + torch.arange(s["cap"], device=off.device)).clamp(max=n - 1)
    row = slot if s["rows"] is None else s["rows"].long()[slot]
    x = _wide_x(s["xq"], s["sx"])[row]
    y = torch.bmm(x, _wide_w(s["wq"], s["sw"]).transpose(1, 2))
    return y[expert, place].to(torch.bfloat16)


def _rms(v, eps):
    return v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + eps)


def _plain_norm(s):
    b = s["y"].float()
    if s["post_weight"] is not None:
        b = _rms(b, s["eps"]) * s["post_weight"].float()
    if s["gate"] is not None:
        b = b * s["gate"].float()
    h = s["residual"].float() + s["scale"] * b
    z = _rms(h, s["eps"]) * s["weight"].float()
    h = h.to(s["residual"].dtype)
    if s["out"] == "bf16":
        return h, z.to(torch.bfloat16)
    return h, *_codes_1x128(z)


def _plain_quantize(s):
    x = s["x"].float()
    if s["gate"] is not None:
        g = s["gate"].float()
        x = g / (1 + torch.exp(-g)) * x
    return _codes_1x128(x)


# --------------------------------------------------------------------- runs --
def _own(s):
    import bit_quantized_gemm_token_amd as w8
    op = s["op"]
    if op == "gemm":
        return w8.block_gemm(s["xq"], s["sx"], s["wq"], s["sw"])
    if op == "grouped":
        return w8.grouped_gemm(s["xq"], s["sx"], s["offsets"], s["wq"], s["sw"], rows=s["rows"])
    if op == "norm":
        return w8.residual_norm(s["y"], s["residual"], s["weight"], post_weight=s["post_weight"],
                                gate=s["gate"], scale=s["scale"], eps=s["eps"],
                                quantize=s["out"] == "codes")
    return w8.block_quantize(s["x"], gate=s["gate"])


def run(state):
    if own:
        return _own(state)
    return {"gemm": _plain_gemm, "grouped": _plain_grouped, "norm": _plain_norm,
            "quantize": _plain_quantize}[state["op"]](state)


# --------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * _groups(K) * (M + _groups(N))
        return {"bytes": M * K + N * K + 2 * M * N + scales, "flops": 2 * M * N * K}
    if op == "grouped":
        T, E, topk, N, K = (case[k] for k in ("T", "E", "topk", "N", "K"))
        n = T * topk
        rows = T if case["gather"] else n
        reached = E * (1 - (1 - topk / E) ** T)  # experts that any token chose, as expected
        b = rows * (K + 4 * _groups(K)) + reached * (N * K + 4 * _groups(N) * _groups(K))
        return {"bytes": b + 2 * n * N + 4 * (E + 1) + (4 * n if case["gather"] else 0),
                "flops": 2 * n * N * K}
    if op == "norm":
        M, D = case["M"], case["D"]
        r = 2 if case["residual"] == "bf16" else 4
        gate = {"none": 0, "channel": 2 * D, "token": 2 * M * D}[case["gate"]]
        out = 2 * M * D if case["out"] == "bf16" else M * (D + 4 * _groups(D))
        return {"bytes": M * D * (2 + 2 * r) + gate + 2 * D * (1 + case["post"]) + out,
                "flops": M * D * (5 + 4 * case["post"])}
    M, K = case["M"], case["K"]
    return {"bytes": M * K * (2 + 2 * case["gated"]) + M * (K + 4 * _groups(K)),
            "flops": M * K * (3 + 5 * case["gated"])}


# -------------------------------------------------------------------- exact --
def _exact_codes(v):
    """Codes and scales of 64-bit values by the definition: the nearest E4M3FN
    value of v / s (ties to even), a grid of 2^-9 below 2^-6 and of three
    fraction bits above."""
    M, K = v.shape
    G = _groups(K)
    p = torch.zeros(M, G * GROUP, dtype=torch.float64, device=v.device)
    p[:, :K] = v
    p = p.reshape(M, G, GROUP)
    top = p.abs().max(dim=2).values
    s = torch.where(top > 0, top / 448, torch.ones_like(top))
    t = p / s.unsqueeze(2)
    _, e = torch.frexp(t)  # |t| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(t), (e - 4).clamp(min=-9))
    q = (torch.round(t / step) * step).clamp(-448, 448)
    return q.reshape(M, G * GROUP)[:, :K], s


def _exact_product(xq, sx, wq, sw):
    M, K = xq.shape
    N = wq.shape[0]
    kg = torch.arange(K, device=xq.device) // GROUP
    ng = torch.arange(N, device=xq.device) // GROUP
    x = xq.double() * sx.double()[:, kg]
    w = wq.double() * sw.double()[ng][:, kg]
    return torch.mm(x, w.T.contiguous())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        return _exact_product(s["xq"], s["sx"], s["wq"], s["sw"])
    if op == "grouped":
        off = s["offsets"].tolist()
        out = torch.zeros(off[-1], case["N"], dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            if lo < hi:
                at = torch.arange(lo, hi, device="cuda") if s["rows"] is None else s["rows"][lo:hi].long()
                out[lo:hi] = _exact_product(s["xq"].view(torch.uint8)[at].view(E4M3), s["sx"][at],
                                            s["wq"][e], s["sw"][e])
        return out
    if op == "norm":
        y, D = s["y"].double(), case["D"]
        if s["post_weight"] is not None:
            y = s["post_weight"].double() * y / torch.sqrt((y * y).sum(1, keepdim=True) / D + s["eps"])
        if s["gate"] is not None:
            y = s["gate"].double() * y
        h = s["residual"].double() + s["scale"] * y
        z = s["weight"].double() * h / torch.sqrt((h * h).sum(1, keepdim=True) / D + s["eps"])
        return (h, z) if case["out"] == "bf16" else (h, *_exact_codes(z))
    x = s["x"].double()
    if s["gate"] is not None:
        x = x * s["gate"].double() * torch.sigmoid(s["gate"].double())
    return _exact_codes(x)
