"""The MoE layer around the grouped products (the C-ABI's w8_moe_route,
w8_moe_combine and w8_moe_layer): the routing that makes the lists which
moe_gemm, moe_linear and grouped_gemm take, the weighted sum of their outputs,
and for a few tokens the experts as a whole in two launches or three.  Like the rest of
the package this module only checks and marshals arguments.
"""
import ctypes

import torch

from . import _capi
from .block import _BF16, _E_WORKSPACE, _F32, _I32, _codes, _flat, _new, _rows, _shape
from .tokens import _current_device, _elsewhere, _new_flat, _one_device

_BLOCK = _capi.FORMATS["Block_FP8"]
_GROUP = _capi.GROUP


def moe_route_workspace_size(T, E, topk):
    """Bytes of workspace moe_route needs for its lists (0 for few tokens)."""
    n = ctypes.c_size_t(0)
    _check(_lib.w8_moe_route_workspace_size(T, E, topk, ctypes.byref(n)))
    return n.value


def moe_route(logits, topk, renormalize=True, scale=1.0, lists=True, workspace=None, stream=None):
    """Top-k routing of T tokens over E experts from the router's logits
    (bf16 or fp32 [T, E]).

    Returns (experts, weights, offsets, rows, slots), or with lists=False
    (experts, weights):

      experts  int32 [T, topk], the topk largest logits' experts in descending
               order, ties to the lowest; -inf and NaN are never chosen, and
               where fewer are left the choice is -1
      weights  fp32 [T, topk]: scale times the softmax over the chosen
               (renormalize) or over all experts; 0 for a choice of -1
      offsets  int32 [E + 1], rows int32 [T * topk]: the entries (token,
               choice) in order, grouped by expert, as moe_gemm, moe_linear and
               grouped_gemm take them (rows: the token of each, 0 behind
               offsets[E])
      slots    int32 [T, topk]: where in rows each choice went, or -1 (for
               moe_combine)

    topk at most 32 and E, E at most 1024.  One launch for T * topk up to 256
    entries (fewer above 256 experts), else two; whole numbers only, the same
    every time.  experts, weights and slots are parts of one allocation, offsets
    and rows of another: one that is kept keeps its allocation.  workspace: as for
    block_gemm.
    """
    lp, ldl = _rows(logits, "logits")
    if logits.dtype is not _F32 and logits.dtype is not _BF16:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    T, E = logits.shape
    if topk < 1:
        moe_route_workspace_size(T, E, topk)  # (raises)
    dev, index, n = logits.device, logits.get_device(), T * topk
    s = _handle(stream, dev)
    op = rp = sp = buf = None
    if lists:
        # two allocations for the five outputs, in rows of topk and flat (a tensor
        # of its own costs the host 1.4 us, a part of one 0.4)
        table, wp, _ = _new(3 * T, topk, _I32, dev, stream)
        weights, experts, slots = _split(table, (T, T, T))
        weights = weights.view(_F32)
        flat, rp = _new_flat(n + E + 1, _I32, dev, stream)
        rows, offsets = _split(flat, (n, E + 1))
        ep, sp, op = wp + 4 * n, wp + 8 * n, rp + 4 * n
        if n > 256 or (E > 256 and T > 16):  # (the calls that may take two launches)
            if workspace is None:
                workspace = _workspace_of(dev, s)
            buf = workspace.buf
    else:
        experts, ep, _ = _new(T, topk, _I32, dev, stream)
        weights, wp, _ = _new(T, topk, _F32, dev, stream)
    for retry in (True, False):
        args = (T, E, topk, lp, ldl, 1 if logits.dtype is _F32 else 0, 1 if renormalize else 0,
                scale, ep, wp, op, rp, sp, None if buf is None else buf.data_ptr(),
                0 if buf is None else buf.numel(), s)
        status = _route(*args) if index == _current_device() else _elsewhere(index, _route, args)
        if status != _E_WORKSPACE or not retry:
            break
        if workspace is None:
            workspace = _workspace_of(dev, s)
        buf = workspace.reserve(moe_route_workspace_size(T, E, topk), stream)
    if status:
        _check(status)
    return (experts, weights, offsets, rows, slots) if lists else (experts, weights)


def _weights_of(weights, T, topk):
    """Pointer of the choices' weights: contiguous fp32 [T, topk].  (As many elements
    in another order, [topk, T] say, are other weights.)"""
    p = _flat(weights, "weights", _F32, T * topk)
    _shape(weights, T, topk, "weights")
    return p


def moe_combine(y, weights, slots, base=None, out=None, stream=None):
    """Each token's sum of its experts' outputs, bf16 [T, D]:

        out[t] = base[t] + sum_j weights[t, j] y[slots[t, j]]

    y: bf16 [n_rows, D], one row an entry (grouped_gemm, moe_gemm); weights
    fp32, slots int32 [T, topk] (moe_route); slots outside [0, n_rows) are left
    out.  base: bf16 [T, D] (a shared expert's output, a residual) or None;
    out may be base.  In fp32 in the order of the choices, rounded once.
    """
    yp, ldy = _rows(y, "y", _BF16)
    n_rows, D = y.shape
    if not isinstance(slots, torch.Tensor) or slots.dim() != 2:
        raise ValueError("slots must be an int32 [T, topk] tensor")
    T, topk = slots.shape
    sp = _flat(slots, "slots", _I32, T * topk)
    wp = _weights_of(weights, T, topk)
    bp, ldb = None, 0
    if base is not None:
        bp, ldb = _rows(base, "base", _BF16)
        _shape(base, T, D, "base")
    index = _one_device(y, weights, slots, base, out)
    dev = y.device
    if out is None:
        out, outp, ldo = _new(T, D, _BF16, dev, stream)
    else:
        _shape(out, T, D, "out")
        outp, ldo = _rows(out, "out", _BF16)
    args = (T, topk, D, yp, ldy, n_rows, wp, sp, bp, ldb, outp, ldo, _handle(stream, dev))
    status = _combine(*args) if index == _current_device() else _elsewhere(index, _combine, args)
    if status:
        _check(status)
    return out


def _scales(s, name, shape):
    """Pointer of contiguous fp32 scales: of that shape, or in another number of
    dimensions."""
    n = 1
    for size in shape:
        n *= size
    p = _flat(s, name, _F32, n)
    if s.dim() == len(shape) and s.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(s.shape)}")
    return p


def moe_layer_workspace_size(T, topk, D, I):
    """Bytes of workspace moe_layer needs."""
    n = ctypes.c_size_t(0)
    _check(_lib.w8_moe_layer_workspace_size(T, topk, D, I, ctypes.byref(n)))
    return n.value


def _layer_weights(f, w, s, name):
    """(E, N, K, pointer, ldw, stride, scales' pointer and stride, tensor) of
    [E, N, K] codes or PackedExperts and their scales."""
    if isinstance(w, PackedExperts):
        if w.fmt != f:
            raise ValueError("experts were packed for another format")
        E, N, K, t = w.E, w.N, w.K, w.data
        ldw, stride = 0, t.stride(0)
    else:
        if not isinstance(w, torch.Tensor) or not w.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor or PackedExperts")
        if w.dim() != 3 or w.element_size() != 1 or w.stride(2) != 1:
            raise ValueError(f"{name} must be [E, N, K] 1-byte codes with unit inner stride")
        E, N, K = w.shape
        stride, ld, _ = w.stride()
        ldw, t = _weight_stride(ld, N, K), w
    per = (N,) if f != _BLOCK else (-(-N // _GROUP), -(-K // _GROUP))
    sp = _scales(s, "the scales of " + name, (E, *per))
    return E, N, K, t.data_ptr(), ldw, stride, sp, per[0] * per[-1] if f == _BLOCK else N, t


def moe_layer(fmt, xq, sx, experts, weights, w1, s1, w2, s2, base=None, y=None, workspace=None,
              stream=None):
    """The experts of a few tokens (T <= 32) as a whole, bf16 [T, D]:

        a = x W1_e^T             [2 I]: gate, then up
        v = silu(a[:I]) * a[I:]  quantized as the format's activations
        y[t] = base[t] + sum_j weights[t, j] (v W2_e^T),   e = experts[t, j]

    fmt: any of the three.  xq, sx: codes [T, D] and scales as the GEMMs take
    them (quantize_act, token_quantize, residual_norm); experts int32, weights
    fp32 [T, topk] (moe_route); experts outside [0, E) are left out, an expert
    chosen twice counts with both weights.  w1: [E, 2 I, D], w2: [E, D, I]
    codes or PackedExperts; s1, s2: their scales, per output channel ([E, 2 I],
    [E, D]) or Block_FP8's per 128 x 128 block.  D and I are multiples of 16
    (Block_FP8: of 128) up to 65536, E at most 1024, topk at most 32.  base:
    bf16 [T, D] (a shared expert's output, a residual) or None; y may be base.

    Two launches (three where many tokens share an expert), no lists, no host
    sync; the hidden values stay fp32 until they are quantized (by a division, as
    token_quantize without reciprocal) and the sum is fp32 in the order of the
    choices, so results are the same every time.  W8A8_INT8's products are exact
    whole numbers, scaled once: a token's outputs are the same bits whoever else
    is in the call.  workspace: as for block_gemm, moe_layer_workspace_size bytes.
    """
    f = _fmt(fmt)
    xp, ldq = _codes(xq, "xq")
    T, D = xq.shape
    sxp = _scales(sx, "sx", (T, -(-D // _GROUP)) if f == _BLOCK else (T,))
    if not isinstance(experts, torch.Tensor) or experts.dim() != 2 or experts.shape[0] != T:
        raise ValueError(f"experts must be an int32 [{T}, topk] tensor")
    topk = experts.shape[1]
    ep = _flat(experts, "experts", _I32, T * topk)
    wp = _weights_of(weights, T, topk)
    E, N1, K1, w1p, ldw1, w1s, s1p, s1s, w1t = _layer_weights(f, w1, s1, "w1")
    E2, N2, I, w2p, ldw2, w2s, s2p, s2s, w2t = _layer_weights(f, w2, s2, "w2")
    if E2 != E or N1 != 2 * I or K1 != D or N2 != D:
        raise ValueError(f"w1 [{E}, {N1}, {K1}] and w2 [{E2}, {N2}, {I}] must be [E, 2 I, {D}] and "
                         f"[E, {D}, I]")
    bp, ldb = None, 0
    if base is not None:
        bp, ldb = _rows(base, "base", _BF16)
        _shape(base, T, D, "base")
    index = _one_device(xq, sx, experts, weights, w1t, s1, w2t, s2, base, y)
    dev = xq.device
    if y is None:
        y, yp, ldy = _new(T, D, _BF16, dev, stream)
    else:
        _shape(y, T, D, "y")
        yp, ldy = _rows(y, "y", _BF16)
    s = _handle(stream, dev)
    if workspace is None:
        workspace = _workspace_of(dev, s)
    buf = workspace.buf
    for retry in (True, False):
        args = (f, E, T, topk, D, I, xp, ldq, sxp, ep, wp, w1p, ldw1, w1s, s1p, s1s, w2p, ldw2,
                w2s, s2p, s2s, bp, ldb, yp, ldy, None if buf is None else buf.data_ptr(),
                0 if buf is None else buf.numel(), s)
        status = _layer(*args) if index == _current_device() else _elsewhere(index, _layer, args)
        if status != _E_WORKSPACE or not retry:
            break
        buf = workspace.reserve(moe_layer_workspace_size(T, topk, D, I), stream)
    if status:
        _check(status)
    return y


# (the package's own helpers; __init__ imports this module after defining them)
from . import (PackedExperts, _check, _fmt, _handle, _lib, _weight_stride,  # noqa: E402
               _workspace_of)

_route, _combine, _layer = _lib.w8_moe_route, _lib.w8_moe_combine, _lib.w8_moe_layer
_split = torch.unsafe_split_with_sizes
