"""The token-scaled formats (W8A8_INT8, FP8_Dynamic) for any token count (the
C-ABI's w8_token_quantize and w8_token_gemm): codes with one scale per token,
with the gated activation in front where there is one, and the product with
weights of one scale per output channel.  Like the rest of the package this
module only checks and marshals arguments.
"""
import ctypes

import torch

from . import _capi
from .block import _BF16, _CODES, _E_WORKSPACE, _F32, _codes, _flat, _new, _rows, _shape

_I8 = torch.int8
_INT8 = _capi.FORMATS["W8A8_INT8"]
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device


def _one_device(x, *others):
    """The index of the device that x and the others (or None) are on."""
    index = x.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on {x.device}, got one on {t.device}")
    return index


def _elsewhere(index, entry, args):
    """entry(*args) on a device that is not the current one (the library launches on that)."""
    with torch.cuda.device(index):
        return entry(*args)


def token_quantize(fmt, x, gate=None, reciprocal=False, xq=None, sx=None, stream=None):
    """Codes [M, K] (int8 or float8_e4m3fn) and fp32 scales [M] of bf16 x [M, K],
    or with gate (bf16 [M, K]) of silu(gate) * x: the gated activation in front
    of a layer's last projection, fused into the quantizer.

    fmt: "W8A8_INT8" or "FP8_Dynamic" (Block_FP8: block_quantize).  Each row
    takes s = amax / 127 or / 448 (1 for a row of zeros) and codes
    round-to-nearest-even(x / s), as quantize_act does; the gated product is
    not rounded before.  Any M; K a multiple of 8 (the GEMMs need 16); x and
    gate may be column slices of one tensor.  A row holding a NaN or an
    infinity gets a non-finite scale.  Codes that it allocates itself have rows of
    whole 128 bytes from K = 512 on.

    reciprocal=True takes s = amax * (1 / Qmax) with the reciprocal rounded
    first, which is what torch's amax / Qmax computes on the GPU: for codes and
    scales bit for bit those of a model that was quantized there.
    """
    f = _fmt(fmt)
    xp, ldx = _rows(x, "x", _BF16)
    M, K = x.shape
    gp, ldg = None, 0
    if gate is not None:
        gp, ldg = _rows(gate, "gate", _BF16)
        _shape(gate, M, K, "gate")
    index = _one_device(x, gate, xq, sx)
    dev = x.device
    if xq is None:
        xq, qp, ldq = _new_codes(M, K, _I8 if f == _INT8 else _CODES, dev, stream)
    else:
        _shape(xq, M, K, "xq")
        qp, ldq = _codes(xq, "xq")
    if sx is None:
        sx, sp = _new_flat(M, _F32, dev, stream)
    else:
        sp = _flat(sx, "sx", _F32, M)
    args = (f, M, K, xp, ldx, gp, ldg, 1 if reciprocal else 0, qp, ldq, sp, _handle(stream, dev))
    status = _quantize(*args) if index == _current_device() else _elsewhere(index, _quantize, args)
    if status:
        _check(status)
    return xq, sx


def _new_codes(M, K, dtype, device, stream):
    """Codes [M, K] and their row stride, which the GEMMs take (a multiple of 16): rows
    of 512 and more begin on 128-byte lines, so that a K-step of one reads one line
    (token_gemm of 496 x 1706 x 7248 in int8, the codes' rows from end to end 19.5 us,
    on lines 15.6, the weights' too 13.4)."""
    ld = (K + 127) // 128 * 128 if K >= 512 else (K + 15) // 16 * 16
    if stream is not None:
        t = _allocate(stream, device, lambda: _new_codes(M, K, dtype, device, None)[0])
    else:
        t = torch.empty_strided((M, K), (ld, 1), dtype=dtype, device=device)
    return t, t.data_ptr(), ld


def _new_flat(n, dtype, device, stream):
    """A new vector of n elements and its pointer."""
    if stream is not None:
        t = _allocate(stream, device, lambda: _new_flat(n, dtype, device, None)[0])
    else:
        t = torch.empty_strided((n,), (1,), dtype=dtype, device=device)
    return t, t.data_ptr()


def token_gemm_workspace_size(fmt, M, N, K, packed=False):
    """Bytes of workspace token_gemm needs for the shape (0 for most)."""
    n = ctypes.c_size_t(0)
    _check(_lib.w8_token_gemm_workspace_size(_fmt(fmt), M, N, K, _layout(packed), ctypes.byref(n)))
    return n.value


def token_gemm_plan(fmt, M, N, K, packed=False):
    """What token_gemm runs for the shape, as block_gemm_plan says it.  Host only."""
    p = _capi.BlockPlan()
    _check(_lib.w8_token_gemm_plan(_fmt(fmt), M, N, K, _layout(packed), ctypes.byref(p)))
    return p.as_dict()


def token_gemm(fmt, xq, sx, wq, sw, y=None, workspace=None, stream=None):
    """Y = dequant(xq) . dequant(wq)^T as bf16 [M, N] in W8A8_INT8 or
    FP8_Dynamic, any M:

        Y[m, n] = sx[m] sw[n] sum_k xq[m, k] wq[n, k]

    xq, sx: codes [M, K] and scales [M] (token_quantize, quantize_act); wq, sw:
    codes [N, K] or a PackedWeight of layout 1, scales [N].  K a multiple of 16
    (packed: of 128).  W8A8_INT8's sums are exact (int32; K at most 131056).  Rows
    of codes are read fastest where they begin on 128-byte lines (row strides of
    whole 128 bytes).

    workspace: a Workspace of the stream's own (calls that overlap must not
    share one), for shapes that token_gemm_workspace_size gives bytes for; None
    takes the package's for the stream.
    """
    f = _fmt(fmt)
    xp, ldq = _codes(xq, "xq")
    M, K = xq.shape
    if isinstance(wq, PackedWeight):
        if wq.fmt != f or wq.layout != 1:
            raise ValueError("packed weights must be of the same format, in layout 1")
        N, wk, wt, ldw, packed = wq.N, wq.K, wq.data, 0, 1
        wp = wt.data_ptr()
    else:
        (wp, ldw), (N, wk), wt, packed = _codes(wq, "wq"), wq.shape, wq, 0
        ldw = _weight_stride(ldw, N, wk)
    if wk != K:
        raise ValueError(f"K mismatch: xq {tuple(xq.shape)} vs weights {(N, wk)}")
    sxp, swp = _flat(sx, "sx", _F32, M), _flat(sw, "sw", _F32, N)
    index = _one_device(xq, sx, wt, sw, y)
    dev = xq.device
    if y is None:
        y, yp, ldy = _new(M, N, _BF16, dev, stream)
    else:
        _shape(y, M, N, "y")
        yp, ldy = _rows(y, "y", _BF16)
    s = _handle(stream, dev)
    if workspace is None:
        workspace = _workspace_of(dev, s)
    # (what the workspace holds is enough for most calls, as in block_gemm)
    buf = workspace.buf
    for retry in (True, False):
        args = (f, M, N, K, xp, ldq, sxp, wp, ldw, swp, yp, ldy,
                None if buf is None else buf.data_ptr(), 0 if buf is None else buf.numel(), s)
        status = _gemm(*args) if index == _current_device() else _elsewhere(index, _gemm, args)
        if status != _E_WORKSPACE or not retry:
            break
        buf = workspace.reserve(token_gemm_workspace_size(f, M, N, K, packed), stream)
    if status:
        _check(status)
    return y


# (the package's own helpers; __init__ imports this module after defining them)
from . import (PackedWeight, _allocate, _check, _fmt, _handle, _layout, _lib,  # noqa: E402
               _weight_stride, _workspace_of)

_quantize, _gemm = _lib.w8_token_quantize, _lib.w8_token_gemm
