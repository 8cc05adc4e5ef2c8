"""Block_FP8 operators for any token count (the C-ABI's w8_block_quantize,
w8_residual_norm, w8_block_gemm and w8_grouped_gemm).

Together they make a Block_FP8 layer whose token count is not bound to the
small-M window of gemm_w8a8 and moe_gemm: the residual update and norm between
two blocks, straight to codes; the quantizer with the gated activation in
front of it; the GEMM; and the GEMM per expert over ragged lists of rows.
Like the rest of the package this module only checks and marshals arguments.
"""
import ctypes

import torch

from . import _capi

GROUP = _capi.GROUP
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_CODES = torch.float8_e4m3fn
_E_WORKSPACE = 3


def _groups(n):
    return (n + GROUP - 1) // GROUP


# One call's checks run before every launch of a few microseconds, so the
# helpers below keep to the cheap attributes and build messages only on error.
def _not_rows(t, name, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return TypeError(f"{name} must be a CUDA (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        return TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ValueError(f"{name} must be a 2-D tensor with unit inner stride")


def _rows(t, name, dtype=None):
    """Pointer and row stride (elements) of a 2-D device tensor with unit inner stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (dtype is not None and
                                                            t.dtype is not dtype):
        raise _not_rows(t, name, dtype)
    st = t.stride()
    if len(st) != 2:
        raise _not_rows(t, name, dtype)
    ld, one = st
    rows, cols = t.shape
    if one != 1 and cols > 1:
        raise _not_rows(t, name, dtype)
    # (a single row's stride is never used, and torch lets it be anything)
    return t.data_ptr(), (ld if rows > 1 or ld >= cols else cols)


def _codes(t, name):
    p_ld = _rows(t, name)
    if t.element_size() != 1:
        raise TypeError(f"{name} must hold 1-byte codes")
    return p_ld


def _flat(t, name, dtype, n):
    """Pointer of a contiguous device tensor of n elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements, got shape "
                         f"{tuple(t.shape)}")
    return t.data_ptr()


def _shape(t, rows, cols, name):
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")


# Outputs that the caller did not give: the tensor, its pointer and row stride,
# which need no checks; allocated for the stream that the kernel runs on.
# (empty_strided costs the host about half of what empty does.)
def _new(rows, cols, dtype, device, stream):
    if stream is not None:
        t = _allocate(stream, device, lambda: _new(rows, cols, dtype, device, None)[0])
    else:
        t = torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)
    return t, t.data_ptr(), cols


def _new_codes(M, K, device, stream):
    """Codes [M, K] whose row stride the GEMMs take (a multiple of 16)."""
    t, p, ld = _new(M, (K + 15) // 16 * 16, _CODES, device, stream)
    return (t if ld == K else t[:, :K]), p, ld


def block_quantize(x, gate=None, xq=None, sx=None, stream=None):
    """E4M3FN codes [M, K] and fp32 scales [M, ceil(K/128)] of bf16 x [M, K],
    or with gate (bf16 [M, K]) of silu(gate) * x: the gated activation in
    front of a layer's last projection, fused into the quantizer.

    Each 1 x 128 group (the last may be shorter) takes s = amax / 448 (1 for
    an all-zero group) and codes round-to-nearest-even(x / s), as quantize_act
    does for Block_FP8; the gated product is not rounded before.  Any M; K a
    multiple of 8 (the GEMMs need 16); x and gate may be column slices of one
    tensor.  A group holding a NaN or an infinity gets a non-finite scale.
    """
    xp, ldx = _rows(x, "x", _BF16)
    M, K = x.shape
    gp, ldg = None, 0
    if gate is not None:
        gp, ldg = _rows(gate, "gate", _BF16)
        _shape(gate, M, K, "gate")
    if xq is None:
        xq, qp, ldq = _new_codes(M, K, x.device, stream)
    else:
        _shape(xq, M, K, "xq")
        qp, ldq = _codes(xq, "xq")
    if sx is None:
        sx, sp, _ = _new(M, _groups(K), _F32, x.device, stream)
    else:
        sp = _flat(sx, "sx", _F32, M * _groups(K))
    _check(_lib.w8_block_quantize(M, K, xp, ldx, gp, ldg, qp, ldq, sp, _handle(stream, x.device)))
    return xq, sx


def residual_norm(y, residual, weight, post_weight=None, gate=None, scale=1.0, eps=1e-6,
                  quantize=False, with_z=False, h=None, out=None, stream=None):
    """The residual update and the norm between two blocks, in one pass:

        h = residual + scale * gate * N(y; post_weight)
        z = N(h; weight),      N(v; w) = w * v / sqrt(mean(v^2) + eps)

    y: bf16 [M, D], a block's output; without post_weight it is taken as it
    is.  residual: bf16 or fp32 [M, D]; h has its type (h=residual updates it
    in place).  weight, post_weight: bf16 [D].  gate: bf16 [D] (the same for
    every row) or [M, D], or None for 1.

    Returns (h, z) with z bf16, or with quantize=True (h, zq, sz): z's
    Block_FP8 codes and scales, as block_quantize gives them for the unrounded
    z; with_z=True then adds z itself, (h, zq, sz, z), for a consumer beside
    the quantized ones (a router).  z is computed from the unrounded h, all in
    fp32.  out: z, or the pair (zq, sz), to write to.  Any M, 1 <= D <= 32768,
    any strides.
    """
    yp, ldy = _rows(y, "y", _BF16)
    M, D = y.shape
    rp, ldr = _rows(residual, "residual")
    if residual.dtype not in (_BF16, _F32):
        raise TypeError(f"residual must be bfloat16 or float32, got {residual.dtype}")
    _shape(residual, M, D, "residual")
    wp = _flat(weight, "weight", _BF16, D)
    pp = None if post_weight is None else _flat(post_weight, "post_weight", _BF16, D)
    gp, ldg = None, 0
    if gate is not None:
        if gate.dim() == 1:
            gp = _flat(gate, "gate", _BF16, D)
        else:
            gp, ldg = _rows(gate, "gate", _BF16)
            _shape(gate, M, D, "gate")
    if h is None:
        h, hp, ldh = _new(M, D, residual.dtype, y.device, stream)
    else:
        _shape(h, M, D, "h")
        hp, ldh = _rows(h, "h", residual.dtype)
    zp = qp = sp = None
    ldz = ldq = 0
    if quantize:
        if out is None:
            zq, qp, ldq = _new_codes(M, D, y.device, stream)
            sz, sp, _ = _new(M, _groups(D), _F32, y.device, stream)
        else:
            zq, sz = out
            _shape(zq, M, D, "zq")
            qp, ldq = _codes(zq, "zq")
            sp = _flat(sz, "sz", _F32, M * _groups(D))
        result = h, zq, sz
        if with_z:
            z, zp, ldz = _new(M, D, _BF16, y.device, stream)
            result = h, zq, sz, z
    else:
        if out is None:
            z, zp, ldz = _new(M, D, _BF16, y.device, stream)
        else:
            z = out
            _shape(z, M, D, "out")
            zp, ldz = _rows(z, "out", _BF16)
        result = h, z
    _check(_lib.w8_residual_norm(M, D, yp, ldy, rp, ldr, residual.dtype == _F32, pp, gp, ldg,
                                 scale, wp, eps, hp, ldh, zp, ldz, qp, ldq, sp,
                                 _handle(stream, y.device)))
    return result


def block_gemm_workspace_size(M, N, K, packed=False):
    """Bytes of workspace block_gemm needs for the shape (0 for most)."""
    n = ctypes.c_size_t(0)
    _check(_lib.w8_block_gemm_workspace_size(M, N, K, _layout(packed), ctypes.byref(n)))
    return n.value


def block_gemm_plan(M, N, K, packed=False):
    """What block_gemm runs for the shape: tile_m x tile_n (tokens x weight
    rows of a workgroup; 0 x 0 where the small-M GEMM runs), split_k, parts
    (pieces of each tile in the last, partial round) and workgroups.  Host only."""
    p = _capi.BlockPlan()
    _check(_lib.w8_block_gemm_plan(M, N, K, _layout(packed), ctypes.byref(p)))
    return p.as_dict()


def grouped_gemm_plan(E, T, N, K, n_rows=None, ldq=None):
    """What grouped_gemm runs for n_rows entries (default T) of E experts on T
    token rows of stride ldq (default K), as block_gemm_plan says it."""
    p = _capi.BlockPlan()
    _check(_lib.w8_grouped_gemm_plan(E, T, N, K, K if ldq is None else ldq,
                                     T if n_rows is None else n_rows, ctypes.byref(p)))
    return p.as_dict()


def block_gemm(xq, sx, wq, sw, y=None, workspace=None, stream=None):
    """Y = dequant(xq) . dequant(wq)^T as bf16 [M, N] in Block_FP8, any M.

    xq, sx: codes [M, K] and scales [M, ceil(K/128)] (block_quantize,
    residual_norm, quantize_act); wq, sw: codes [N, K] or a PackedWeight of
    layout 1, scales [ceil(N/128), ceil(K/128)] (quantize_weight).  K a
    multiple of 16 (packed: of 128); its last group may be shorter.

    workspace: a Workspace of the stream's own (calls that overlap must not
    share one), for shapes that block_gemm_workspace_size gives bytes for;
    None takes the package's for the stream.
    """
    xp, ldq = _codes(xq, "xq")
    M, K = xq.shape
    if isinstance(wq, PackedWeight):
        if wq.fmt != _capi.FORMATS["Block_FP8"] or wq.layout != 1:
            raise ValueError("packed weights must be Block_FP8 in layout 1")
        N, wk, wp, ldw, packed = wq.N, wq.K, wq.data.data_ptr(), 0, 1
    else:
        (wp, ldw), (N, wk), packed = _codes(wq, "wq"), wq.shape, 0
        ldw = _weight_stride(ldw, N, wk)
    if wk != K:
        raise ValueError(f"K mismatch: xq {tuple(xq.shape)} vs weights {(N, wk)}")
    G = _groups(K)
    sxp, swp = _flat(sx, "sx", _F32, M * G), _flat(sw, "sw", _F32, _groups(N) * G)
    if y is None:
        y, yp, ldy = _new(M, N, _BF16, xq.device, stream)
    else:
        _shape(y, M, N, "y")
        yp, ldy = _rows(y, "y", _BF16)
    s = _handle(stream, xq.device)
    if workspace is None:
        workspace = _workspace_of(xq.device, s)
    # what the workspace holds is enough for most calls: its size is asked for
    # only when the library says it is not
    buf = workspace.buf
    for retry in (True, False):
        status = _lib.w8_block_gemm(M, N, K, xp, ldq, sxp, wp, ldw, swp, yp, ldy,
                                    None if buf is None else buf.data_ptr(),
                                    0 if buf is None else buf.numel(), s)
        if status != _E_WORKSPACE or not retry:
            break
        buf = workspace.reserve(block_gemm_workspace_size(M, N, K, packed), stream)
    _check(status)
    return y


def grouped_gemm(xq, sx, offsets, wq, sw, rows=None, y=None, stream=None):
    """The Block_FP8 GEMM per expert over ragged lists of rows, any counts:
    for entry i of expert e (offsets[e] <= i < offsets[e + 1])

        Y[i] = dequant(xq[rows[i]]) . dequant(wq[e])^T      (bf16 [n_rows, N])

    xq, sx: codes [T, K] and scales [T, ceil(K/128)]; offsets: int32 [E + 1]
    on the device, ascending from 0 to the number of entries; rows: int32
    [n_rows], the token row of each entry, or None where the entries are the
    rows of xq in order; wq: [E, N, K] codes or PackedExperts; sw: [E,
    ceil(N/128), ceil(K/128)].  Experts without entries read nothing.  One
    launch, no host sync; bad offsets and rows are clamped to the arrays.
    """
    xp, ldq = _codes(xq, "xq")
    T, K = xq.shape
    if isinstance(wq, PackedExperts):
        if wq.fmt != _capi.FORMATS["Block_FP8"]:
            raise ValueError("experts were packed for another format")
        E, N, wk = wq.E, wq.N, wq.K
        wp, ldw, w_stride = wq.data.data_ptr(), 0, wq.data.stride(0)
    else:
        if not isinstance(wq, torch.Tensor) or not wq.is_cuda:
            raise TypeError("wq must be a CUDA (HIP) tensor or PackedExperts")
        if wq.dim() != 3 or wq.element_size() != 1 or wq.stride(2) != 1:
            raise ValueError("wq must be [E, N, K] 1-byte codes with unit inner stride")
        E, N, wk = wq.shape
        wp, ldw, w_stride = wq.data_ptr(), _weight_stride(wq.stride(1), N, wk), wq.stride(0)
    if wk != K:
        raise ValueError(f"K mismatch: xq {tuple(xq.shape)} vs experts' K {wk}")
    G = _groups(K)
    sxp = _flat(sx, "sx", _F32, T * G)
    per = _groups(N) * G
    swp = _flat(sw, "sw", _F32, E * per)
    op = _flat(offsets, "offsets", _I32, E + 1)
    n_rows = T if rows is None else rows.numel()
    rwp = None if rows is None else _flat(rows, "rows", _I32, n_rows)
    if y is None:
        y, yp, ldy = _new(n_rows, N, _BF16, xq.device, stream)
    else:
        _shape(y, n_rows, N, "y")
        yp, ldy = _rows(y, "y", _BF16)
    _check(_lib.w8_grouped_gemm(E, T, N, K, xp, ldq, sxp, op, rwp, n_rows, wp, ldw, w_stride,
                                swp, per, yp, ldy, _handle(stream, xq.device)))
    return y


# (the package's own helpers; __init__ imports this module after defining them)
from . import (PackedExperts, PackedWeight, _allocate, _check, _handle, _layout, _lib,  # noqa: E402
               _weight_stride, _workspace_of)
