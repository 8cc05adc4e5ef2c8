"""The tiled Block_FP8 GEMM's kernels compiled for the CPU and run there, one
workgroup at a time (hip/hip_runtime.h beside this file says how): what each
kernel reads and writes, and whether its result depends on which wavefront runs
first or on when a load arrives, can be checked without a GPU."""
import ctypes
import os
import shutil
import subprocess

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(os.path.dirname(HERE)), "bit_quantized_gemm_token_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"

# tile ids, tokens x weight rows (w8_block.hpp)
TILES = {"16x128": (0, 16, 128), "64x64": (1, 64, 64), "64x128": (2, 64, 128),
         "128x128": (3, 128, 128), "256x256": (4, 256, 256)}
COUNTERS = 16384 * 32  # words of the workspace's counter region
UNITS = 256            # compute units that a launch plan counts with
POISON = 0x7FC1        # a NaN that no kernel writes

_INTS = ("tile", "grouped", "packed", "descending", "late", "M", "N", "K", "split_k", "whole",
         "parts", "tiles_m", "tiles_n", "n_experts", "xrow_max")
_STRIDES = ("ldq", "ldw", "ldy", "w_stride", "sw_stride")
_POINTERS = ("xq", "sx", "wq", "sw", "y", "part", "counters", "offsets", "rows")
_BYTES = ("xq_bytes", "sx_bytes", "wq_bytes", "sw_bytes", "part_bytes")


class _Launch(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in _INTS] + [("wgs", ctypes.c_uint)] +
                [(n, ctypes.c_longlong) for n in _STRIDES] +
                [(n, ctypes.c_void_p) for n in _POINTERS] +
                [(n, ctypes.c_longlong) for n in _BYTES])


def build(folder):
    """Compiles the kernels into `folder`; returns the loaded library."""
    for name in ("w8_block_gemm.hip", "w8_block.hpp", "w8_device.hpp", "w8_launch.hpp"):
        shutil.copy(os.path.join(CSRC, name), folder)
    for name in ("w8_lds.hpp", "block_gemm.cpp"):
        shutil.copy(os.path.join(HERE, name), folder)
    out = os.path.join(folder, "block_gemm_host.so")
    subprocess.run([CLANG, "-O1", "-std=c++17", "-fPIC", "-shared", "-mavx2", "-w", "-I", HERE,
                    "-I", folder, "-o", out, os.path.join(folder, "block_gemm.cpp")], check=True)
    lib = ctypes.CDLL(out)
    lib.emu_gemm.argtypes, lib.emu_gemm.restype = [ctypes.POINTER(_Launch)], ctypes.c_longlong
    lib.emu_text.restype, lib.emu_loads.restype = ctypes.c_char_p, ctypes.c_longlong
    return lib


def pack(codes):
    """Codes [N, K] in the packed layout: fragments of 16 rows x 128 bytes in
    the order the lanes of an MFMA take them (two halves of 16 bytes a lane)."""
    N, K = codes.shape
    p = np.zeros((-(-N // 16) * 16, K), dtype=np.uint8)
    p[:N] = codes
    # [block, row, step, half, quarter of 16 bytes]: lane = 16 quarter + row
    v = p.reshape(-1, 16, K // 128, 2, 4, 16)
    return np.ascontiguousarray(v.transpose(0, 2, 3, 4, 1, 5)).reshape(-1)


def pieces(tiles):
    """Pieces of each tile of the largest tile's last round (w8_block.hpp)."""
    rest = tiles % UNITS
    return 1 if rest == 0 or rest > UNITS // 2 else 4 if rest <= UNITS // 4 else 2


def run(lib, tile, xq, sx, wq, sw, split_k=1, parts=None, packed=False, ldw=None, offsets=None,
        rows=None, descending=False, late=False, hide=0):
    """(y as float64 [M, N], faults, their text) of one launch.

    xq [T, K], sx [T, G]; wq [N, K] (with offsets [E, N, K]) and sw as the
    entry points take them.  Every buffer ends where its last row's K codes
    end.  parts: of the largest tile's tiles (1, 2 or 4; default as planned).
    hide: bytes at the weights' end that count as not theirs.
    """
    T, K = xq.shape
    grouped = offsets is not None
    N = wq.shape[-2]
    id_, bm, bn = TILES[tile]
    M = T if rows is None else len(rows)
    G = -(-K // 128)
    a = _Launch(tile=id_, grouped=grouped, packed=packed, descending=descending, late=late, M=M,
                N=N, K=K, split_k=split_k, xrow_max=T - 1, ldq=K, ldy=N + 3)
    keep = []

    def buffer(v):
        v = np.ascontiguousarray(v)
        raw = np.zeros(v.nbytes + 512, dtype=np.uint8)
        at = -raw.ctypes.data % 256 + 16  # 16-byte aligned, no more
        raw[at:at + v.nbytes] = v.reshape(-1).view(np.uint8)
        keep.append(raw)
        return raw.ctypes.data + at, v.nbytes

    a.xq, a.xq_bytes = buffer(xq)
    a.sx, a.sx_bytes = buffer(sx.astype(np.float32))
    a.sw, a.sw_bytes = buffer(sw.astype(np.float32))
    if packed:
        w = np.concatenate([pack(e) for e in wq]) if grouped else pack(wq)
        a.ldw = 0
    else:
        a.ldw = ldw or K
        w = np.full(wq.shape[:-1] + (a.ldw,), 0x7F, dtype=np.uint8)
        w[..., :K] = wq
        w = w.reshape(-1)[:w.size - (a.ldw - K)]
    a.wq, a.wq_bytes = buffer(w)
    a.wq_bytes -= hide
    E = wq.shape[0] if grouped else 1
    a.w_stride = len(w) // E if packed else N * a.ldw
    a.sw_stride = sw[0].size if grouped else 0
    a.tiles_n = -(-N // bn)
    if grouped:
        a.n_experts = E
        a.tiles_m = M // bm + min(E, M)
        a.wgs = a.tiles_m * a.tiles_n + (3 * UNITS // 4 if tile == "256x256" else 0)
        off = np.ascontiguousarray(offsets, dtype=np.int32)
        keep.append(off)
        a.offsets = off.ctypes.data
        if rows is not None:
            r = np.ascontiguousarray(rows, dtype=np.int32)
            keep.append(r)
            a.rows = r.ctypes.data
    else:
        a.tiles_m = -(-M // bm)
        tiles = a.tiles_m * a.tiles_n
        a.parts = (pieces(tiles) if parts is None else parts) if tile == "256x256" else 1
        a.whole = tiles if a.parts == 1 else tiles // UNITS * UNITS
        a.wgs = (a.whole + a.parts * (tiles - a.whole)) * split_k
        if split_k > 1:
            part = np.full(tiles * split_k * bm * bn, np.nan, dtype=np.float32)
            counters = np.zeros(COUNTERS, dtype=np.uint32)
            keep += [part, counters]
            a.part, a.part_bytes, a.counters = part.ctypes.data, part.nbytes, counters.ctypes.data
    guard = 64
    y = np.full(2 * guard + M * a.ldy, POISON, dtype=np.uint16)
    a.y = y.ctypes.data + 2 * guard
    faults = lib.emu_gemm(ctypes.byref(a))
    text = lib.emu_text().decode()
    body = y[guard:-guard].reshape(M, a.ldy)
    if (y[:guard] != POISON).any() or (y[-guard:] != POISON).any() or (body[:, N:] != POISON).any():
        faults += 1
        text += "a store outside the output's rows\n"
    out = (body[:, :N].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return out, faults, text
