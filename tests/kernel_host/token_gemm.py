"""The tiled GEMM of the token-scaled formats compiled for the CPU and run there,
one workgroup at a time, as gemm.py does it for Block_FP8."""
import ctypes
import os
import shutil
import subprocess

import numpy as np

from .gemm import CLANG, COUNTERS, CSRC, HERE, POISON, TILES, UNITS, pack, pieces

FMT = {"FP8_Dynamic": 0, "W8A8_INT8": 1}

_INTS = ("fmt", "tile", "packed", "descending", "late", "M", "N", "K", "split_k", "whole",
         "parts", "tiles_m", "tiles_n")
_STRIDES = ("ldq", "ldw", "ldy")
_POINTERS = ("xq", "sx", "wq", "sw", "y", "part", "counters")
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
    for name in ("w8_lds.hpp", "token_gemm.cpp"):
        shutil.copy(os.path.join(HERE, name), folder)
    out = os.path.join(folder, "token_gemm_host.so")
    subprocess.run([CLANG, "-O1", "-std=c++17", "-fPIC", "-shared", "-mavx2", "-w", "-I", HERE,
                    "-I", folder, "-o", out, os.path.join(folder, "token_gemm.cpp")], check=True)
    lib = ctypes.CDLL(out)
    lib.emu_token.argtypes, lib.emu_token.restype = [ctypes.POINTER(_Launch)], ctypes.c_longlong
    lib.emu_text.restype = ctypes.c_char_p
    return lib


def run(lib, fmt, tile, xq, sx, wq, sw, split_k=1, parts=None, packed=False, descending=False,
        late=False, hide=None):
    """(y's bf16 bits [M, N], faults, their text) of one launch.  Every buffer
    ends where its last element does; hide: the name of a buffer whose last 16
    bytes count as not its own."""
    M, K = xq.shape
    N = len(wq)
    id_, bm, bn = TILES[tile]
    a = _Launch(fmt=FMT[fmt], tile=id_, packed=packed, descending=descending, late=late, M=M, N=N,
                K=K, split_k=split_k, ldq=K, ldw=0 if packed else K, ldy=N + 3)
    keep = []

    def buffer(name, v):
        v = np.ascontiguousarray(v)
        raw = np.zeros(v.nbytes + 512, dtype=np.uint8)
        at = -raw.ctypes.data % 256 + 16  # 16-byte aligned, no more
        raw[at:at + v.nbytes] = v.reshape(-1).view(np.uint8)
        keep.append(raw)
        setattr(a, name, raw.ctypes.data + at)
        setattr(a, name + "_bytes", v.nbytes - (16 if hide == name else 0))

    buffer("xq", xq)
    buffer("sx", sx)
    buffer("wq", pack(wq) if packed else wq)
    buffer("sw", sw)
    a.tiles_m, a.tiles_n = -(-M // bm), -(-N // bn)
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
    faults = lib.emu_token(ctypes.byref(a))
    text = lib.emu_text().decode()
    body = y[guard:-guard].reshape(M, a.ldy)
    if (y[:guard] != POISON).any() or (y[-guard:] != POISON).any() or (body[:, N:] != POISON).any():
        faults += 1
        text += "a store outside the output's rows\n"
    return body[:, :N], faults, text
