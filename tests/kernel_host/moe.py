"""The MoE operators and the token-scaled quantizer compiled for the CPU and run
there, launch by launch and workgroup by workgroup, behind their C-ABI.  Every
buffer ends (or begins) at a page that cannot be touched."""
import ctypes
import os
import re
import subprocess

import numpy as np

from .gemm import CLANG, CSRC, HERE

FMT = {"FP8_Dynamic": 0, "W8A8_INT8": 1, "Block_FP8": 2}
GUARD = 0x5A


def build(folder):
    """Compiles the kernels into `folder`; returns the loaded library."""
    with open(os.path.join(CSRC, "w8_moe_layer.hip")) as f:
        source = f.read()
    # the dynamic LDS by a pointer, which a launch sets
    source, n = re.subn(r"extern __shared__ __align__\(16\) uint8_t codes\[\];",
                        "}\nextern uint8_t* g_dynamic_lds;\nnamespace {\nuint8_t*& codes = g_dynamic_lds;",
                        source)
    assert n == 1
    layer = os.path.join(folder, "w8_moe_layer.hip")
    with open(layer, "w") as f:
        f.write(source)
    files = [layer, *(os.path.join(CSRC, n) for n in ("w8_route.hip", "w8_rows.hip", "w8_route.cpp")),
             os.path.join(HERE, "moe.cpp")]
    jobs, objects = [], []
    for f in files:
        objects.append(os.path.join(folder, os.path.basename(f) + ".o"))
        jobs.append(subprocess.Popen(
            [CLANG, "-x", "c++", "-O1", "-std=c++17", "-fPIC", "-mavx2", "-mfma", "-w",
             "-ffp-contract=off", "-I", HERE, "-I", CSRC, "-include",
             os.path.join(HERE, "moe_device.hpp"), "-c", f, "-o", objects[-1]]))
    assert all([j.wait() == 0 for j in jobs])
    out = os.path.join(folder, "moe_host.so")
    subprocess.run([CLANG, "-shared", "-o", out, *objects], check=True)
    lib = ctypes.CDLL(out)
    lib.emu_buffer.restype = ctypes.c_void_p
    lib.emu_text.restype = ctypes.c_char_p
    lib.emu_layer_workspace.restype = lib.emu_route_workspace.restype = ctypes.c_longlong
    return lib


class Buffers:
    """The arrays of one call, each in pages of its own."""

    def __init__(self, lib, at_end, short=None):
        self.lib, self.at_end, self.short, self.of = lib, at_end, short, {}
        lib.emu_free_all()
        lib.emu_lds_at_end(int(at_end))

    def new(self, name, nbytes):
        p = self.lib.emu_buffer(name.encode(), ctypes.c_longlong(nbytes), int(self.at_end))
        self.of[name] = ctypes.c_void_p(p)
        return self.of[name]

    def put(self, name, v):
        v = np.ascontiguousarray(v)
        # (short: the name of an array whose last element, or 16 codes, are not there)
        nbytes = v.nbytes - (0 if name != self.short else 16 if v.itemsize == 1 else v.itemsize)
        p = self.new(name, nbytes)
        ctypes.memmove(p, v.ctypes.data, nbytes)
        return p

    def rows(self, name, v, ld):
        """A matrix of rows `ld` elements apart, nothing behind the last one's end."""
        v = np.ascontiguousarray(v)
        flat = np.full((len(v) - 1) * ld + v.shape[1], np.frombuffer(bytes([GUARD] * v.itemsize), v.dtype)[0])
        for i, r in enumerate(v):
            flat[i * ld:i * ld + len(r)] = r
        return self.put(name, flat)

    def get(self, name, dtype, n):
        p = self.of[name].value
        return np.frombuffer((ctypes.c_uint8 * (n * np.dtype(dtype).itemsize)).from_address(p),
                             dtype=dtype, count=n).copy()

    def get_rows(self, name, rows, cols, ld):
        """(bf16 bits [rows, cols], whether what lies between the rows is as it was)."""
        flat = self.get(name, np.uint16, (rows - 1) * ld + cols)
        flat = np.concatenate([flat, np.full(ld - cols, GUARD * 257, np.uint16)]).reshape(rows, ld)
        return flat[:, :cols], bool((flat[:, cols:] == GUARD * 257).all())


def _i64(v):
    return ctypes.c_longlong(v)


def status(lib, rc):
    """None, or what was wrong with a call."""
    return None if rc == 0 else f"{rc}: {lib.emu_text().decode()}"


def layer(lib, fmt, xq, sx, experts, weights, w1, s1, w2, s2, base=None, packed=(False, False),
          pack=None, descending=False, at_end=True, pad=16, short=None):
    """(y's bf16 bits [T, D], what was wrong or None) of one call; codes in rows
    `pad` bytes apart, the workspace NaN behind its counters."""
    T, D = xq.shape
    E, _, I = w2.shape
    topk = experts.shape[1]
    b = Buffers(lib, at_end, short)

    def codes(name, w, is_packed):
        if is_packed:
            one = np.stack([pack(fmt, e) for e in w])
            return b.put(name, one), 0, one[0].nbytes
        E, N, K = w.shape
        return b.rows(name, w.reshape(E * N, K), K + pad), K + pad, N * (K + pad)

    xp = b.rows("xq", xq, D + pad)
    w1p, ld1, st1 = codes("w1", w1, packed[0])
    w2p, ld2, st2 = codes("w2", w2, packed[1])
    args = [int(descending), FMT[fmt], E, T, topk, D, I, xp, _i64(D + pad), b.put("sx", sx),
            b.put("experts", experts.astype(np.int32)), b.put("weights", weights),
            w1p, _i64(ld1), _i64(st1), b.put("s1", s1), _i64(s1.size // E),
            w2p, _i64(ld2), _i64(st2), b.put("s2", s2), _i64(s2.size // E)]
    args += [None, _i64(0)] if base is None else [b.rows("base", base, D + 3), _i64(D + 3)]
    ldy = D + 5
    y = b.rows("y", np.full((T, D), GUARD * 257, np.uint16), ldy)
    need = lib.emu_layer_workspace(T, topk, D, I)
    counters = lib.emu_layer_workspace(1, 1, 16, 16) - 4 * 256  # (four arrays of a line or two)
    room = np.full(need, 255, np.uint8)
    room[:counters] = 0
    args += [y, _i64(ldy), b.put("workspace", room), _i64(need)]
    wrong = status(lib, lib.emu_layer(*args))
    got, untouched = b.get_rows("y", T, D, ldy)
    if wrong is None and not untouched:
        wrong = "a store between the output's rows"
    if wrong is None and b.get("workspace", np.uint8, counters).any():
        wrong = "counters that are not zero"
    return got, wrong


def pack(fmt, w):
    """One expert's codes [N, K] in the packed layout, zeros past its ends: fragments of
    16 rows by a K-step in the order the lanes of an MFMA take them."""
    step = 64 if fmt == "W8A8_INT8" else 128
    N, K = w.shape
    p = np.zeros((-(-N // 16) * 16, -(-K // step) * step), dtype=np.uint8)
    p[:N, :K] = w
    # [block, row, step, half, quarter of 16 bytes]: lane = 16 quarter + row
    v = p.reshape(len(p) // 16, 16, p.shape[1] // step, step // 64, 4, 16)
    return np.ascontiguousarray(v.transpose(0, 2, 3, 4, 1, 5)).reshape(-1)


def route(lib, logits, topk, renormalize=True, scale=1.0, lists=True, ld=None, descending=False,
          at_end=True):
    """((experts, weights, offsets, rows, slots), what was wrong or None); logits fp32 or
    bf16 bits (uint16) [T, E], rows `ld` elements apart."""
    T, E = logits.shape
    ld = ld or E
    b = Buffers(lib, at_end)
    lp = b.rows("logits", logits, ld)
    i32 = lambda name, n: b.put(name, np.full(n, -77, np.int32))
    out = [i32("experts", T * topk), i32("weights", T * topk)]
    out += [i32("offsets", E + 1), i32("rows", T * topk), i32("slots", T * topk)] if lists else [None] * 3
    need = lib.emu_route_workspace(T, E, topk) if lists else 0
    counters = lib.emu_layer_workspace(1, 1, 16, 16) - 4 * 256
    room = np.full(need, 255, np.uint8)
    room[:counters] = 0
    wrong = status(lib, lib.emu_route(
        int(descending), T, E, topk, lp, _i64(ld), int(logits.dtype == np.float32), int(renormalize),
        ctypes.c_float(scale), *out, b.put("workspace", room) if need else None, _i64(need)))
    got = [b.get("experts", np.int32, T * topk).reshape(T, topk),
           b.get("weights", np.float32, T * topk).reshape(T, topk)]
    if lists:
        got += [b.get("offsets", np.int32, E + 1), b.get("rows", np.int32, T * topk),
                b.get("slots", np.int32, T * topk).reshape(T, topk)]
    return got, wrong


def combine(lib, y, weights, slots, base=None, in_place=False, descending=False, at_end=True):
    """(bf16 bits [T, D], what was wrong or None); y and base bf16 bits."""
    T, topk = slots.shape
    D = y.shape[1]
    b = Buffers(lib, at_end)
    args = [int(descending), T, topk, D, b.rows("y", y, D + 1) if len(y) else None, _i64(D + 1),
            len(y), b.put("weights", weights), b.put("slots", slots.astype(np.int32))]
    args += [None, _i64(0)] if base is None else [b.rows("base", base, D + 3), _i64(D + 3)]
    if in_place:
        out, ldo = b.of["base"], D + 3
        b.of["out"] = out
    else:
        ldo = D + 2
        out = b.rows("out", np.zeros((T, D), np.uint16), ldo)
    wrong = status(lib, lib.emu_combine(*args, out, _i64(ldo)))
    got, untouched = b.get_rows("out", T, D, ldo)
    return got, wrong if wrong or untouched else "a store between the output's rows"


def quantize(lib, fmt, x, gate=None, reciprocal=False, descending=False, at_end=True):
    """(codes [M, K], scales [M], what was wrong or None) of bf16 bits."""
    M, K = x.shape
    b = Buffers(lib, at_end)
    ld = K + 8
    args = [int(descending), FMT[fmt], M, K, b.rows("x", x, ld), _i64(ld)]
    args += [None, _i64(0)] if gate is None else [b.rows("gate", gate, ld), _i64(ld)]
    args += [int(reciprocal), b.rows("xq", np.zeros((M, K), np.uint8), ld), _i64(ld),
             b.put("sx", np.zeros(M, np.float32))]
    wrong = status(lib, lib.emu_quantize(*args))
    flat = np.concatenate([b.get("xq", np.uint8, (M - 1) * ld + K), np.full(8, GUARD, np.uint8)])
    rows = flat.reshape(M, ld)
    if wrong is None and (rows[:, K:] != GUARD).any():
        wrong = "a store between the codes' rows"
    return rows[:, :K], b.get("sx", np.float32, M), wrong
