"""Registers that the kernels' inline assembly writes are named to the compiler."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_quantized_gemm_token_amd", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"asm volatile\((.*?)\);", text, re.S):
            yield os.path.basename(path), m.group(1)


def test_m0_is_named_where_it_is_written():
    writes = [(name, s) for name, s in statements() if re.search(r"s_mov_b32 m0\b", s)]
    assert writes
    for name, s in writes:
        assert s.rstrip().endswith(': "m0"'), f"{name}: {s}"
