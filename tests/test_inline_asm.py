"""Inline assembly names the special registers that it writes: the compiler
would otherwise take them for unchanged."""
import glob
import os
import re

import pytest

PKG = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "microscaling_quantized_convolution_mx_amd")
SOURCES = sorted(glob.glob(os.path.join(PKG, "csrc*", "*")))


def statements(text):
    """The asm statements without comments, each with its strings joined as they stand."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"\basm\b(?:\s+volatile)?\s*\((?:[^;\"]|\"(?:[^\"\\]|\\.)*\")*\)\s*;", text)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_registers_that_assembly_writes_are_clobbers(path):
    with open(path) as f:
        for s in statements(f.read()):
            for reg in ("m0", "vcc", "exec"):
                if re.search(rf"\b[sv]_\w+ {reg}\b", s):
                    assert f'"{reg}"' in s, s


def test_the_check_sees_a_missing_clobber():
    bad = 'asm volatile("s_mov_b32 m0, %0\\n\\tglobal_x %1" : : "s"(d), "v"(o) : "memory");'
    assert statements("int x;\n" + bad) == [bad]
    assert statements("// " + bad) == []
    with open(os.path.join(PKG, "csrc_linear", "linear_gemm.hip")) as f:
        assert sum("m0" in s for s in statements(f.read())) == 2
