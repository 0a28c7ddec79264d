"""Inline assembly of the kernels names every register that it writes by name."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "structured_sparse_gemm_amd", "csrc")


def _statements(text):
    """The asm statements of a source: (their text, whole statement)."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        whole = text[m.end():i - 1]
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', whole.split(":")[0])), whole


def _written(code):
    """Registers named as a destination in assembly text: scalar moves to m0, vcc, exec and numbered registers."""
    for line in re.split(r"\\n|\\t|;", code):
        m = re.match(r"\s*s_\w+\s+(m0|vcc|exec|s\d+|s\[\d+:\d+\])\s*,", line)
        if m:
            yield m.group(1)


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h"))),
                         ids=os.path.basename)
def test_named_registers_are_declared(path):
    for code, whole in _statements(open(path).read()):
        clobbers = whole.split(":")[-1]
        for reg in _written(code):
            assert f'"{reg}"' in clobbers, f"{reg} is written and not declared in: {whole}"


def test_the_scan_sees_a_write():
    found = list(_statements('asm volatile("s_mov_b32 m0, %0\\n\\tbuffer_load %1" :: "s"(a), "v"(b) : "memory");'))
    assert len(found) == 1 and list(_written(found[0][0])) == ["m0"]
