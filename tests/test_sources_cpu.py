"""Checks of the kernels' source text that need no GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_compressed_adaptive_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.h*")))


def _asm(text):
    """(instructions, operands and clobbers) of every asm statement."""
    for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\)\s*;", text, re.S):
        body = m.group(1)
        strings = re.match(r'\s*(?:"(?:[^"\\]|\\.)*"\s*)+', body).group(0)
        yield strings, body[len(strings):]


def test_the_sources_are_found():
    found = [a for p in SOURCES for a in _asm(open(p).read())]
    assert any("buffer_load" in a for a, _ in found) and any("s_barrier" in a for a, _ in found)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_asm_names_the_fixed_registers_it_uses(path):
    """An instruction in asm that reads or writes m0, vcc or exec says so to the
    compiler (buffer loads to LDS read m0)."""
    for text, operands in _asm(open(path).read()):
        used = {r for r in ("m0", "vcc", "exec") if re.search(rf"\b{r}(_lo|_hi)?\b", text)}
        if re.search(r"\blds\b", text):
            used.add("m0")
        for r in used:
            assert re.search(rf'"(=|\+)?\{{?{r}\}}?"', operands), (os.path.basename(path), text)
