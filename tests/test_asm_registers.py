"""Inline assembly names what it overwrites: a statement that sets m0 without saying so leaves the compiler free to expect a
value of its own there afterwards."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "all_reduce_reduction_ring_amd", "csrc")
SETS = re.compile(r"\b(?:s|v)_(?!store|cmp)\w+\s+(m0|vcc(?:_lo|_hi)?|exec(?:_lo|_hi)?)\b")


def statements(text):
    """(instructions, clobbers) of every asm statement."""
    for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if c == '"' and text[at - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            at += 1
        body = text[m.end():at - 1]
        first = re.match(r'\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', body).group(1)
        parts = re.split(r":(?=(?:[^\"]*\"[^\"]*\")*[^\"]*$)", body[len(first):].replace("::", ": :"))
        yield first, parts[3] if len(parts) > 3 else ""


def undeclared(text):
    return [(code, reg) for code, clobbers in statements(text) for reg in SETS.findall(code) if f'"{reg}"' not in clobbers]


@pytest.mark.parametrize("name", sorted(n for n in os.listdir(CSRC) if n.endswith((".hip", ".h"))))
def test_every_statement_names_the_registers_it_sets(name):
    assert undeclared(open(os.path.join(CSRC, name)).read()) == []


def test_the_scan_itself():
    assert undeclared('asm volatile("s_mov_b32 m0, %0\\n\\ts_nop 4" ::"s"(f(x)) : "memory");') == [
        ('"s_mov_b32 m0, %0\\n\\ts_nop 4" ', "m0")]
    assert undeclared('asm volatile("s_mov_b32 m0, %0" ::"s"(x) : "memory", "m0");') == []
    assert undeclared('asm("s_mov_b64 vcc, %1" : "=s"(y) : "s"(x) : "vcc");') == []
    assert undeclared('asm("s_mov_b32 %0, m0" : "=s"(y));') == []
    found = [c for n in os.listdir(CSRC) if n.endswith(".hip") for c, _ in statements(open(os.path.join(CSRC, n)).read())]
    assert any("m0" in c for c in found)  # the loads into LDS are seen
