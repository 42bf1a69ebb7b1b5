"""Inline assembly that the compiler must leave where it is written."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "precision_moe_numerics_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def statements(text):
    """(line, qualifiers, body) of each asm statement: its parentheses, strings aside, closed"""
    for m in re.finditer(r"\basm\b([^;(\"]*)\(", text):
        depth, i = 1, m.end()
        while depth:
            if text[i] == '"':
                i = re.compile(r'(?:[^"\\]|\\.)*"').match(text, i + 1).end()
                continue
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text.count("\n", 0, m.start()) + 1, m.group(1), text[m.end():i]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_instructions_that_lanes_execute_together_are_volatile(path):
    """An asm that is not volatile may move to where its result is used, into a branch too; an instruction that
    names all lanes of a warp (.sync, .aligned) then waits for lanes that never come."""
    with open(path) as f:
        found = list(statements(f.read()))
    moved = [line for line, how, body in found if re.search(r"\.(sync|aligned)\b", body) and "volatile" not in how]
    assert not moved, moved


def test_statements_are_found():
    text = 'asm("a.sync %0; (" : "=r"(x) : "r"(f(y)));\nasm volatile("b\\";" ::: "memory");'
    assert [(n, "volatile" in q) for n, q, _ in statements(text)] == [(1, False), (2, True)]
    assert sum(len(list(statements(open(p).read()))) for p in SOURCES) > 100
