"""Source check of the tensor-core kernels (no GPU needed): registers that a TMEM load fills are named by the wait after it.

A tcgen05.ld returns before its registers are written.  The wait for it is a statement of its own, and arithmetic on the
registers is an ordinary expression, which the compiler may place before any statement that does not mention them: a wait that
clobbers memory alone orders nothing.  Whether a build shows it depends on instruction scheduling, so the sources are
checked instead of a result."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "structured_sparse_long_gb300", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))
LOAD = re.compile(r"\btmem_ld\d+\((.*)\)$", re.S)
WAIT = re.compile(r"\btmem_wait_ld\w*\((.*)\)$", re.S)


def statements(text):
    """The statements of a source without comments, in order."""
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    text = re.sub(r"//[^\n]*", " ", text)
    return [s.strip() for s in re.split(r"[;{}]", text)]


def arguments(text):
    """A call's arguments, split at the commas outside parentheses."""
    out, depth = [""], 0
    for c in text:
        depth += (c == "(") - (c == ")")
        if c == "," and depth == 0:
            out.append("")
        else:
            out[-1] += c
    return [x.strip() for x in out]


def unnamed(text):
    """Statements at which registers of an earlier load are in flight, and that are neither another load nor the wait that names
    them all."""
    found, pending = [], set()
    for s in statements(text):
        if "__device__" in s:  # the building blocks' own definitions
            continue
        load, wait = LOAD.search(s), WAIT.search(s)
        if load:
            pending.add(arguments(load.group(1))[1].split("+")[0].strip())
        elif wait:
            if {a.split("+")[0].strip() for a in arguments(wait.group(1))} != pending:
                found.append(s)
            pending = set()
        elif pending:
            found.append(s)
            pending = set()
    return found


def test_the_check_sees_what_it_looks_for():
    good = "tmem_ld32(a + 1, x); tmem_ld16(b, y); tmem_wait_ld(x, y); f(x[0]);"
    assert not unnamed(good)
    for bad in (good.replace("(x, y)", "()"), good.replace("(x, y)", "(x)"), good.replace("tmem_wait_ld(x, y); ", ""),
                good.replace("tmem_wait_ld(x, y); f(x[0]);", "f(x[0]); tmem_wait_ld(x, y);")):
        assert unnamed(bad)


@pytest.mark.parametrize("name", SOURCES)
def test_waits_name_the_registers_they_wait_for(name):
    with open(os.path.join(CSRC, name)) as fh:
        assert unnamed(fh.read()) == []
