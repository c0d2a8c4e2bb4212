"""What the kernels' inline PTX has to say for the compiler to leave it in place."""
import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "mxfp4_block_quantization_gb300", "csrc", "*.cu*")))


def statements():
    """(file, line, whether volatile, text) of every asm statement."""
    for path in SOURCES:
        text = open(path).read()
        for m in re.finditer(r"\basm\s*(volatile)?\s*\(", text):
            depth, at, quoted = 1, m.end(), False
            while depth:
                c = text[at]
                if c == '"' and text[at - 1] != "\\":
                    quoted = not quoted
                elif not quoted:
                    depth += (c == "(") - (c == ")")
                at += 1
            yield os.path.basename(path), text[:m.start()].count("\n") + 1, bool(m.group(1)), text[m.end():at - 1]


def test_the_statements_are_found():
    found = list(statements())
    assert len(found) > 50 and any("tcgen05.mma" in s[3] for s in found)


@pytest.mark.parametrize("name", ["redux.sync", "shfl.sync", "vote.sync", "match.", "elect.sync", "activemask", "bar.", "barrier."])
def test_what_all_lanes_take_part_in_is_volatile(name):
    """Else a result that only some lanes use may be computed by those lanes alone."""
    bad = [s[:2] for s in statements() if name in s[3] and not s[2]]
    assert not bad, bad


def test_loads_from_tensor_memory_wait_for_their_words():
    """tcgen05.ld names its registers at once and fills them later: only a wait in the
    same statement keeps what uses them behind it."""
    loads = [s for s in statements() if "tcgen05.ld" in s[3]]
    assert loads
    bad = [s[:2] for s in loads if "tcgen05.wait::ld" not in s[3]]
    assert not bad, bad
