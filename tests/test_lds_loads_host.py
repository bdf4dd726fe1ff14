"""Loads that go straight into LDS take their address from m0.  Between a
scalar write of m0 and such a load gfx950 needs a wait state, which nobody
inserts inside a block of inline assembly: every block carries its own."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gram_newton_schulz_amd", "csrc")
BLOCKS = []
for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
    with open(path) as f:
        text = f.read()
    for found in re.finditer(r'asm(?:\s+volatile)?\s*\(((?:\s*"(?:[^"\\]|\\.)*")+)', text):
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', found.group(1)))
        lines = [line.strip() for line in re.split(r"\\n|;", code.replace("\\t", " ")) if line.strip()]
        where = f"{os.path.basename(path)}:{text.count(chr(10), 0, found.start()) + 1}"
        BLOCKS.append((where, lines))
LOADS = [(where, lines) for where, lines in BLOCKS if any(re.search(r"\blds\b", line) for line in lines)]


def test_there_are_such_loads():
    assert len(LOADS) == 5


@pytest.mark.parametrize("where,lines", LOADS, ids=[where for where, _ in LOADS])
def test_wait_state_between_m0_and_the_load(where, lines):
    written = None
    for i, line in enumerate(lines):
        if re.match(r"s_\w+ m0,", line):
            written = i
        if re.search(r"\blds\b", line):
            assert written is not None, "m0 is set in the same block"
            assert i - written >= 2, lines
