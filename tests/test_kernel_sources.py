"""Rules of the kernel sources that a run cannot show.  No GPU needed."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "birkhoff_projection_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h")))


def asm_statements(text):
    """The text of every asm statement, parentheses matched."""
    out = []
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            ch = text[i]
            if ch == "\\" and quoted:
                i += 1
            elif ch == '"':
                quoted = not quoted
            elif not quoted:
                depth += {"(": 1, ")": -1}.get(ch, 0)
            i += 1
        out.append(text[m.start():i])
    return out


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_assembly_names_the_m0_it_writes(path):
    """m0 is the compiler's too: an asm statement that writes it says so."""
    with open(path, encoding="utf-8") as f:
        for a in asm_statements(f.read()):
            if re.search(r"s_mov_b32\s+m0\b", a):
                assert '"m0"' in a.rsplit(":", 1)[-1], a


def test_the_copies_to_lds_are_found():
    """The rule above looks at something."""
    text = "".join(open(p, encoding="utf-8").read() for p in SOURCES)
    assert sum("s_mov_b32 m0" in a for a in asm_statements(text)) == 2
