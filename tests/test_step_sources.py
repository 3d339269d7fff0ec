"""Properties of the kernels' sources that no run can show."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "exact_replay_decode_amd", "csrc")
FILES = sorted(f for f in glob.glob(os.path.join(CSRC, "*")) if f.endswith((".hip", ".hpp")))


def asm_statements(text):
    """(instructions, clobbers) of every asm statement."""
    for m in re.finditer(r"\basm(?:\s+volatile)?\s*\(", text):
        depth, at, quoted, parts = 1, m.end(), False, [""]
        while depth:
            ch = text[at]
            if ch == '"':
                quoted = not quoted
            elif not quoted:
                depth += (ch == "(") - (ch == ")")
            if ch == ":" and not quoted and depth == 1:
                parts.append("")
            elif depth:
                parts[-1] += ch
            at += 1
        yield parts[0], parts[3] if len(parts) > 3 else ""


def test_the_statements_are_found():
    assert sum(len(list(asm_statements(open(f).read()))) for f in FILES) >= 5
    assert list(asm_statements('asm volatile("a: (%0" : "=v"(x) : : "memory", "m0");')) == [
        ('"a: (%0" ', ' "memory", "m0"')]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_registers_that_asm_writes_by_name_are_clobbered(path):
    """The compiler may keep m0, vcc, scc or exec of its own across a statement
    that does not say that it writes them."""
    for code, clobbers in asm_statements(open(path).read()):
        for reg in ("m0", "vcc", "exec"):
            if re.search(rf"\bs_\w+\s+{reg}\b|\bv_cmp\w*\s+{reg}\b", code):
                assert f'"{reg}"' in clobbers, (reg, code)
