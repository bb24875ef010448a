"""Loads from tensor memory and their waits, checked on the sources' text: a load's registers are valid only
behind tcgen05.wait::ld, and the compiler knows that only where the wait names them or stands in the load's
own statement."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prefix_shared_chunkwise_gb300", "csrc")
# Loads that are issued alone, for a later wait that names their registers.
ISSUE_ONLY = {"tmem_ld32_issue", "tmem_ld16_issue", "tld16", "tld8", "tld4"}
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def _statements(text):
    """The asm statements, from the keyword to the closing parenthesis."""
    for m in re.finditer(r"\basm\b(?: volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.start():i], re.findall(r"void (\w+)\(", text[:m.start()])[-1:]


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(p) for p in FILES])
def test_a_wait_names_the_registers_it_is_for(path):
    text = open(path).read()
    for s, function in _statements(text):
        load, wait = "tcgen05.ld." in s, "tcgen05.wait::ld" in s
        if load and not wait:
            assert function[0] in ISSUE_ONLY, function
        if wait and not load:
            assert '"+r"' in s or "HARTS_R" in s, s[:80]
