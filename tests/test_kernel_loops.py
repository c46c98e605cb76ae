"""Every loop of the kernels has an end in its head, or says above it how often it goes round at most: none
goes on until data that another stream may have changed in between lets it stop."""
import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "paged_kv_cache_39_gb300" / "csrc"
ENDLESS = re.compile(r"\bfor\s*\([^;()]*(?:\([^()]*\)[^;()]*)*;\s*;|\bwhile\s*\(\s*(?:true|1)\s*\)")


def endless(text):
    """Numbers of the lines with such a loop that have no "at most" in the comment right above."""
    out, above = [], ""
    for number, line in enumerate(text.splitlines(), 1):
        code, _, comment = line.partition("//")
        if ENDLESS.search(code) and "at most" not in above:
            out.append(number)
        above = "" if code.strip() else above + comment
    return out


@pytest.mark.parametrize("path", sorted(CSRC.glob("*.cu*")), ids=lambda p: p.name)
def test_loops_have_a_condition(path):
    assert endless(path.read_text()) == []


@pytest.mark.parametrize("text,found", [
    ("for (int i = from + lane;; i += 32) {", True), ("for (;;)", True), ("while (true) {", True), ("while ( 1 )", True),
    ("for (int i = min(a, b); ; ++i)", True), ("for (int hi = 7; x < hi;) {", False), ("while (x > 1)", False),
    ("// at most 3\n// times\nwhile (true)", False), ("// at most 3\nx = 1;\nwhile (true)", True),
    ("for (int i = f(a); i < n; ++i) g();", False),
])
def test_the_pattern(text, found):
    assert bool(endless(text)) == found
