"""Inline assembly names what it writes (CPU: reads the kernel sources)."""
from __future__ import annotations

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_kimi_delta_amd", "csrc")


def undeclared_m0(text: str):
    """asm statements that write M0 without naming it among their clobbers."""
    return [m.group(0) for m in re.finditer(r"\basm\b[^;]*?\((?:\"(?:\\.|[^\"\\])*\"|[^;\"])*\)\s*;", text)
            if re.search(r"s_mov\w*\s+m0\b", m.group(0)) and '"m0"' not in m.group(0)]


def test_detector_finds_an_undeclared_write():
    bad = 'asm volatile("s_mov_b32 m0, %0\\n\\tglobal_load_lds_dwordx4 %1, %2" :: "s"(a), "v"(o), "s"(b) : "memory");'
    assert len(undeclared_m0(bad)) == 1
    assert undeclared_m0(bad.replace('"memory")', '"memory", "m0")')) == []


def test_writes_of_m0_are_declared():
    sources = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip")))
    text = {os.path.basename(s): open(s).read() for s in sources}
    assert any("s_mov_b32 m0" in t for t in text.values())
    bad = {n: undeclared_m0(t) for n, t in text.items()}
    assert not any(bad.values()), bad
