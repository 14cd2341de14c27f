"""Inline assembly in the kernels: a register that its text names is among its
clobbers, so the compiler keeps nothing there."""
import glob
import os
import re

from zero_partitioned_mixed_flatten_amd import build

FIXED = r"\b(m0|vcc|exec|scc|s\d+|v\d+|a\d+|s\[\d+:\d+\]|v\[\d+:\d+\]|a\[\d+:\d+\])"


def _statements(text):
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1]


def test_named_registers_are_clobbered():
    seen = 0
    for path in glob.glob(os.path.join(build.CSRC, "*.h*")):
        for body in _statements(open(path).read()):
            template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body.split(" :")[0]))
            clobbers = set(re.findall(r'"([^"]*)"', body.rsplit(":", 1)[1])) if body.count(":") >= 3 else set()
            for name in set(re.findall(FIXED, template.replace("\\n", " ").replace("\\t", " "))):
                seen += 1
                assert name in clobbers, (os.path.basename(path), body)
    assert seen                                            # m0 of the loads straight into LDS
