"""Inline assembly in the kernels: registers that the compiler reserves are left as they were."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rank_adapter_gemm_build_amd", "csrc")


def statements():
    """(file, instructions) of every asm statement."""
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        for m in re.finditer(r'\basm\s*(?:volatile)?\s*\(\s*((?:"(?:[^"\\]|\\.)*"\s*)+)', text):
            body = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(1)))
            yield name, [line.strip() for line in body.replace("\\t", " ").split("\\n")]


def test_m0_is_put_back():
    """A clobber of m0 is not honoured, so code that writes it saves it first and restores it last."""
    writes = [(name, lines) for name, lines in statements() if any(re.match(r"\w+ m0\b", line) for line in lines)]
    assert writes
    for name, lines in writes:
        kept = re.fullmatch(r"s_mov_b32 (%\d+), m0", lines[0])
        assert kept and lines[-1] == f"s_mov_b32 m0, {kept.group(1)}", (name, lines)
