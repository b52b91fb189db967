"""Inline assembly of the loss operators' kernels: no register is written or read behind
the compiler's back."""
import os
import re

from zero_sharded_optimizer_amd import build_lib


def test_registers_are_known_to_the_compiler():
    """A block writes no register by name unless its clobbers say so, and a load into LDS
    has its address in M0 as an operand."""
    with open(os.path.join(build_lib.CSRC, "zero_loss.hip")) as f:
        source = f.read()
    blocks = re.findall(r"asm\s+volatile\s*\((.*?)\);", source, re.S)
    assert len(blocks) >= 4
    loads = 0
    for block in blocks:
        code, *lists = re.split(r"\n\s*:|\s:\s", block)
        written = set(re.findall(r"\bs_\w+ (m0|vcc\w*|exec\w*|s\d+)\b", code))
        named = set(re.findall(r'"(\w+)"', lists[-1])) if len(lists) >= 3 else set()
        assert written <= named, f"{written - named} written behind the compiler's back: {block}"
        if "load_lds" in code:
            loads += 1
            assert '"{m0}"' in lists[1], f"M0 is read behind the compiler's back: {block}"
    assert loads == 1
