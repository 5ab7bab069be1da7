"""Assembly in the kernels' sources says what it changes: a register that an
instruction writes by name is among the statement's clobbers, or the compiler
may keep something of its own there."""
import glob
import os
import re

from moe_token_re_amd import build


def statements():
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.hip")) + glob.glob(os.path.join(build.CSRC, "*.h"))):
        for found in re.finditer(r"\basm\s+volatile\s*\((.*?)\)\s*;", open(path).read(), flags=re.S):
            yield os.path.basename(path), found[1]


def test_named_registers_are_clobbers():
    seen = 0
    for path, text in statements():
        code = re.match(r"(\s*\"(?:[^\"\\]|\\.)*\")+", text)[0]
        clobbers = re.findall(r"\"(\w+)\"", text.rsplit(":", 1)[1]) if ":" in text[len(code):] else []
        for written in re.findall(r"(?:^|\\n\\t|\")\s*[sv]_\w+\s+(m0|vcc|exec|s\d+|v\d+)\s*,", code):
            seen += 1
            assert written in clobbers, f"{path}: {text.strip()} writes {written}"
    assert seen > 0
