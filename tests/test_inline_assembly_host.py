"""Inline assembly of the kernels says what it changes."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def statements():
    """(file, text) of every asm statement under csrc."""
    for path in sorted(glob.glob(os.path.join(ROOT, "linear_algebra_amd", "csrc", "*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\s+volatile\s*\(", text):
            depth, end, quoted = 1, m.end(), False
            while depth:
                c = text[end]
                quoted ^= c == '"' and text[end - 1] != "\\"
                depth += 0 if quoted else (c == "(") - (c == ")")
                end += 1
            yield os.path.basename(path), text[m.end():end - 1]


def test_the_statements_are_found():
    assert len(list(statements())) > 20


def test_registers_that_are_written_are_named():
    """A statement that writes m0 or vcc names it among what it clobbers."""
    found = 0
    for name, text in statements():
        parts = re.split(r":(?=(?:[^\"]*\"[^\"]*\")*[^\"]*$)", text)
        code, clobbers = parts[0], parts[3] if len(parts) > 3 else ""
        for register in ("m0", "vcc"):
            if re.search(rf"\b[sv]_\w+\s+{register}\b", code):
                found += 1
                assert f'"{register}"' in clobbers, (name, text)
    assert found > 0
