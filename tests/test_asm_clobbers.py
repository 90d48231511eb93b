"""Inline assembly of the kernels says which fixed registers it writes (no GPU needed): the compiler keeps values in any
register that a statement does not name, m0 among them."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "shared_routed_expert_amd", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.hpp"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            yield os.path.basename(path), text[m.end():i - 1]


def test_fixed_registers_are_declared():
    """What a statement writes stands in its clobbers; a load to LDS, which reads m0, has it written by the statement or
    bound as an operand."""
    seen = 0
    for name, body in statements():
        seen += 1
        code = body.split(":")[0]
        operands = body[len(code):]
        written = set(re.findall(r"\b[sv]_\w+\s+(m0|vcc|exec|scc|[sv]\d+)\b", code))
        for reg in written:
            assert f'"{reg}"' in operands, f"{name}: {reg} is written and not listed:\n{body}"
        if "_load_lds_" in code:
            assert "m0" in written or '"{m0}"' in operands, f"{name}: m0 is read and not bound:\n{body}"
    assert seen
