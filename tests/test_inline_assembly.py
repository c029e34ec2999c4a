"""Inline assembly of the kernels' sources tells the compiler every register that it writes by name."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zero_order_recurrent_amd", "csrc")
NAMED = re.compile(r"\b(m0|vcc|exec|scc|s\d+|v\d+|a\d+)\b")


def blocks(text):
    """Each asm statement as (instructions, clobbers)."""
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        depth, i = 1, m.end()
        quoted = False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        body = text[m.end():i - 1]
        parts, quoted, start = [], False, 0
        for j, c in enumerate(body):
            if c == '"':
                quoted = not quoted
            elif c == ":" and not quoted:
                parts.append(body[start:j])
                start = j + 1
        parts.append(body[start:])
        yield "".join(re.findall(r'"([^"]*)"', parts[0])), re.findall(r'"([^"]*)"', parts[3]) if len(parts) > 3 else []


def test_written_registers_are_clobbers():
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        for code, clobbers in blocks(open(path).read()):
            for line in re.split(r"\\n|;", code):
                words = line.replace("\\t", " ").split(None, 1)
                if len(words) < 2:
                    continue
                found += 1
                first = words[1].split(",")[0].strip()
                if NAMED.fullmatch(first):
                    assert first in clobbers, f"{os.path.basename(path)}: {line.strip()} writes {first}"
    assert found
