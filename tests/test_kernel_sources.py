"""What the compiler has to be told about inline assembly, checked in the source text."""
import glob
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def statements(text):
    """The argument lists of the asm statements."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.end():i - 1]


def test_assembly_that_writes_m0_declares_it():
    found = 0
    for path in glob.glob(os.path.join(ROOT, "message_allreduce_amd", "csrc", "*")) + \
            glob.glob(os.path.join(ROOT, "include", "*")):
        with open(path) as f:
            for s in statements(f.read()):
                if re.search(r"\bs_\w+ m0\b", s):
                    found += 1
                    # the last colon outside the strings starts the clobbers
                    clobbers = re.sub(r'"[^"]*"', lambda q: q.group().replace(":", " "), s).rsplit(":", 1)[1]
                    assert '"m0"' in clobbers, (os.path.basename(path), s)
    assert found
