"""Rules that the kernel sources keep."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hpc_linear_algebra_amd", "csrc")


def statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[i], 0)
                i += 1
            yield os.path.basename(path), text[m.end():i - 1]


def test_assembly_gets_m0_from_the_compiler():
    """m0 is reserved: a statement cannot declare that it writes it.  One that needs it takes an operand there."""
    found = 0
    for name, body in statements():
        template = re.search(r'"((?:[^"\\]|\\.)*)"', body)[1]
        assert not re.search(r"\bm0\b", template), (name, body)
        if re.search(r"\blds\b", template):
            found += 1
            assert '"{m0}"' in body, (name, body)
    assert found
