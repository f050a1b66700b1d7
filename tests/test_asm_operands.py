"""Inline assembly and m0, the register that loads to LDS take their LDS address from: a statement gets
it as an operand.  One that wrote it by itself would change it behind the compiler's back."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "expert_cache_offload_amd", "csrc")


def _statements(text):
    """The bodies of the asm statements of a source."""
    for at in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        depth, quoted, i = 1, False, at.end()
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[at.end():i - 1]


def test_m0_is_an_operand():
    loads = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        with open(path) as f:
            for body in _statements(f.read()):
                assert not re.search(r"\bm0\s*,", body), (path, body)
                if re.search(r"_load_lds_", body):
                    loads += 1
                    assert '"{m0}"(' in body, (path, body)
    assert loads >= 2
