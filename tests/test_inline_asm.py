"""Inline assembly of the kernels tells the compiler of the registers it uses (no GPU)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STATEMENT = re.compile(r"\basm\s+(?:volatile\s*)?\((.*?)\)\s*;", re.S)
TEXT = re.compile(r'"((?:[^"\\]|\\.)*)"')


def test_m0_is_the_compilers():
    """m0 cannot be named as clobbered, so no statement writes it; one that loads to LDS, whose address is in m0, takes it
    as an operand."""
    found = 0
    for path in sorted(glob.glob(os.path.join(ROOT, "tile_binned_gaussian_amd", "csrc", "**", "*.h*"), recursive=True)):
        with open(path) as f:
            source = f.read()
        for statement in STATEMENT.findall(source):
            code = "".join(TEXT.findall(statement.split(":")[0])).replace("\\n", "\n").replace("\\t", " ")
            assert not re.search(r"\b[sv]_\w+\s+m0\b", code), f"{path}: {code}"
            if "_load_lds_" in code:
                found += 1
                assert '"{m0}"' in statement, f"{path}: {code}"
    assert found >= 1
