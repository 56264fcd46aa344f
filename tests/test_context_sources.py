"""CPU: rules of the context kernels' sources that no run shows reliably."""
import glob
import os
import re

CONTEXT = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "paged_kv_gqa_block_amd", "csrc", "context")


def test_inline_asm_holds_waits_only():
    """The compiler puts no wait between a matrix product and inline asm that reads
    its result, so no instruction that takes a register stands in inline asm:
    only waits, and empty statements that order values."""
    found = []
    for path in sorted(glob.glob(os.path.join(CONTEXT, "*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(\s*((?:\"(?:[^\"\\]|\\.)*\"\s*)+)", text):
            code = "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))
            found.append((os.path.basename(path), code))
    assert found, "the pattern above matches the sources"
    bad = [x for x in found if x[1] and not re.fullmatch(r"s_waitcnt \w+\(\d+\)", x[1])]
    assert not bad, bad
