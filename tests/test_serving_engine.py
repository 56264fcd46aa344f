"""CPU: what the serving operators' classes refuse without a GPU, and rules of their
sources that no run shows reliably."""
import glob
import os
import re

import pytest
import torch

from paged_kv_gqa_block_amd import _lib, engine

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_gqa_block_amd", "csrc")


@pytest.mark.skipif(not hasattr(_lib.LIB, "pkv_attend_kv8"),
                    reason="this build holds other host code only")
def test_buffers_in_host_memory_are_refused():
    prob = engine.make_problem(2, 8, 2, 128, 16, 8, 4, "f16")
    pool = torch.zeros(8, 2, 32 * 128, dtype=torch.uint8)
    scales = torch.zeros(8, 2, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        engine.Kv8Cache(prob, pool=pool, scales=scales)
    with pytest.raises(ValueError, match="together"):
        engine.Kv8Cache(prob, pool=pool)
    with pytest.raises(ValueError, match="together"):
        engine.Kv8Cache(prob, scales=scales)
    with pytest.raises(ValueError, match="GPU"):
        engine.Kv8Cache(prob, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        engine.Kv8Step(prob, splits=1, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        engine.CrossStep(prob, 4, splits=1, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        engine.PageTable(prob, 4, device="cpu")


def test_inline_asm_holds_waits_only():
    """As in the context kernels: the compiler puts no wait between a matrix product
    and inline asm that reads its result."""
    paths = sorted(glob.glob(os.path.join(CSRC, "serving", "*")))
    assert paths
    for path in paths:
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(\s*((?:\"(?:[^\"\\]|\\.)*\"\s*)+)", text):
            code = "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", m.group(1)))
            assert not code or re.fullmatch(r"s_waitcnt \w+\(\d+\)", code), (path, code)
