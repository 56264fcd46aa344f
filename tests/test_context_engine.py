"""CPU: what the context operators' classes refuse without a GPU."""
import pytest
import torch

from paged_kv_gqa_block_amd import _context, engine

pytestmark = pytest.mark.skipif(not hasattr(_context.LIB, "pkv_attend_kv4"),
                                reason="this build holds the decode engine's host code only")


def test_buffers_in_host_memory_are_refused():
    prob = engine.make_problem(2, 8, 2, 128, 16, 8, 4, "f16")
    pool = torch.zeros(8, 2, 17 * 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        engine.Kv4Cache(prob, pool=pool)
    with pytest.raises(ValueError, match="GPU"):
        engine.Kv4Cache(prob, device="cpu")
    for cls in (engine.WindowStep, engine.Kv4Step):
        with pytest.raises(ValueError, match="GPU"):
            cls(prob, splits=1, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        engine.PromptStep(prob, 4, splits=1, device="cpu")
    kv = torch.zeros(2, 2, 128, dtype=torch.float16)
    kp = torch.zeros(8, 2, 16, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        engine.store_kv(prob, kv, kv, torch.zeros(2, 4, dtype=torch.int32),
                        torch.ones(2, dtype=torch.int32), None, kp, kp.clone())
