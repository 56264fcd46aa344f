"""GPU: the context operators at their edges: non-finite tokens, weights far
apart, steps built on one stream and run on another, ranges of every kind.
Bounds as derived in tests/context_cases.py."""
import numpy as np
import pytest
import torch

from paged_kv_gqa_block_amd import engine
from tests.context_cases import Batch
from tests.parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def _step(b, splits=None):
    cls = engine.Kv4Step if b.kv4 else engine.WindowStep
    return cls(b.problem(), b.window, b.sinks, splits)


def _same(a, b):
    view = {2: torch.int16, 4: torch.int32, 1: torch.uint8}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_seen_token_stays_in_its_row(value, kv4, dtype):
    """A NaN or an infinity in K of a token that queries see: those queries give what
    the formula gives, and every other row keeps its bits."""
    lens, new, row, tok = [300, 200, 90, 64], [40, 70, 90, 3], 1, 150
    for many in (False, True):
        say(f"[non-finite] {value} kv4={kv4} {dtype} prompt={many}")
        b = Batch(41, lens, new if many else None, hkv=2, group=4, dtype=dtype, kv4=kv4)
        w = b.device()
        step = engine.PromptStep(b.problem(), int(b.new.sum())) if many else _step(b)
        out, lse = (t.clone() for t in step.run(w))
        page = int(b.table[row, tok // 16])
        if kv4:
            w["kv4_pool"][page, :, 16 * 128 + (tok % 16) * 4] = 255  # a block that held it
        else:
            w["k_pool"][page, :, tok % 16, 3] = value
        bad_out, bad_lse = step.run(w)
        torch.cuda.synchronize()
        at = np.concatenate([[0], np.cumsum(b.new)])
        for r in range(4):
            span = slice(int(at[r]), int(at[r + 1]))
            if r != row:
                assert _same(out[span], bad_out[span]) and _same(lse[span], bad_lse[span]), r
        first = int(at[row]) + max(0, tok - (lens[row] - int(b.new[row])))
        hit = bad_out[first:int(at[row + 1])]
        q = w["q"][first:int(at[row + 1])]
        # A score of +inf makes its query's weights NaN, one of -inf weighs nothing.
        want = torch.ones_like(q[..., 3], dtype=torch.bool) if kv4 or value != value \
            else q[..., 3].float() * value > 0
        assert torch.equal(torch.isnan(hit).all(-1), want)
        assert torch.equal(torch.isfinite(hit).all(-1), ~want)
