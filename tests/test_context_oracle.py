"""The context operators' oracle, pinned on the CPU: attention with a view
against torch's masked attention and plain loops, the 4-bit block against
its definition by exhaustive search, the page layout as a bijection."""
import math

import numpy as np
import pytest
import torch

from oracle import context as oc
from tests.context_cases import Batch, f64


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 0), (5, 2), (64, 3), (3, 40), (16, 16)])
def test_view_attention_matches_torch_masked_attention(window, sinks):
    rng = np.random.default_rng(window * 100 + sinks)
    n, m, hkv, grp, d = 37, 9, 2, 3, 16
    q, k, v = (rng.standard_normal(s) for s in ((m, hkv * grp, d), (n, hkv, d), (n, hkv, d)))
    pos = range(n - m, n)
    out, lse, _ = oc.attend_row(q, pos, k, v, 0.3, window, sinks)
    mask = np.zeros((m, n), dtype=bool)
    for i, p in enumerate(pos):
        for t in range(n):  # the definition, one pair at a time
            mask[i, t] = t <= p and (window == 0 or t > p - window or t < sinks)
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1)[None] for x in (q, k, v))
    ref = torch.nn.functional.scaled_dot_product_attention(
        tq, tk, tv, attn_mask=torch.from_numpy(mask), scale=0.3, enable_gqa=True)
    np.testing.assert_allclose(out, ref[0].transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)
    for i in range(m):
        x = [0.3 * float(k[t, 1] @ q[i, 4]) for t in range(n) if mask[i, t]]
        assert lse[i, 4] == pytest.approx(math.log(sum(math.exp(y) for y in x)), abs=1e-12)


def test_a_query_that_sees_nothing():
    out, lse, (_, _, count) = oc.attend_row(np.ones((2, 1, 4)), [-2, -1], np.ones((3, 1, 4)),
                                            np.ones((3, 1, 4)), 1.0)
    assert not out.any() and np.isneginf(lse).all() and not count.any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantised_block_is_the_nearest_element(dtype):
    """Every element is a nearest multiple (ties to the even code), and no
    element is off by more than its block's scale."""
    rng = np.random.default_rng(3)
    t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    for spread in (1e-6, 1e-3, 1.0, 300.0):
        x = f64(torch.from_numpy(rng.standard_normal((40, 64), dtype=np.float32) * spread).to(t))
        codes, scales = oc.kv4_quantise(x, dtype)
        y = oc.kv4_values(codes, scales)
        unit = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, -1)
        assert (np.abs(y - x) <= unit).all()
        grid = np.array(oc.E2M1 + tuple(-e for e in oc.E2M1))
        best = np.abs(x[..., None] - grid * unit[..., None]).min(-1)
        np.testing.assert_array_equal(np.abs(y - x), best)
        back = torch.from_numpy(y).to(t).double().numpy()
        np.testing.assert_array_equal(back, y)  # exact in the 16-bit type


def test_hand_worked_block():
    x = np.zeros(32)
    x[:10] = [6.0, -6.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0]
    codes, scales = oc.kv4_quantise(x, "f16")  # top 6.5: exponent 0, ties to even
    assert scales.tolist() == [127]
    assert oc.kv4_values(codes, scales)[:10].tolist() == [6, -6, 0, 1, 1, 2, 2, 4, 4, -0.0]
    assert codes[9] == 8
    x[1] = -7.25  # over 7: the next scale, 2^1
    codes, scales = oc.kv4_quantise(x, "f16")
    assert scales.tolist() == [128]
    assert oc.kv4_values(codes, scales)[:4].tolist() == [6, -8, 0, 1]
    x[5] = np.inf
    assert oc.kv4_quantise(x, "f16")[1].tolist() == [255]
    assert oc.kv4_quantise(np.zeros(32), "bf16")[1].tolist() == [127 - 120]
    x[5] = 65504.0  # the next scale's 4 would be infinite in f16: saturates at 6 * 2^13
    codes, scales = oc.kv4_quantise(x, "f16")
    assert scales.tolist() == [140] and oc.kv4_values(codes, scales)[5] == 49152


@pytest.mark.parametrize("d", [64, 128])
def test_page_layout_is_a_bijection(d):
    k, v, ks, vs = oc.kv4_places(d)
    nibbles = list(k.values()) + list(v.values()) + [(b, n) for b in ks.values() for n in (0, 1)] + \
        [(b, n) for b in vs.values() for n in (0, 1)]
    assert len(nibbles) == len(set(nibbles)) == 2 * 17 * d
    assert min(nibbles) == (0, 0) and max(nibbles) == (17 * d - 1, 1)
    for places in (k, v):  # a byte belongs to one token
        owner = {}
        for (t, _), (b, _) in places.items():
            assert owner.setdefault(b, t) == t


@pytest.mark.parametrize("d", [64, 128])
def test_page_bytes_round_trip(d):
    rng = np.random.default_rng(d)
    page = rng.integers(0, 256, 17 * d).astype(np.uint8)
    before = {w: oc.kv4_read(page, w) for w in "kv"}
    codes, scales = rng.integers(0, 16, d), rng.integers(0, 255, d // 32)
    oc.kv4_write(page, 5, codes, scales, "v")
    for w in "kv":
        c, s = oc.kv4_read(page, w)
        for t in range(16):
            want = (codes, scales) if (w, t) == ("v", 5) else (before[w][0][t], before[w][1][t])
            np.testing.assert_array_equal(c[t], want[0])
            np.testing.assert_array_equal(s[t], want[1])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_batch_helper_matches_the_oracle(dtype):
    b = Batch(1, [20, 0, 17], dtype=dtype, kv4=True, d=64, window=6, sinks=2)
    x = np.random.default_rng(0).standard_normal((5, 64)) * np.array([[1e-7], [1e-3], [1], [50], [0]])
    x = f64(torch.from_numpy(x.astype(np.float32)).to({"f16": torch.float16,
                                                       "bf16": torch.bfloat16}[dtype]))
    for got, want in zip(b._quick(x), oc.kv4_quantise(x, dtype)):
        np.testing.assert_array_equal(got, want)
    for row, n in enumerate(b.lens):
        for tok in range(n):
            codes, scales = oc.kv4_read(b.pool4[b.table[row, tok // 16], 1], "v")
            val = oc.kv4_values(codes, scales)[tok % 16]
            if oc.sees(n - 1, tok, 6, 2):
                np.testing.assert_array_equal(val, b.kv[row][1][tok, 1])
            else:
                assert np.isnan(val).all()
