"""CPU: the oracle of the 8-bit cache, cross attention and page tables."""
import numpy as np
import pytest
import torch

from oracle import serving as sv
from oracle.context import attend_row
from tests.serving_cases import Batch8, cross_reference, make_cross


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(sv.E4M3, want)


def test_rounding_is_torchs_and_the_nearest():
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 9, 20000),
                        (sv.E4M3[:126] + sv.E4M3[1:127]) / 2, sv.E4M3[:127], [1e-300, 0.0]])
    y = np.concatenate([y, -y])
    y = y[np.abs(y) <= 448].astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = sv.e4m3_round(y)
    np.testing.assert_array_equal(got, want)
    near = np.abs(y.astype(np.float64)[:, None] - sv.E4M3[:127] * np.where(
        np.signbit(y), -1, 1)[:, None]).min(1)
    np.testing.assert_array_equal(np.abs(sv.E4M3[got] - y), near)
    assert (sv.e4m3_round([1e9, -1e9, np.inf, -np.inf, np.nan]) & 127).tolist() == [126, 126, 127,
                                                                                   127, 127]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_exponents(dtype):
    lo, hi = sv.EXP8[dtype]
    assert sv.exponent_for(0.0, dtype) == lo
    for e in range(lo, hi):
        assert sv.exponent_for(448 * 2.0 ** e, dtype) == e
        assert sv.exponent_for(np.nextafter(448 * 2.0 ** e, np.inf), dtype) == e + 1
    assert sv.exponent_for(1e300, dtype) == hi
    # Every value at the two ends is exact in the type.
    t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    for e in (lo, hi):
        x = torch.from_numpy(sv.E4M3[:127] * 2.0 ** e)
        assert torch.equal(x.to(t).double(), x)


@pytest.mark.parametrize("d", [64, 128])
def test_places_are_a_bijection(d):
    k, v = sv.kv8_places(d)
    assert sorted(np.concatenate([k.ravel(), v.ravel()])) == list(range(32 * d))


def test_errors_are_half_steps():
    """Off by at most 2^-4 of an element or 2^(e - 10): half a step of the codes."""
    rng = np.random.default_rng(1)
    for dtype, t in (("f16", torch.float16), ("bf16", torch.bfloat16)):
        x = rng.standard_normal((16, 2, 3, 64)) * 2.0 ** rng.integers(-14, 3, (16, 2, 3, 64))
        x = torch.from_numpy(x).to(t).double().numpy()
        c = sv.Cache8(1, 3, 64, dtype)
        c.store(0, 0, x)
        for s in range(16):
            y = c.values(0, s)
            e = c.scales[0].astype(int).T[..., None] - 127
            assert (np.abs(y - x[s]) <= np.maximum(2.0 ** -4 * np.abs(x[s]), 2.0 ** (e - 10.0))).all()


def test_growing_blocks_round_again():
    c = sv.Cache8(1, 1, 64, "f16")
    x = np.full((1, 2, 1, 64), 1.125)
    c.store(0, 0, x)
    assert c.scales[0, 0, 0] == 127 - 8 and c.values(0, 0)[0, 0, 0] == 1.125
    big = np.full((2, 2, 1, 64), 500.0)
    c.store(0, 1, big)
    assert c.scales[0, 0, 0] == 128 and c.values(0, 0)[0, 0, 0] == 1.125  # 0.5625: still exact
    c.store(0, 3, np.full((1, 2, 1, 64), 60000.0))
    assert c.scales[0, 0, 0] == 127 + 7 and c.values(0, 1)[0, 0, 0] == 512.0
    assert c.values(0, 0)[0, 0, 0] == 1.0  # 1.125 / 128 = 4.5 * 2^-9: a tie, to even: 4
    c.store(0, 3, np.full((1, 2, 1, 64), 0.5))
    assert c.scales[0, 0, 0] == 127 + 7  # does not shrink
    c.store(0, 0, np.full((1, 2, 1, 64), 0.5))
    assert c.scales[0, 0, 0] == 127 - 9  # starts anew


def test_cross_reference_is_torchs_attention():
    b = make_cross(16, 3, [33, 7, 0], [3, 0, 2], hkv=2, group=2, d=64)
    out, lse, _ = cross_reference(b)
    q = b.q[:3].double()
    k, v = (torch.from_numpy(x).repeat_interleave(2, 1) for x in b.kv[0])
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), scale=b.scale).transpose(0, 1)
    np.testing.assert_allclose(out[:3], want.numpy(), rtol=1e-12, atol=1e-12)
    assert (out[3:] == 0).all() and np.isneginf(lse[3:]).all()


def test_batch8_keeps_what_queries_see():
    b = Batch8(2, [40, 17], [1, 1], window=10, sinks=2, d=64)
    out, _, (_, _, count) = b.reference()
    assert count.tolist() == [12, 12] and np.isfinite(out).all()
    k, _ = b.kv[0]
    again = attend_row(np.asarray(b.q[:1].double()), [39], k, b.kv[0][1], b.scale, 10, 2)
    np.testing.assert_array_equal(again[0][0], out[0])


def test_pages_restore_and_never_double():
    rng = np.random.default_rng(4)
    width, pool, rows = 6, 20, 7
    p = sv.Pages([0] * rows, [[-1] * width] * rows, rng.permutation(pool), pool, width)
    for step in range(200):
        before = (list(p.lens), [list(r) for r in p.table], list(p.free))
        counts = rng.integers(-1, 40, rows) * (rng.random(rows) < 0.4)
        seq, off, slots, positions, denied = p.take(counts, 100)
        held = [p.table[r][e] for r in range(rows) for e in range(-(-p.lens[r] // 16))]
        assert sorted(held + p.free) == list(range(pool))
        good = [s for s in slots.values() if s >= 0]
        assert len(set(good)) == len(good)
        if step % 3 == 0:  # all of it back
            p.release(before[0])
            assert p.lens == before[0] and p.free == before[2]
        else:
            p.release([int(x) if x < 90 else -1 for x in rng.integers(0, 100, rows)])
    assert any(p.lens)


def test_a_row_short_of_pages_holds_up_those_behind_it():
    p = sv.Pages([16, 16, 16, 15], [[0, -1], [1, -1], [2, -1], [3, -1]], [9, 8], 10, 2)
    seq, off, slots, positions, denied = p.take([1, 0, 40, 1], 50)
    # Row 2 would pass the table: it asks for nothing; row 3 has room in its page.
    assert seq == [17, 16, 0, 16] and off == [0, 1, 1, 41, 42] and denied == 1
    p = sv.Pages([16] * 4, [[0, -1, -1], [1, -1, -1], [2, -1, -1], [3, -1, -1]], [9], 10, 3)
    seq, off, slots, positions, denied = p.take([17, 1, 0, 1], 50)
    assert seq == [0, 0, 16, 0] and denied == 3 and p.free == [9]


def test_rows_without_tokens_stay_as_long_as_they_are():
    """Behind a row whose tokens pass the arrays, before it, and under a table that is
    full: nothing of theirs lies outside."""
    p = sv.Pages([20, 33, 0, 64, 16], [[0, 1, -1, -1], [2, 3, 4, -1], [-1] * 4, [5, 6, 7, 8],
                                       [9, -1, -1, -1]], [10, 11], 12, 4)
    seq, off, slots, positions, denied = p.take([0, 9, 0, -3, 2], 8)
    assert seq == [20, 0, 0, 64, 0] and off == [0, 0, 8, 8, 8, 8] and denied == 2
    assert p.lens == [20, 33, 0, 64, 16] and p.free == [10, 11]
    assert set(slots.values()) == set(positions.values()) == {-1}


def test_entries_that_name_no_page_do_not_come_back():
    p = sv.Pages([64, 20], [[5, -1, 9, 7], [6, 2, -1, -1]], [1, 0], 8, 4)
    p.release([10, 0])
    assert p.free == [1, 0, 2, 6, 7] and p.table == [[5, -1, -1, -1], [-1] * 4]
    seq, _, slots, _, denied = p.take([0, 64], 64)
    assert denied == 0 and seq == [10, 64] and min(slots.values()) >= 0
    # Room for three: the last row's two, then one that is none.
    p = sv.Pages([48, 32], [[0, 1, 8, -1], [2, 3, -1, -1]], [4, 5, 6, 7, 4], 8, 4)
    p.release([0, 0])
    assert p.free == [4, 5, 6, 7, 4, 3, 2]


def test_errors_of_growing_blocks():
    """Off by at most 2^-4 of the element, or less than 2^(e - 9), at the block's last
    exponent, however often it has grown; 2^(e - 10) and no more where it has not."""
    def run(steps, dtype):
        """Values and elements of a block whose tokens come one after the other."""
        c = sv.Cache8(1, 1, 64, dtype)
        x = np.zeros((len(steps), 2, 1, 64))
        for t, z in enumerate(steps):
            x[t] = z
            c.store(0, t, x[t:t + 1])
        return np.stack([c.values(0, t) for t in range(len(steps))]), x, c.scales

    # 2.5 steps of a subnormal code: 2, then nothing; more than 2^(e - 10) in all.
    small = np.zeros(64)
    small[:2] = 448.0, 2.5 * 2.0 ** -9
    y, x, scales = run([small, 1792.0], "f16")
    assert scales[0, 0, 0] == 127 + 2 and y[0, 0, 0, 1] == 0.0
    assert 2.0 ** (2 - 10) < abs(y[0, 0, 0, 1] - x[0, 0, 0, 1]) < 2.0 ** (2 - 9)

    rng = np.random.default_rng(6)
    past = 0
    for trial in range(300):
        dtype, t = (("f16", torch.float16), ("bf16", torch.bfloat16))[trial % 2]
        tops = 2.0 ** np.sort(rng.integers(-12, 14, 16))
        z = rng.uniform(0.5, 1, (16, 64)) * tops[:, None] * 2.0 ** rng.integers(-18, 1, (16, 64))
        z[:, 0] = tops
        z = torch.from_numpy(z * rng.choice([-1, 1], z.shape)).to(t).double().numpy()
        y, x, scales = run(z[:, None, None], dtype)
        e = scales[0].astype(int).T[..., None] - 127
        off, rel = np.abs(y - x), 2.0 ** -4 * np.abs(x)
        assert ((off <= rel) | (off < 2.0 ** (e - 9.0))).all()
        last = off[-1]  # never rounded again
        assert (last <= np.maximum(rel[-1], 2.0 ** (e - 10.0))).all()
        past += int((off > np.maximum(rel, 2.0 ** (e - 10.0))).sum())
    assert past  # the bound of one rounding does not hold for all

    # Where 2^-4 of the element no longer holds: below 2^(e - 6), 2^-13 of any largest.
    for top in (240.0, 448.0):
        z = np.full(64, 7.5 * 2.0 ** -9)
        z[0] = top
        y, x, _ = run([z], "f16")
        assert abs(y - x).max() == 2.0 ** -10 > 2.0 ** -4 * 7.5 * 2.0 ** -9
    z = np.concatenate([[225.0], 225.0 * 2.0 ** -13 * np.linspace(1, 2, 63)])
    y, x, scales = run([z], "bf16")
    assert scales[0, 0, 0] == 127 and (np.abs(y - x) <= 2.0 ** -4 * np.abs(x)).all()
