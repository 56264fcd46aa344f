"""GPU: the 8-bit cache, cross attention and page tables, through the engine and the
C ABI, against the fp64 oracle; poison everywhere no query looks.  Tolerances are
derived in tests/context_cases.py; what is held in 8 bits and whole numbers are
equal."""
import numpy as np
import pytest
import torch

from oracle import context as oc
from oracle import serving as sv
from paged_kv_gqa_block_amd import _lib, _serving, engine
from tests.context_cases import TORCH, check, f64
from tests.parity import say
from tests.serving_cases import Batch8, cross_reference, make_cross

pytestmark = pytest.mark.gpu

LENS = [0, 1, 15, 16, 17, 33, 100, 250, 700]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def _same(a, b):
    view = {8: torch.int64, 2: torch.int16, 4: torch.int32, 1: torch.uint8}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


def _i32(x):
    return torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()


def _offsets(counts):
    return _i32(np.concatenate([[0], np.cumsum(counts)]))


def _equal_codes(got, want):
    """Pool bytes, either sign of a NaN alike."""
    nan = ((got & 127) == 127) & ((want & 127) == 127)
    np.testing.assert_array_equal(np.where(nan, 0, got), np.where(nan, 0, want))


# ---- the 8-bit cache ---------------------------------------------------------------

def _special(n, hkv, d, dtype, seed):
    """New tokens [n][2][Hkv][d] of every size: powers of two apart, ties between
    codes, signed zeros, the largest numbers, infinities and NaN."""
    rng = np.random.default_rng(seed)
    lo, hi = (-20, 15) if dtype == "f16" else (-126, 127)
    x = rng.standard_normal((n, 2, hkv, d)) * 2.0 ** rng.integers(lo, hi, (n, 2, hkv, 1))
    kind = rng.integers(0, 10, (n, 2, hkv, 1))
    ties = (rng.integers(0, 128, x.shape) + 0.5) / 64 * rng.choice([-1, 1], x.shape)
    x = np.where(kind == 0, 0.0, x)
    x = np.where(kind == 1, ties, x)
    x = np.where(kind == 2, rng.standard_normal(x.shape), x)
    x = np.where((kind == 3) & (rng.random(x.shape) < 0.05), np.inf, x)
    x = np.where((kind == 4) & (rng.random(x.shape) < 0.05), np.nan, x)
    big = 65504.0 if dtype == "f16" else 3.3895e38
    x = np.where((kind == 5) & (rng.random(x.shape) < 0.1), -big, x)
    with np.errstate(over="ignore"):
        return torch.from_numpy(x.astype(np.float32)).to(TORCH[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,hkv,runs", [
    (128, 2, [[5, 0, 33, 16, 64, 17], [3, 1, 20, 1, 0, 15], [9, 1, 1, 1, 1, 1]]),
    (64, 3, [[1, 40, 15, 100], [17, 0, 2, 49]] + [[1, 1, 1, 1]] * 5),
    (128, 1, [[200], [7], [1], [300]]),
    (64, 8, [[1, 1, 1]] * 9),
])
def test_store_writes_the_oracle_bytes_and_load_reads_them(d, hkv, runs, dtype):
    """Run after run into the same rows: blocks that start anew, that grow, that do not."""
    say(f"[kv8 store/load] d={d} Hkv={hkv} {dtype} runs={runs}")
    b = len(runs[0])
    final = np.sum(runs, 0)
    rng = np.random.default_rng(d + hkv)
    width = int(final.max()) // 16 + 2
    pages = b * width + 3
    table = rng.permutation(pages)[:b * width].reshape(b, width).astype(np.int32)
    prob = engine.make_problem(b, 4 * hkv, hkv, d, 16, pages, width, dtype)
    ref = sv.Cache8(pages, hkv, d, dtype)
    ref.codes[:] = rng.integers(0, 256, ref.codes.shape)  # what dead bytes hold does not matter
    ref.scales[:] = rng.integers(0, 256, ref.scales.shape)
    cache = engine.Kv8Cache(prob, pool=torch.from_numpy(ref.bytes()).cuda(),
                            scales=torch.from_numpy(ref.scales.copy()).cuda())
    bt, lens = _i32(table), np.zeros(b, dtype=np.int64)
    for i, new in enumerate(runs):
        n = sum(new)
        kv = _special(n, hkv, d, dtype, 10 * i + d)
        dev = kv.cuda()
        lens += new
        off = None if all(m == 1 for m in new) else _offsets(new)
        cache.store(dev[:, 0], dev[:, 1], bt, _i32(lens), off)
        out = [torch.full((n, hkv, d), 7.0, dtype=TORCH[dtype], device="cuda") for _ in range(2)]
        cache.load(bt, _i32(lens), off, *out)
        torch.cuda.synchronize()
        want = np.zeros((n, 2, hkv, d))
        at = 0
        for r, m in enumerate(new):
            p, end = lens[r] - m, lens[r]
            while p < end:
                k = min(end, p // 16 * 16 + 16) - p
                page = table[r, p // 16]
                ref.store(page, p % 16, f64(kv[at:at + k]))
                for j in range(k):
                    want[at + j] = ref.values(page, p % 16 + j)
                at, p = at + k, p + k
        np.testing.assert_array_equal(cache.scales.cpu().numpy(), ref.scales)
        _equal_codes(cache.pool.cpu().numpy(), ref.bytes())
        for x in range(2):
            np.testing.assert_array_equal(f64(out[x]), want[:, x])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_finite_value_quantises_like_the_oracle(dtype):
    """All finite 16-bit values: sorted by size, so that every exponent is a block's
    own, and shuffled beside a largest element of every exponent."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(TORCH[dtype])
    x = x[torch.isfinite(x)]
    parts = [x[x.double().abs().argsort()]]
    lo, hi = (-24, 16) if dtype == "f16" else (-130, 128)
    rng = np.random.default_rng(2)
    tops = [2.0 ** e * 1.75 for e in range(lo, hi, 1 if dtype == "f16" else 9)]
    for top in tops:
        y = x[x.double().abs() <= top]
        y = y[torch.from_numpy(rng.permutation(y.numel()))][:64 * 60]
        parts.append(torch.cat([y, y.new_zeros(-y.numel() % 60)]).view(-1, 60).double())
        parts[-1] = torch.cat([parts[-1], torch.full((parts[-1].shape[0], 4), top).double()],
                              1).to(TORCH[dtype]).flatten()
    v = torch.cat([p for p in parts])
    v = torch.cat([v, v.new_zeros(-v.numel() % 1024)]).view(-1, 1, 64)
    n = v.shape[0]
    width = n // 16
    prob = engine.make_problem(1, 1, 1, 64, 16, width, width, dtype)
    cache = engine.Kv8Cache(prob)
    bt = torch.arange(width, dtype=torch.int32).view(1, -1).cuda()
    dev = v.cuda()
    neg = (-v).cuda()
    cache.store(dev, neg, bt, _i32([n]), _i32([0, n]))
    k, w = torch.empty_like(dev), torch.empty_like(dev)
    cache.load(bt, _i32([n]), _i32([0, n]), k, w)
    torch.cuda.synchronize()
    ref = sv.Cache8(1, 1, 64, dtype)
    want = np.zeros((n, 64))
    for p in range(width):
        z = f64(v[16 * p:16 * p + 16])[:, None]
        ref.store(0, 0, np.concatenate([z, -z], 1))
        assert tuple(cache.scales[p, 0].tolist()) == tuple(ref.scales[0, 0])
        for s in range(16):
            want[16 * p + s] = ref.values(0, s)[0, 0]
    np.testing.assert_array_equal(f64(k)[:, 0], want)
    np.testing.assert_array_equal(f64(w)[:, 0], -want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_code_rounds_again_like_the_oracle(dtype):
    """All codes in earlier tokens of blocks that grow by 0 to 22 binades."""
    d, hkv = 128, 1
    lo, hi = sv.EXP8[dtype]
    grow = list(range(23))
    pages = len(grow)
    ref = sv.Cache8(pages, hkv, d, dtype)
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    base = lo if dtype == "f16" else -20
    new = np.zeros((pages, 2, hkv, d))
    for p, by in enumerate(grow):
        ref.codes[p, 0, :, 0:2] = codes
        ref.codes[p, 0, :, 2:15] = np.arange(13)[:, None] + codes[0] // 2
        ref.scales[p] = base + 127
        new[p, :, 0, 7] = 300.0 * 2.0 ** (base + by)
    kv = torch.from_numpy(new.astype(np.float32)).to(TORCH[dtype])
    prob = engine.make_problem(pages, 4, hkv, d, 16, pages, 1, dtype)
    cache = engine.Kv8Cache(prob, pool=torch.from_numpy(ref.bytes()).cuda(),
                            scales=torch.from_numpy(ref.scales.copy()).cuda())
    bt = torch.arange(pages, dtype=torch.int32).view(-1, 1).cuda()
    dev = kv.cuda()
    cache.store(dev[:, 0], dev[:, 1], bt, _i32([16] * pages))
    torch.cuda.synchronize()
    for p in range(pages):
        ref.store(p, 15, f64(kv[p:p + 1]))
    np.testing.assert_array_equal(cache.scales.cpu().numpy(), ref.scales)
    _equal_codes(cache.pool.cpu().numpy(), ref.bytes())


def test_store_and_load_skip_what_is_not_in_the_cache():
    """Rows with a length outside the table, tokens at negative positions and
    pages outside the pool: nothing is stored, nothing is read back, and rows
    behind the last offset stay as they were."""
    d, hkv, width, pages = 128, 2, 3, 9
    lens = [40, -5, 1000, 3, 33]
    new = [40, 2, 4, 6, 20]  # row 3: three of its tokens at negative positions
    table = np.arange(15, dtype=np.int32).reshape(5, 3) % pages
    table[0], table[3], table[4] = [0, -1, 9], [3, 0, 0], [1, 4, 2 ** 31 - 1]
    n = sum(new) + 2
    say("[kv8 skips]")
    prob = engine.make_problem(5, 4, hkv, d, 16, pages, width, "f16")
    x = torch.randn(n, hkv, d, generator=torch.Generator().manual_seed(0)).half().cuda()
    bt, sl, off = _i32(table), _i32(lens), _offsets(new)
    cache = engine.Kv8Cache(prob)
    cache.pool.fill_(99)
    cache.scales.fill_(98)
    cache.store(x, x, bt, sl, off)
    got = [torch.full_like(x, 5.0) for _ in range(2)]
    cache.load(bt, sl, off, *got)
    torch.cuda.synchronize()
    written, at = {}, 0
    for row in range(5):
        for i in range(new[row]):
            p = lens[row] - new[row] + i
            if 0 <= lens[row] <= width * 16 and p >= 0 and 0 <= table[row, p // 16] < pages:
                written[table[row, p // 16], p % 16] = at
            at += 1
    back = set(written.values())
    for tok in range(n):
        untouched = bool((got[0][tok] == 5).all()) and bool((got[1][tok] == 5).all())
        assert untouched == (tok not in back), tok
    pool, scales = cache.pool.cpu().numpy(), cache.scales.cpu().numpy()
    k_at, v_at = sv.kv8_places(d)
    for pg in range(pages):
        slots = [s for p, s in written if p == pg]
        assert (scales[pg] == 98).all() == (not slots), pg
        # Row 4 enters page 1 at slot 13: what lies before are earlier tokens, whose
        # block grows.
        dead = [s for s in range(16) if s not in slots and not (pg == 1 and s < 13)]
        assert (pool[pg][:, k_at[dead].ravel()] == 99).all(), pg
        assert (pool[pg][:, v_at[dead].ravel()] == 99).all(), pg


# ---- decode and prompts over it --------------------------------------------------------

VIEWS = [(0, 0), (1, 0), (1, 1), (15, 4), (16, 16), (17, 40), (100, 5), (250, 0), (10 ** 6, 3),
         (64, 10 ** 6), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("d,dtype", [(128, "f16"), (128, "bf16"), (64, "f16"), (64, "bf16")])
@pytest.mark.parametrize("window,sinks", VIEWS)
def test_decode_view(window, sinks, d, dtype):
    seed = VIEWS.index((window, sinks))
    group, hkv = [(4, 2), (1, 3), (8, 1), (16, 1), (5, 2), (2, 8), (3, 1)][seed % 7]
    b = Batch8(seed, LENS, hkv=hkv, group=group, d=d, dtype=dtype, window=window, sinks=sinks)
    ref, w = b.reference(), b.device()
    for splits in (None, 1, 3, 100):
        say(f"[kv8 view] W={window} S={sinks} d={d} {dtype} G={group} Hkv={hkv} splits={splits}")
        step = engine.Kv8Step(b.problem(), window, sinks, splits)
        out, lse = step.run(w)
        torch.cuda.synchronize()
        check(out, lse, ref, dtype, d, b.vmax, False, f"splits {splits}")
        first = out.clone()
        step.run(w)
        torch.cuda.synchronize()
        assert _same(first, step.out)  # the workspace carries nothing over


@pytest.mark.parametrize("group,hkv", [(1, 1), (2, 1), (3, 2), (6, 1), (7, 1), (9, 1), (13, 2), (16, 2)])
def test_decode_head_groups(group, hkv):
    for d in (64, 128):
        say(f"[kv8 groups] G={group} Hkv={hkv} d={d}")
        b = Batch8(group, [37, 600, 0, 129], hkv=hkv, group=group, d=d, window=90, sinks=3)
        out, lse = engine.Kv8Step(b.problem(), 90, 3).run(b.device())
        torch.cuda.synchronize()
        check(out, lse, b.reference(), "f16", d, b.vmax, False, "groups")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("scale,spread", [(-0.2, 1.0), (0.0, 1.0), (1.0, 2.0), (1e-30, 1.0)])
def test_scales(scale, spread, many):
    """A negative scale, zero, and scores far apart."""
    for dtype in ("f16", "bf16"):
        say(f"[kv8 scale] {scale} {dtype} prompt={many}")
        b = Batch8(5, [70, 300], [70, 9] if many else None, scale=scale, spread=spread, dtype=dtype)
        step = engine.PromptStep(b.problem(), 79) if many else engine.Kv8Step(b.problem())
        out, lse = step.run(b.device())
        torch.cuda.synchronize()
        check(out, lse, b.reference(), dtype, 128, b.vmax, many, f"scale {scale}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("spread", [2.0 ** -9, 2.0 ** 9])
def test_values_of_other_sizes(spread, dtype):
    """Scales far from one: K and V a few binades above the type's floor, and large."""
    say(f"[kv8 spread] {spread} {dtype}")
    b = Batch8(15, [120, 33], [60, 33], scale=1 / (11 * spread), spread=spread, dtype=dtype, d=64)
    w = b.device()
    out, lse = engine.PromptStep(b.problem(), 93).run(w)
    torch.cuda.synchronize()
    check(out, lse, b.reference(), dtype, 64, b.vmax, True, "prompt")
    b.new[:] = 1
    b.q = b.q[:2].contiguous()
    out, lse = engine.Kv8Step(b.problem()).run(dict(w, q=b.q.cuda()))
    torch.cuda.synchronize()
    check(out, lse, b.reference(), dtype, 64, b.vmax, False, "decode")


def test_bad_rows_and_pages():
    """A length outside the table makes the row empty; a page outside the pool
    holds no tokens, also where it is all that a row has."""
    b = Batch8(3, [100, 50, 20, 33, 16], window=60, sinks=2)
    pool = b.pool8.shape[0]
    cap = b.table.shape[1] * 16
    w = b.device()
    w["seq_lens"] = _i32([100, -3, cap + 1, 33, 16])
    bt = b.table.copy()
    bt[0, 4], bt[3, 0], bt[4, 0] = -1, pool, 2 ** 31 - 1
    w["block_table"] = _i32(bt)
    ref = b.reference(lens=[100, 0, 0, 33, 16], present=lambda r, pg: 0 <= bt[r, pg] < pool)
    for splits in (1, 4):
        say(f"[kv8 bad pages] splits={splits}")
        out, lse = engine.Kv8Step(b.problem(), 60, 2, splits).run(w)
        torch.cuda.synchronize()
        check(out, lse, ref, "f16", 128, b.vmax, False, "bad pages")
    assert not out[1].any() and not out[4].any()


def test_decode_long_and_many_rows():
    b = Batch8(8, [20011, 17], hkv=1, group=4, dtype="bf16")
    ref, w = b.reference(), b.device()
    for splits in (None, 2, 500):
        say(f"[kv8 long row] splits={splits}")
        out, lse = engine.Kv8Step(b.problem(), splits=splits).run(w)
        torch.cuda.synchronize()
        check(out, lse, ref, "bf16", 128, b.vmax, False, "long")
    b = Batch8(9, np.random.default_rng(1).integers(0, 41, 150), hkv=1, group=2, d=64, window=20,
               sinks=1)
    ref = b.reference()
    for splits in (1, 2):
        say(f"[kv8 many rows] splits={splits}")
        out, lse = engine.Kv8Step(b.problem(), 20, 1, splits).run(b.device())
        torch.cuda.synchronize()
        check(out, lse, ref, "f16", 64, b.vmax, False, "many rows")


RUNS = [
    ([1], [1]),
    ([70], [70]),
    ([300, 0, 17, 45, 200], [300, 0, 1, 20, 7]),
    ([129, 64, 65, 16, 15], [129, 64, 65, 16, 15]),
    ([400, 600], [3, 150]),
]


@pytest.mark.parametrize("d,dtype", [(128, "f16"), (128, "bf16"), (64, "f16"), (64, "bf16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (16, 4), (50, 33), (64, 0),
                                          (190, 17), (10 ** 6, 0)])
@pytest.mark.parametrize("run", range(len(RUNS)))
def test_prompt(run, window, sinks, d, dtype):
    lens, new = RUNS[run]
    group, hkv = [(4, 2), (1, 1), (8, 1), (5, 1), (16, 1)][(run + window) % 5]
    say(f"[kv8 prompt] lens={lens} new={new} W={window} S={sinks} d={d} {dtype} G={group} "
        f"Hkv={hkv}")
    b = Batch8(run, lens, new, hkv=hkv, group=group, d=d, dtype=dtype, window=window, sinks=sinks)
    step = engine.PromptStep(b.problem(), int(b.new.sum()), window, sinks)
    out, lse = step.run(b.device())
    torch.cuda.synchronize()
    check(out, lse, b.reference(), dtype, d, b.vmax, True, "prompt")


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40])
def test_prompt_splits(splits):
    """Few queries over long contexts, the keys cut into ranges; twice on one
    workspace, with the same bits."""
    for d, dtype in ((128, "bf16"), (64, "f16")):
        say(f"[kv8 prompt splits] {splits} d={d} {dtype}")
        b = Batch8(splits, [1500, 0, 70, 900], [3, 0, 70, 33], hkv=2, group=4, d=d, dtype=dtype)
        step = engine.PromptStep(b.problem(), 106, splits=splits)
        out, lse = step.run(b.device())
        torch.cuda.synchronize()
        check(out, lse, b.reference(), dtype, d, b.vmax, True, "splits")
        first = out.clone()
        step.run(b.device())
        torch.cuda.synchronize()
        assert _same(first, step.out)


# Tiles of uneven cost in even shares: rows of 1 to 94 steps, some of one token, one empty.
UNEVEN = ([6000, 40, 900, 0, 300], [70, 40, 100, 5, 33])


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 3)])
def test_prompt_in_shares(window, sinks, d, dtype):
    lens, new = UNEVEN
    b = Batch8(71, lens, new, hkv=2, group=4, d=d, dtype=dtype, window=window, sinks=sinks)
    ref, w = b.reference(), b.device()
    for splits in (None, 2, 3, 5, 9, 40):
        say(f"[kv8 shares] W={window} d={d} {dtype} splits={splits}")
        step = engine.PromptStep(b.problem(), int(b.new.sum()), window, sinks, splits)
        for _ in range(2):  # on one workspace, with the same bits
            out, lse = step.run(w)
            torch.cuda.synchronize()
            check(out, lse, ref, dtype, d, b.vmax, True, f"splits {splits}")
            first = out.clone() if _ == 0 else first
        assert _same(first, out) and not step.workspace[:256 << 10].any()


@pytest.mark.parametrize("kind", [16, 4, 8])
@pytest.mark.parametrize("d,dtype", [(128, "f16"), (64, "bf16")])
def test_cross_in_shares(d, dtype, kind):
    lens, queries = UNEVEN
    b = make_cross(kind, 72, lens, queries, hkv=2, group=4, d=d, dtype=dtype)
    ref, w = cross_reference(b), b.device()
    for splits in (None, 2, 3, 5, 9, 40, 200):
        say(f"[cross shares] d={d} {dtype} bits={kind} splits={splits}")
        step = engine.CrossStep(b.problem(), int(b.new.sum()), splits)
        out, lse = step.run(w)
        torch.cuda.synchronize()
        check(out, lse, ref, dtype, d, b.vmax, True, f"splits {splits}")
        assert not step.workspace[:256 << 10].any()


def test_shares_over_many_rows():
    """More rows than a wave holds, one of them long; prompts and cross attention."""
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 60, 90)
    lens[77] = 4000
    new = np.minimum(lens, rng.integers(0, 50, 90))
    new[77] = 130
    n = int(new.sum())
    for splits in (None, 6):
        say(f"[shares, rows] splits={splits}")
        b = Batch8(73, lens, new, hkv=1, group=3, d=64)
        step = engine.PromptStep(b.problem(), n, splits=splits)
        out, lse = step.run(b.device())
        torch.cuda.synchronize()
        check(out, lse, b.reference(), "f16", 64, b.vmax, True, "prompt")
        b = make_cross(8, 74, lens, new, hkv=1, group=3, d=64)
        out, lse = engine.CrossStep(b.problem(), n, splits).run(b.device())
        torch.cuda.synchronize()
        check(out, lse, cross_reference(b), "f16", 64, b.vmax, True, "cross")


def test_prompt_outside_the_row_and_behind_the_last():
    """Runs longer than their rows, invalid lengths, pages outside the pool; output
    rows behind the last offset stay as they were."""
    b = Batch8(7, [30, 60, 20, 50], [45, 60, 5, 9], window=25, sinks=1, dtype="bf16")
    pool = b.pool8.shape[0]
    bt = b.table.copy()
    bt[1, 1], bt[3, 3] = -7, pool
    w = b.device()
    w["block_table"], w["seq_lens"] = _i32(bt), _i32([30, 60, 10 ** 9, 50])
    ref = b.reference(lens=[30, 60, 0, 50], present=lambda r, pg: 0 <= bt[r, pg] < pool)
    n = int(b.new.sum())
    w["q"] = torch.cat([w["q"], torch.zeros_like(w["q"][:3])])
    step = engine.PromptStep(b.problem(), n + 3, 25, 1)
    step.out.fill_(3.0)
    step.lse.fill_(3.0)
    say("[kv8 prompt outside]")
    out, lse = step.run(w)
    torch.cuda.synchronize()
    check(out[:n], lse[:n], ref, "bf16", 128, b.vmax, True, "outside")
    assert (out[n:] == 3).all() and (lse[n:] == 3).all()


def test_non_finite_seen_token_stays_in_its_row():
    """A NaN stored in K of a token that queries see: those of its row that see it give
    NaN, and every other row keeps its bits."""
    lens, new, row, tok = [300, 200, 90, 64], [40, 70, 90, 3], 1, 150
    for many in (False, True):
        say(f"[kv8 non-finite] prompt={many}")
        b = Batch8(41, lens, new if many else None, hkv=2, group=4)
        w = b.device()
        step = (engine.PromptStep(b.problem(), int(b.new.sum())) if many
                else engine.Kv8Step(b.problem()))
        out = step.run(w)[0].clone()
        k_at, _ = sv.kv8_places(128)
        w["kv8_pool"][int(b.table[row, tok // 16]), :, int(k_at[tok % 16, 3])] = 0x7f
        bad, _ = step.run(w)
        torch.cuda.synchronize()
        at = np.concatenate([[0], np.cumsum(b.new)])
        for r in range(4):
            span = slice(int(at[r]), int(at[r + 1]))
            if r != row:
                assert _same(out[span], bad[span]), r
        first = int(at[row]) + max(0, tok - (lens[row] - int(b.new[row])))
        assert torch.isnan(bad[first:int(at[row + 1])]).all()


@pytest.mark.parametrize("kind", ["kv8", "cross"])
def test_pages_beyond_4_gib(kind):
    """The same rows in a small pool and at the far end of a pool whose byte
    offsets pass 2^32: every call gives the same bits."""
    b = Batch8(21, [300, 77], [40, 77], hkv=8, group=2, window=100, sinks=3, dtype="bf16",
               everything=True)
    w = b.device()
    small = w["kv8_pool"].shape[0]
    big = (1 << 32) // (8 * 4096) + 1000
    shift = big - small
    far = dict(w, block_table=w["block_table"] + shift)
    say(f"[kv8 far pages] {kind} pages={big}")
    for name in ("kv8_pool", "kv8_scales"):
        far[name] = torch.zeros(big, *w[name].shape[1:], dtype=torch.uint8, device="cuda")
        far[name][shift:] = w[name]
    n = int(b.new.sum())
    qd = {"q": w["q"][:2].contiguous(), "tok_offsets": None}
    outs = []
    for pr, x in ((b.problem(), w), (b.problem(num_pool_pages=big), far)):
        if kind == "cross":
            got = [t.clone() for t in engine.CrossStep(pr, n).run(x)]
            got += [t.clone() for t in engine.CrossStep(pr, 2).run(dict(x, **qd))]
        else:
            got = [t.clone() for t in engine.PromptStep(pr, n, 100, 3).run(x)]
            got += [t.clone() for t in engine.Kv8Step(pr, 100, 3).run(dict(x, **qd))]
            kv = torch.linspace(-3, 3, n * 8 * 128, device="cuda").to(torch.bfloat16).view(n, 8, 128)
            args = (x["block_table"], x["seq_lens"], x["tok_offsets"])
            cache = engine.Kv8Cache(pr, pool=x["kv8_pool"], scales=x["kv8_scales"])
            cache.store(kv, kv, *args)
            got += list(cache.load(*args, torch.empty_like(kv), torch.empty_like(kv)))
            got += [x["kv8_pool"][-small:].clone(), x["kv8_scales"][-small:].clone()]
        torch.cuda.synchronize()
        outs.append(got)
    for a, c in zip(*outs):
        assert _same(a, c)


# ---- cross attention ---------------------------------------------------------------------

# Few queries a row (tiles of sixteen) and many (of 128); rows without queries, rows
# without states, runs that end inside a tile and pass one.
CROSS = [
    ([33], [1]),
    ([700, 0, 1, 16, 250], [1, 2, 1, 3, 0]),
    ([100, 45, 900], [5, 1, 17]),
    ([129, 64, 0, 15, 333], [64, 65, 5, 0, 200]),
    ([1500, 20], [3, 150]),
]


def _takes_few(b):
    """Whether the call takes tiles of sixteen queries: by the average alone, and more
    where pairs of row and KV head are few."""
    return _few(int(b.new.sum()) * b.group, len(b.lens), b.hkv)


def _few(queries, rows, hkv):
    return queries <= (64 if rows * hkv <= 64 else 32) * rows


@pytest.mark.parametrize("kind", [16, 4, 8])
@pytest.mark.parametrize("d,dtype", [(128, "f16"), (128, "bf16"), (64, "f16"), (64, "bf16")])
@pytest.mark.parametrize("run", range(len(CROSS)))
def test_cross(run, d, dtype, kind):
    lens, queries = CROSS[run]
    for group, hkv in ((4, 2), (1, 3), (16, 1), (5, 2)):
        b = make_cross(kind, run, lens, queries, hkv=hkv, group=group, d=d, dtype=dtype)
        ref, w, n = cross_reference(b), b.device(), int(b.new.sum())
        for splits in (None, 1, 3):
            say(f"[cross] lens={lens} queries={queries} d={d} {dtype} bits={kind} G={group} "
                f"Hkv={hkv} splits={splits} few={_takes_few(b)}")
            step = engine.CrossStep(b.problem(), n, splits)
            out, lse = step.run(w)
            torch.cuda.synchronize()
            check(out, lse, ref, dtype, d, b.vmax, not _takes_few(b), f"splits {splits}")
            first = out.clone()
            step.run(w)
            torch.cuda.synchronize()
            assert _same(first, step.out)
            assert not step.workspace[:256 << 10].any()


@pytest.mark.parametrize("kind", [16, 4, 8])
def test_cross_one_query_per_row_without_offsets(kind):
    b = make_cross(kind, 6, LENS, [1] * len(LENS), hkv=2, group=8)
    w = b.device()
    del w["tok_offsets"]
    for splits in (None, 1, 5):
        say(f"[cross, no offsets] bits={kind} splits={splits}")
        out, lse = engine.CrossStep(b.problem(), len(LENS), splits).run(w)
        torch.cuda.synchronize()
        check(out, lse, cross_reference(b), "f16", 128, b.vmax, False, "no offsets")


def test_cross_agrees_with_decode_over_the_whole_row():
    """One query a row sees what a decode step without a window sees."""
    b = make_cross(16, 4, [500, 3, 0, 129], [1] * 4)
    w = b.device()
    out, lse = engine.CrossStep(b.problem(), 4).run(w)
    want, want_lse = engine.WindowStep(b.problem()).run(w)
    torch.cuda.synchronize()
    assert (out.float() - want.float()).abs().max() <= 2e-3
    torch.testing.assert_close(lse, want_lse, rtol=0, atol=4e-4)


@pytest.mark.parametrize("scale,spread", [(-0.3, 1.0), (0.0, 1.0), (1.0, 2.0)])
@pytest.mark.parametrize("queries", [[2, 3], [90, 40]])
def test_cross_scales(queries, scale, spread):
    for kind, dtype in ((16, "bf16"), (8, "f16"), (4, "f16")):
        say(f"[cross scale] {scale} queries={queries} bits={kind}")
        b = make_cross(kind, 2, [90, 310], queries, scale=scale, dtype=dtype, spread=spread)
        out, lse = engine.CrossStep(b.problem(), sum(queries)).run(b.device())
        torch.cuda.synchronize()
        check(out, lse, cross_reference(b), dtype, 128, b.vmax, not _takes_few(b), "scale")


@pytest.mark.parametrize("kind", [16, 4, 8])
@pytest.mark.parametrize("queries", [[3, 1, 2, 4, 1], [45, 60, 5, 9, 30]])
def test_cross_bad_rows_and_pages(queries, kind):
    """Lengths outside the table and pages outside the pool; output rows behind the
    last offset stay as they were."""
    b = make_cross(kind, 7, [100, 60, 20, 50, 16], queries, dtype="bf16")
    pool = (b.pool4 if kind == 4 else b.pool8 if kind == 8 else b.kp).shape[0]
    bt = b.table.copy()
    bt[0, 4], bt[1, 1], bt[3, 3], bt[4, 0] = -1, -7, pool, 2 ** 31 - 1
    w = b.device()
    w["block_table"], w["seq_lens"] = _i32(bt), _i32([100, 60, 10 ** 9, 50, 16])
    ref = cross_reference(b, lens=[100, 60, 0, 50, 16],
                          present=lambda r, pg: 0 <= bt[r, pg] < pool)
    n = int(b.new.sum())
    w["q"] = torch.cat([w["q"], torch.zeros_like(w["q"][:3])])
    for splits in (None, 1, 3):
        say(f"[cross bad pages] bits={kind} queries={queries} splits={splits}")
        step = engine.CrossStep(b.problem(), n + 3, splits)
        step.out.fill_(3.0)
        step.lse.fill_(3.0)
        out, lse = step.run(w)
        torch.cuda.synchronize()
        check(out[:n], lse[:n], ref, "bf16", 128, b.vmax, not _takes_few(b), "bad pages")
        assert (out[n:] == 3).all() and (lse[n:] == 3).all()


@pytest.mark.parametrize("rows", [63, 64, 65, 150])
def test_cross_of_many_rows(rows):
    """Rows around and beyond what a wave holds, some without queries or states."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, 90, rows) * (rng.random(rows) < 0.9)
    for most in (4, 40):
        queries = rng.integers(0, most, rows)
        b = make_cross(8, rows, lens, queries, hkv=1, group=3, d=64)
        ref = cross_reference(b)
        for splits in (None, 4):
            say(f"[cross rows] rows={rows} queries={queries.sum()} splits={splits}")
            out, lse = engine.CrossStep(b.problem(), int(queries.sum()), splits).run(b.device())
            torch.cuda.synchronize()
            check(out, lse, ref, "f16", 64, b.vmax, not _takes_few(b), "many rows")


def test_cross_rows_that_share_pages():
    """Beams as queries of one row, and as rows over the same pages: both within the
    bounds (not the same bits: a tile's running maxima move together)."""
    b = make_cross(8, 12, [400], [4], group=4)
    w = b.device()
    out, lse = engine.CrossStep(b.problem(), 4, splits=1).run(w)
    prob = b.problem(batch=4)
    apart = dict(w, block_table=w["block_table"].repeat(4, 1), seq_lens=w["seq_lens"].repeat(4),
                 tok_offsets=None)
    out4, lse4 = engine.CrossStep(prob, 4, splits=1).run(apart)
    torch.cuda.synchronize()
    for got in ((out, lse), (out4, lse4)):
        check(*got, cross_reference(b), "f16", 128, b.vmax, False, "beams")


def test_workspace_of_all_shapes():
    """One workspace, in turn, for calls of every kind and size."""
    a = make_cross(8, 1, [900, 77], [3, 2], hkv=2, group=4)
    c = make_cross(16, 2, [1500, 600, 8], [100, 1, 30], hkv=1, group=8, d=64)
    e = Batch8(3, [2000, 50, 300], hkv=2, group=4)
    p = Batch8(4, [2100, 60], [30, 20], hkv=2, group=4)
    steps = [(engine.CrossStep(a.problem(), 5, 6), a.device(), cross_reference(a), a, False),
             (engine.CrossStep(c.problem(), 131, 4), c.device(), cross_reference(c), c, True),
             (engine.Kv8Step(e.problem(), splits=9), e.device(), e.reference(), e, False),
             (engine.PromptStep(p.problem(), 50, splits=7), p.device(), p.reference(), p, True)]
    ws = torch.zeros(max(s.workspace.numel() for s, *_ in steps), dtype=torch.uint8, device="cuda")
    for s, *_ in steps:
        s._own = (ws.data_ptr(), ws.numel(), *s._own[2:])
    for i in range(3):
        say(f"[one workspace] {i}")
        for s, w, ref, b, one_part in steps:
            out, lse = s.run(w)
            torch.cuda.synchronize()
            check(out, lse, ref, "f16", b.d, b.vmax, one_part, type(s).__name__)
    assert not ws[:256 << 10].any()


@pytest.mark.parametrize("kind", [16, 4, 8])
def test_cross_in_a_workspace_of_fewer_ranges(kind):
    """As many ranges as the workspace holds, and nothing behind it is written."""
    b = make_cross(kind, 7, [3000, 1200, 40], [3, 2, 6], hkv=2, group=4)
    prob, w = b.problem(), b.device()
    step, ref = engine.CrossStep(prob, 11, 40), cross_reference(b)
    for room in (2, 3, 7, 39):
        n = _serving.pkv_cross_workspace_bytes(prob, 11, False, room) + 15
        ws = torch.zeros(n + (1 << 20), dtype=torch.uint8, device="cuda")
        ws[n:] = 77
        step._own = (ws.data_ptr(), n, *step._own[2:])
        for i in range(2):
            say(f"[room for {room} ranges] {i}")
            step.out.fill_(float("nan"))
            out, lse = step.run(w)
            torch.cuda.synchronize()
            check(out, lse, ref, "f16", 128, b.vmax, False, f"{room} ranges")
        assert (ws[n:] == 77).all() and not ws[:256 << 10].any()
        assert ws[256 << 10:n - 15].any()


def _shares_step():
    """A prompt whose 8-bit shares take more workspace than its ranges."""
    b = Batch8(71, [3000, 2500], [40, 24], hkv=4, group=4)
    prob = b.problem()
    step = engine.PromptStep(prob, 64)
    step.splits, step.splits8 = 1, 12  # as a larger problem's caps would have it
    step.workspace = torch.empty(0, dtype=torch.uint8, device="cuda")
    step._own = (0, 0, *step._own[2:])
    step._bytes8 = _serving.pkv_prompt_kv8_workspace_bytes(prob, 64, False, 12)
    assert step._bytes8 > 0
    return b, step


def test_prompts_over_other_caches_pay_for_no_shares():
    """A step's workspace is that of its ranges; 8 bits get theirs at their first call."""
    from paged_kv_gqa_block_amd import _context
    for heads, new, rows in ((32, 1024, 8), (32, 1900, 1), (64, 289, 8)):
        prob = engine.make_problem(rows, heads, 8, 128, 16, 64, 512, "bf16")
        cus = torch.cuda.get_device_properties(0).multi_processor_count
        step = engine.PromptStep(prob, new)
        n = _context.pkv_prompt_splits(prob, step.view, new, False, cus)
        assert step.workspace.numel() == _context.pkv_prompt_workspace_bytes(prob, new, False, n)
    b, step = _shares_step()
    w, ref = b.device(), b.reference()
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for i, stream in enumerate((None, torch.cuda.Stream(), torch.cuda.Stream())):
        say(f"[workspace of shares] {i}")
        out, lse = step.run(w, stream)
        torch.cuda.synchronize()
        check(out, lse, ref, "f16", 128, b.vmax, True, "shares")
        if i == 0:
            grown = torch.cuda.memory_allocated() - held
            assert step._bytes8 <= grown < step._bytes8 + (4 << 20)
    assert torch.cuda.memory_allocated() - held <= grown
    assert not step._workspace8[:256 << 10].any()


def test_workspace_of_shares_first_needed_on_a_busy_stream():
    """Its counters are zero before the call, on whatever stream the step was built."""
    building, running = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(building):
        b, step = _shares_step()
        w = b.device()
    torch.cuda.synchronize()
    say("[workspace of shares] busy streams")
    with torch.cuda.stream(building):
        junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        del junk
        _busy(building)
        step.run(w, running)  # the workspace is made here
        running.synchronize()
        out, lse = step.run(w)
    torch.cuda.synchronize()
    check(out, lse, b.reference(), "f16", 128, b.vmax, True, "shares")
    assert not step._workspace8[:256 << 10].any()


@pytest.mark.parametrize("null", [False, True])
def test_workspace_of_shares_first_needed_on_a_stream_given_by_number(null):
    b, step = _shares_step()
    w = b.device()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    say("[workspace of shares] stream by number")
    for number in (0 if null else side.cuda_stream, side.cuda_stream):
        step.out.fill_(float("nan"))
        torch.cuda.synchronize()
        out, lse = step.run(w, number)
        torch.cuda.synchronize()
        check(out, lse, b.reference(), "f16", 128, b.vmax, True, "shares")
    assert not step._workspace8[:256 << 10].any()


def test_workspace_of_shares_first_needed_in_a_capture():
    """The graph clears the workspace it was captured with; eager calls before and between
    its replays have their own."""
    b, step = _shares_step()
    w, ref = b.device(), b.reference()
    q = w["q"].clone()
    graph, again = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step.run(w)
        out, lse = step.run(w)
    with torch.cuda.graph(again):
        step.run(w)
    assert step._workspace8 is None
    for i in range(4):
        for what in (graph.replay, lambda: step.run(w), again.replay, lambda: step.run(w)):
            say(f"[workspace of shares] replay {i}")
            out.fill_(float("nan"))
            w["q"].copy_(q if i % 2 == 0 else -q)
            what()
            torch.cuda.synchronize()
            if i % 2 == 0:
                check(out, lse, ref, "f16", 128, b.vmax, True, "shares")
            assert torch.isfinite(out).all()
    assert step._workspace8.data_ptr() != step._captured8.data_ptr()


# ---- page tables -------------------------------------------------------------------------

def _table(lens, free, pool, width, num_tokens, rng):
    """A PageTable and its oracle: rows of `lens` tokens, `free` pages left."""
    held = [max(0, -(-n // 16)) if n <= width * 16 else 0 for n in lens]
    order = rng.permutation(pool)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = order[at:at + h]
        at += h
    assert at + free <= pool
    t = engine.PageTable(engine.make_problem(len(lens), 1, 1, 64, 16, pool, width, "f16"),
                         num_tokens)
    t.block_table.copy_(_i32(table))
    t.lens.copy_(_i32(lens))
    stack = order[at:at + free]
    t.free_pages[:free] = _i32(stack)
    t.state[0] = free
    return t, sv.Pages(lens, table, stack, pool, width)


def _check_table(t, ref):
    assert t.lens.tolist() == ref.lens and t.block_table.tolist() == ref.table
    assert t.state[0].item() == len(ref.free) and t.state[2].item() == 0
    assert t.free_pages[:len(ref.free)].tolist() == ref.free


def _check_take(t, ref, counts, num_tokens, got):
    seq, off, slots, positions, denied = ref.take(counts, num_tokens)
    assert got["seq_lens"].tolist() == seq and got["tok_offsets"].tolist() == off
    n = off[-1]
    assert got["slots"][:n].tolist() == [slots[i] for i in range(n)]
    assert got["positions"][:n].tolist() == [positions[i] for i in range(n)]
    assert t.state[1].item() == denied
    _check_table(t, ref)
    return n


@pytest.mark.parametrize("rows,most,num_tokens", [(1, 3, 3), (3, 40, 100), (7, 1, 7), (64, 1, 64),
                                                  (65, 30, 700), (300, 20, 4000),
                                                  (1023, 2, 1500), (1030, 4, 512),
                                                  (2100, 3, 9000), (4, 5000, 14000),
                                                  (16, 3, 20000), (1024, 1, 3000)])
def test_page_tables_follow_the_oracle(rows, most, num_tokens):
    """Steps of any counts, rows cut down and ended, lists that run short; one
    workgroup and several, rows beyond one scan."""
    rng = np.random.default_rng(rows)
    width = 40 if most < 100 else 1000
    lens = rng.integers(0, 9 * 16, rows).tolist()
    held = sum(-(-n // 16) for n in lens)
    pool = held + max(4, rows * most // 20)
    t, ref = _table(lens, pool - held, pool, width, num_tokens, rng)
    for i in range(6):
        say(f"[pages] rows={rows} most={most} step {i}")
        counts = rng.integers(-1, most + 1, rows) * (rng.random(rows) < 0.8)
        t.slots.fill_(-9)
        t.positions.fill_(-9)
        got = t.take(_i32(counts))
        torch.cuda.synchronize()
        n = _check_take(t, ref, counts, num_tokens, got)
        assert (t.slots[n:] == -9).all() and (t.positions[n:] == -9).all()
        # All of a row, some of it, or nothing; negative: nothing.
        kind = rng.integers(0, 5, rows)
        keep = np.where(kind == 0, 0, np.where(kind == 1, rng.integers(0, 200, rows),
                                               np.where(kind == 2, -3, 2 ** 31 - 1)))
        if i == 4:
            keep[:] = 0
        t.release(_i32(keep))
        torch.cuda.synchronize()
        ref.release(keep)
        _check_table(t, ref)


def test_many_pages_at_once():
    """A prompt batch of 100000 tokens in, all pages back: many workgroups of both."""
    rng = np.random.default_rng(0)
    counts = rng.integers(0, 3000, 70)
    n = int(counts.sum())
    t, ref = _table([0] * 70, 8000, 8000, 200, n, rng)
    free = list(ref.free)
    say(f"[pages] {n} tokens at once")
    got = t.take(_i32(counts))
    torch.cuda.synchronize()
    _check_take(t, ref, counts, n, got)
    t.release(torch.zeros(70, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    ref.release([0] * 70)
    _check_table(t, ref)
    assert ref.free == free  # the stack as it was


def test_tables_that_do_not_hold_together():
    """Lengths outside the table, counts that overflow, pages outside the pool, more
    or fewer free pages than there can be: rows are turned down, nothing else is touched."""
    rng = np.random.default_rng(3)
    big = 2 ** 31 - 1
    lens, width, pool = [5, -1, 100, 48, 17, 2 ** 30, 0], 3, 30
    t, ref = _table(lens, 12, pool, width, 90, rng)
    t.block_table[4, 1], ref.table[4][1] = pool, pool  # its page lies outside the pool
    for counts in ([1, 2, 3, 1, 4, 5, 20], [big, big, 1, 0, 1, big, 1], [0] * 7, [-5] * 7,
                   [3, 0, 0, 0, 2, 0, 86], [1] * 7):
        say(f"[pages] odd counts {counts}")
        got = t.take(_i32(counts))
        torch.cuda.synchronize()
        _check_take(t, ref, counts, 90, got)
    t.release(_i32([-1, 0, 0, 17, 0, 3, 0]))
    torch.cuda.synchronize()
    ref.release([-1, 0, 0, 17, 0, 3, 0])
    _check_table(t, ref)
    for count in (-4, pool + 7):  # clamped
        t.state[0] = count
        t.lens.zero_()
        t.take(_i32([16] + [0] * 6))
        torch.cuda.synchronize()
        assert t.state[0].item() == (0 if count < 0 else pool - 1)


@pytest.mark.parametrize("rows,num_tokens", [(2, 8), (70, 600), (1100, 40), (1100, 600)])
def test_rows_without_tokens_behind_those_that_overflow(rows, num_tokens):
    """They keep their length: one workgroup and several, rows of a later scan too."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(1, 40, rows).tolist()
    held = sum(-(-n // 16) for n in lens)
    t, ref = _table(lens, 40, held + 40, 60, num_tokens, rng)
    counts = np.zeros(rows, dtype=np.int64)
    counts[0], counts[rows // 2] = num_tokens // 2 + 1, num_tokens // 2
    say(f"[pages] {rows} rows, {num_tokens} tokens and one more")
    got = t.take(_i32(counts))
    torch.cuda.synchronize()
    _check_take(t, ref, counts, num_tokens, got)
    assert got["seq_lens"].tolist()[-1] == (lens[-1] if rows > 2 else 0)
    assert got["seq_lens"].tolist()[1:rows // 2] == lens[1:rows // 2]
    assert t.state[1].item() == 1


@pytest.mark.parametrize("rows,longest,every", [(1, 60, 2), (5, 900, 7), (60, 3000, 50),
                                                (60, 3000, 1), (1500, 100, 30)])
def test_entries_that_name_no_page_do_not_come_back(rows, longest, every):
    """Released by one workgroup and by several: the list holds pages alone, in their
    order, and rows that take them are whole."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(1, longest + 1, rows).tolist()
    held = sum(-(-n // 16) for n in lens)
    t, ref = _table(lens, 9, held + 9, 400, 5000, rng)
    table = np.array(ref.table)
    bad = (rng.integers(0, every, table.shape) == 0) & (table >= 0)
    table[bad] = rng.choice([-1, held + 9, 2 ** 31 - 1, -2 ** 31], int(bad.sum()))
    ref.table = table.tolist()
    t.block_table.copy_(_i32(table))
    say(f"[pages] {int(bad.sum())} of {held} entries name no page")
    for keep in (rng.integers(0, longest, rows), np.zeros(rows, dtype=np.int64)):
        t.release(_i32(keep))
        torch.cuda.synchronize()
        ref.release(keep)
        _check_table(t, ref)
    assert not bad.any() or len(ref.free) < held + 9
    counts = rng.integers(0, 2 * 5000 // rows + 1, rows)
    got = t.take(_i32(counts))
    torch.cuda.synchronize()
    n = _check_take(t, ref, counts, 5000, got)
    served = torch.repeat_interleave(got["seq_lens"] > 0, got["tok_offsets"].diff())
    assert (got["slots"][:n][served] >= 0).all()


def test_new_table_and_no_tokens():
    prob = engine.make_problem(2, 1, 1, 64, 16, 5, 4, "f16")
    t = engine.PageTable(prob, 40)
    got = t.take(_i32([17, 3]))
    torch.cuda.synchronize()
    assert t.block_table.tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]]
    assert got["slots"][:20].tolist() == list(range(17)) + [32, 33, 34]
    assert (got["slots"][20:] == -1).all() and t.state[0].item() == 2
    none = engine.PageTable(prob, 0)
    got = none.take(_i32([1, 0]))  # no room for tokens: turned down
    torch.cuda.synchronize()
    assert got["seq_lens"].tolist() == [0, 0] and none.state.tolist() == [5, 1, 0, 0]
    _serving.pkv_pages_take(prob, _i32([4, 0]), 40, t.lens, t.block_table, t.free_pages, t.state,
                            t.seq_lens, t.tok_offsets)  # without slots and positions
    torch.cuda.synchronize()
    assert t.seq_lens.tolist() == [21, 3] and t.tok_offsets.tolist() == [0, 4, 4]
    with pytest.raises(ValueError, match="counts"):
        t.take(torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="keep"):
        t.release(torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="tokens"):
        engine.PageTable(prob, -1)


# ---- together, as they are used -----------------------------------------------------------

def test_requests_from_start_to_end():
    """Requests come, are cut down and end; pages from the table, prompts and decode
    steps over the 8-bit cache and cross attention to an encoder's states, every call on
    a side stream and every output against the oracle over the caches' values."""
    rng = np.random.default_rng(11)
    hkv, group, d, dtype, rows, width = 2, 4, 128, "f16", 4, 12
    prob = engine.make_problem(rows, hkv * group, hkv, d, 16, 17, width, dtype)
    enc = make_cross(8, 5, [200, 33, 0, 61], [0] * rows, hkv=hkv, group=group, d=d, dtype=dtype)
    ew = enc.device()
    # (tokens per row, lengths to keep afterwards: -1 leaves a row alone)
    plan = [([100, 30, 0, 17], [-1] * 4), ([24, 27, 16, 1], [-1, 50, -1, -1]),
            ([1, 1, 1, 1], [-1] * 4), ([1, 1, 1, 1], [0, -1, -1, 10]), ([60, 1, 40, 90], [-1] * 4),
            ([1, 1, 1, 1], [-1] * 4)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        cache, pages = engine.Kv8Cache(prob), engine.PageTable(prob, 256)
        decode = engine.Kv8Step(prob)
        ref = sv.Pages([0] * rows, [[-1] * width] * rows, range(16, -1, -1), 17, width)
        logic = sv.Cache8(17, hkv, d, dtype)
        for counts, keep in plan:
            say(f"[requests] lens={ref.lens} + {counts}")
            n = sum(counts)
            qkv = torch.from_numpy(rng.standard_normal((n, hkv * (group + 2), d),
                                                       dtype=np.float32)).to(TORCH[dtype])
            dev = qkv.cuda()
            q, k, v = dev.split([hkv * group, hkv, hkv], 1)
            w = pages.take(_i32(counts))
            cache.store(k, v, w["block_table"], w["seq_lens"], w["tok_offsets"])
            one = all(c == 1 for c in counts)
            w.update(q=q.contiguous(), kv8_pool=cache.pool, kv8_scales=cache.scales)
            out, lse = (decode if one else engine.PromptStep(prob, n)).run(w)
            c_out, c_lse = engine.CrossStep(enc.problem(), n).run(
                dict(ew, q=w["q"], tok_offsets=w["tok_offsets"]))
            stream.synchronize()
            before = list(ref.lens)
            _check_take(pages, ref, counts, 256, w)
            at = 0
            for r, m in enumerate(counts):
                got = slice(at, at + m)
                q64 = f64(w["q"][got])
                served = ref.lens[r] == before[r] + m
                p = before[r]
                while served and p < ref.lens[r]:
                    step = min(ref.lens[r], p // 16 * 16 + 16) - p
                    x = np.stack([f64(k[at + p - before[r]:][:step]),
                                  f64(v[at + p - before[r]:][:step])], 1)
                    logic.store(ref.table[r][p // 16], p % 16, x)
                    p += step
                if m and served:
                    kv = np.stack([logic.values(ref.table[r][t // 16], t % 16)
                                   for t in range(ref.lens[r])])
                    want = oc.attend_row(q64, range(before[r], ref.lens[r]), kv[:, 0], kv[:, 1],
                                         prob.sm_scale)
                    check(out[got], lse[got], want, dtype, d, np.abs(kv[:, 1]).max(), not one,
                          f"row {r}")
                elif m:
                    assert not out[got].any() and torch.isneginf(lse[got]).all()
                if m:
                    ek, ev = enc.kv[r]
                    want = sv.cross_row(q64, ek, ev, enc.scale)
                    few = _few(n * group, rows, hkv)
                    check(c_out[got], c_lse[got], want, dtype, d, enc.vmax, not few, f"cross {r}")
                at += m
            pages.release(_i32(keep))
            stream.synchronize()
            ref.release(keep)
            _check_table(pages, ref)
    assert ref.lens[0] == 61 and ref.lens[3] == 11  # row 3's 90 tokens had no pages


def test_offsets_outside_the_arrays():
    """Offsets below zero and behind the last token are taken as the arrays' ends: by
    stores, prompts and cross attention of either kind."""
    lens, new = [40, 25, 60], [10, 5, 12]
    off = _i32([-7, 10, 15, 99])
    say("[offsets outside]")
    b = Batch8(61, lens, new, hkv=2, group=4, everything=True)
    w = dict(b.device(), tok_offsets=off)
    out, lse = engine.PromptStep(b.problem(), 27).run(w)
    torch.cuda.synchronize()
    check(out, lse, b.reference(), "f16", 128, b.vmax, True, "prompt")
    for queries in (new, [1, 2, 3]):
        c = make_cross(8, 62, lens, queries)
        n = sum(queries)
        bad = _i32([-1, queries[0], queries[0] + queries[1], n + 5])
        out, lse = engine.CrossStep(c.problem(), n).run(dict(c.device(), tok_offsets=bad))
        torch.cuda.synchronize()
        check(out, lse, cross_reference(c), "f16", 128, c.vmax, not _takes_few(c), "cross")
    caches = [engine.Kv8Cache(b.problem()) for _ in range(2)]
    kv = torch.randn(27, 2, 2, 128, generator=torch.Generator().manual_seed(3)).half().cuda()
    for cache, o in zip(caches, (off, _offsets(new))):
        cache.store(kv[:, 0], kv[:, 1], w["block_table"], w["seq_lens"], o)
    torch.cuda.synchronize()
    assert _same(caches[0].pool, caches[1].pool) and _same(caches[0].scales, caches[1].scales)


def test_graph_replays():
    """Take, store, decode, cross attention and release captured once, replayed while
    counts, queries and tokens change on the device, with eager work of the same kind
    between."""
    b = Batch8(13, [200, 90, 33], hkv=2, group=4)
    enc = make_cross(16, 14, [300, 0, 70], [1, 1, 1])
    ew = enc.device()
    prob = engine.make_problem(3, 8, 2, 128, 16, 60, 20, "f16")
    rng = np.random.default_rng(3)
    kv = torch.zeros(3, 2, 2, 128, dtype=torch.float16, device="cuda")
    q = torch.zeros(3, 8, 128, dtype=torch.float16, device="cuda")
    counts, keep = _i32([1, 1, 1]), _i32([-1, -1, -1])

    def build():
        cache, pages = engine.Kv8Cache(prob), engine.PageTable(prob, 3)
        step, cross = engine.Kv8Step(prob), engine.CrossStep(enc.problem(), 3)

        def run():
            pages.release(keep)
            w = pages.take(counts)
            cache.store(kv[:, 0], kv[:, 1], w["block_table"], w["seq_lens"], w["tok_offsets"])
            step.run(dict(w, q=q, kv8_pool=cache.pool, kv8_scales=cache.scales))
            cross.run(dict(ew, q=q, tok_offsets=w["tok_offsets"]))
            return (step.out, step.lse, cross.out, cross.lse, cache.pool, cache.scales, pages.lens,
                    pages.slots, pages.state, pages.block_table)
        return run
    captured, eager = build(), build()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured()
    torch.cuda.current_stream().wait_stream(side)
    eager()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = captured()
    for i in range(24):
        counts.copy_(_i32([1, i % 2, 1]))
        keep.copy_(_i32([-1, -1, 5 if i == 9 else 0 if i == 15 else -1]))
        q.copy_(torch.from_numpy(rng.standard_normal(tuple(q.shape), dtype=np.float32)))
        kv.copy_(torch.from_numpy(rng.standard_normal(tuple(kv.shape), dtype=np.float32) * (i + 1)))
        graph.replay()
        torch.cuda.synchronize()
        want = eager()
        torch.cuda.synchronize()
        if i % 6 == 0:
            say(f"[graph] replay {i} lens={got[6].tolist()}")
        assert all(_same(x, y) for x, y in zip(got, want)), i
    assert got[6].tolist()[0] == 25


def test_two_streams_with_their_own_steps():
    """Steps with workspaces of their own run at once on two streams."""
    a, b = (make_cross(8, s, [900, 450, 77], [2, 3, 1]) for s in (1, 2))
    say("[two streams]")
    pairs = [(x, x.device(), engine.CrossStep(x.problem(), 6, 16), torch.cuda.Stream())
             for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, step, stream in pairs:
            step.run(w, stream)
    torch.cuda.synchronize()
    for x, w, step, stream in pairs:
        check(step.out, step.lse, cross_reference(x), "f16", 128, x.vmax, False, "stream")


def _busy(stream, ms=60):
    """Keep `stream` at work for a while: passes over 1 GiB of its own."""
    with torch.cuda.stream(stream):
        x = torch.zeros(1 << 28, dtype=torch.float32, device="cuda")
        for _ in range(2 * ms):
            x.add_(1)


@pytest.mark.parametrize("kind", ["cross", "table", "cache"])
def test_built_on_a_busy_stream_runs_on_another(kind):
    """What an object fills is there before its first call on any stream."""
    building, running = torch.cuda.Stream(), torch.cuda.Stream()
    b = make_cross(8, 51, [900, 450, 77], [2, 1, 1])
    w = b.device()
    kv = torch.randn(4, 2, 128, generator=torch.Generator().manual_seed(0)).half().cuda()
    counts = _i32([2, 1, 1])
    torch.cuda.synchronize()
    say(f"[built elsewhere] {kind}")
    with torch.cuda.stream(building):
        junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        del junk
        _busy(building)
        x = (engine.CrossStep(b.problem(), 4, 16) if kind == "cross" else
             engine.PageTable(b.problem(), 4) if kind == "table" else engine.Kv8Cache(b.problem()))
    if kind == "cross":
        out, lse = x.run(w, running)
    elif kind == "table":
        got = x.take(counts, running)
    else:
        x.store(kv, kv, w["block_table"], w["seq_lens"], w["tok_offsets"], running)
    running.synchronize()
    building.synchronize()
    if kind == "cross":
        check(out, lse, cross_reference(b), "f16", 128, b.vmax, False, kind)
    elif kind == "table":
        assert got["seq_lens"].tolist() == [2, 1, 1] and x.lens.tolist() == [2, 1, 1]
    else:
        k = x.load(w["block_table"], w["seq_lens"], w["tok_offsets"], torch.empty_like(kv),
                   torch.empty_like(kv))[0]
        assert ((k - kv).abs().float() <= kv.abs().float() / 16 + 2.0 ** -16).all()


def test_refusals_on_the_device():
    b = Batch8(1, [20, 30])
    prob, w = b.problem(), b.device()
    step = engine.Kv8Step(prob)
    with pytest.raises(ValueError, match="kv8_scales"):
        step.run(dict(w, kv8_scales=w["kv8_scales"][:-1]))
    with pytest.raises(ValueError, match="kv8_pool"):
        step.run(dict(w, kv8_pool=w["kv8_pool"].view(torch.int8)))
    with pytest.raises(ValueError, match="wrong kind"):
        engine.WindowStep(prob).run(w)
    with pytest.raises(ValueError, match="wrong kind"):
        engine.Kv4Step(prob).run(w)
    with pytest.raises(ValueError, match="tok_offsets"):
        engine.CrossStep(prob, 5).run(dict(w, q=w["q"].repeat(3, 1, 1)[:5], tok_offsets=None))
    with pytest.raises(ValueError, match="q"):
        engine.CrossStep(prob, 2).run(dict(w, q=w["q"].float()))
    with pytest.raises(_lib.PkvError):
        engine.Kv8Step(prob, window=-1, splits=1).run(w)
    cross = engine.CrossStep(prob, 2, splits=2)
    with pytest.raises(_lib.PkvError):
        _serving.pkv_cross_kv8(prob, w["tok_offsets"], 2, w["seq_lens"], 2, w["q"], w["kv8_pool"],
                               w["kv8_scales"], w["block_table"], cross.workspace[:16], cross.out)
    _serving.pkv_cross_kv8(prob, w["tok_offsets"], 2, w["seq_lens"], 1, w["q"], w["kv8_pool"],
                           w["kv8_scales"], w["block_table"], None, cross.out)
    torch.cuda.synchronize()
