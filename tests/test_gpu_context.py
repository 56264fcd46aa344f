"""GPU: windowed and prompt attention and the 4-bit cache, through the engine
and the C ABI, against the fp64 oracle; poison everywhere no query looks.
Tolerances are derived in tests/context_cases.py."""
import numpy as np
import pytest
import torch

from oracle import context as oc
from paged_kv_gqa_block_amd import _context, _lib, engine
from tests.context_cases import TORCH, Batch, check, f64
from tests.parity import say

pytestmark = pytest.mark.gpu

LENS = [0, 1, 15, 16, 17, 33, 100, 250, 700]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"


def _step(b, splits=None):
    cls = engine.Kv4Step if b.kv4 else engine.WindowStep
    return cls(b.problem(), b.window, b.sinks, splits)


def _same(a, b):
    view = {2: torch.int16, 4: torch.int32, 1: torch.uint8}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


# ---- the 4-bit cache ---------------------------------------------------------------

def _special_tokens(n, hkv, d, dtype, seed):
    """Values of every size, ties, signed zeros, infinities and NaN."""
    rng = np.random.default_rng(seed)
    lo, hi = (-22, 14) if dtype == "f16" else (-126, 126)
    x = rng.standard_normal((n, hkv, d)) * 2.0 ** rng.integers(lo, hi, (n, hkv, d // 32)).repeat(32, -1)
    kind = rng.integers(0, 12, (n, hkv, d // 32)).repeat(32, -1)
    grid = rng.choice([0, .25, .5, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 6.5, 7, -0.0, -.25, -5],
                      (n, hkv, d))
    x = np.where(kind == 0, 0.0, x)
    x = np.where(kind == 1, grid, x)
    x = np.where(kind == 2, grid * 2.0 ** (lo + 1), x)
    x = np.where((kind == 3) & (rng.random(x.shape) < 0.1), np.inf, x)
    x = np.where((kind == 4) & (rng.random(x.shape) < 0.1), np.nan, x)
    x = np.where(kind == 5, np.where(rng.random(x.shape) < 0.5, 1, -1) * (65504.0 if dtype == "f16"
                                                                        else 3.3895e38), x)
    with np.errstate(over="ignore"):
        return torch.from_numpy(x.astype(np.float32)).to(TORCH[dtype])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d,hkv,lens,new", [
    (128, 2, [5, 0, 33, 16, 64, 17], [5, 0, 20, 1, 64, 3]),
    (64, 3, [1, 40, 15, 100], [1, 17, 15, 49]),
    (128, 1, [200], [200]),
    (64, 8, [16, 31, 32], None),
])
def test_kv4_store_writes_the_oracle_bytes_and_load_reads_them(d, hkv, lens, new, dtype):
    say(f"[kv4 store/load] d={d} Hkv={hkv} {dtype} lens={lens} new={new}")
    counts = [1] * len(lens) if new is None else new
    rng = np.random.default_rng(d + hkv)
    width = max(-(-n // 16) for n in lens) + 2
    pool_pages = len(lens) * width + 3
    table = rng.permutation(pool_pages)[:len(lens) * width].reshape(len(lens), width).astype(np.int32)
    n = sum(counts)
    kv = _special_tokens(n, 2 * hkv, d, dtype, 7).view(n, 2, hkv, d)  # a fused projection's rows
    before = rng.integers(0, 256, (pool_pages, hkv, 17 * d)).astype(np.uint8)
    prob = engine.make_problem(len(lens), 4 * hkv, hkv, d, 16, pool_pages, width, dtype)
    cache = engine.Kv4Cache(prob, pool=torch.from_numpy(before.copy()).cuda())
    dev = kv.cuda()
    bt, sl = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    off = None if new is None else torch.from_numpy(
        np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    cache.store(dev[:, 0], dev[:, 1], bt, sl, off)
    out = [torch.full((n, hkv, d), 7.0, dtype=TORCH[dtype], device="cuda") for _ in range(2)]
    cache.load(bt, sl, off, *out)
    torch.cuda.synchronize()
    want = before.copy()
    values = np.zeros((n, 2, hkv, d))
    at = 0
    for row, (length, m) in enumerate(zip(lens, counts)):
        for p in range(length - m, length):
            for x, which in enumerate("kv"):
                codes, scales = oc.kv4_quantise(f64(kv[at, x]), dtype)
                values[at, x] = oc.kv4_values(codes, scales)
                for h in range(hkv):
                    oc.kv4_write(want[table[row, p // 16], h], p % 16, codes[h], scales[h], which)
            at += 1
    np.testing.assert_array_equal(cache.pool.cpu().numpy(), want)
    for x in range(2):
        np.testing.assert_array_equal(f64(out[x]), values[:, x])  # NaN where NaN


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_kv4_every_finite_value_quantises_like_the_oracle(dtype):
    """All finite 16-bit values, once alone in their block (its maximum) and
    once beside a maximum of every exponent."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(TORCH[dtype])
    x = x[torch.isfinite(x)]
    rng = np.random.default_rng(2)
    blocks = torch.zeros(2 * x.numel(), 32, dtype=TORCH[dtype])
    blocks[:x.numel(), 5] = x
    blocks[x.numel():, 9] = x
    blocks[x.numel():, 30] = x[torch.from_numpy(rng.permutation(x.numel()))]
    n = -(-blocks.shape[0] // 4)
    kv = torch.zeros(n * 4, 32, dtype=TORCH[dtype])
    kv[:blocks.shape[0]] = blocks
    kv = kv.view(n, 1, 128)
    width = -(-n // 16)
    prob = engine.make_problem(1, 1, 1, 128, 16, width, width, dtype)
    cache = engine.Kv4Cache(prob)
    bt = torch.arange(width, dtype=torch.int32).view(1, -1).cuda()
    sl = torch.tensor([n], dtype=torch.int32).cuda()
    off = torch.tensor([0, n], dtype=torch.int32).cuda()
    cache.store(kv.cuda(), kv.cuda(), bt, sl, off)
    k, v = (torch.empty(n, 1, 128, dtype=TORCH[dtype], device="cuda") for _ in range(2))
    cache.load(bt, sl, off, k, v)
    torch.cuda.synchronize()
    codes, scales = oc.kv4_quantise(f64(kv.view(-1, 128)), dtype)
    want = oc.kv4_values(codes, scales)
    np.testing.assert_array_equal(f64(k).reshape(-1, 128), want)
    np.testing.assert_array_equal(f64(v).reshape(-1, 128), want)


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
    for kv4 in (True, False):
        say(f"[store skips] kv4={kv4}")
        prob = engine.make_problem(5, 4, hkv, d, 16, pages, width, "f16")
        x = torch.randn(n, hkv, d, generator=torch.Generator().manual_seed(0)).half().cuda()
        bt, sl = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        off = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        if kv4:
            cache = engine.Kv4Cache(prob)
            cache.pool.fill_(99)
            cache.store(x, x, bt, sl, off)
        else:
            kp = torch.full((pages, hkv, 16, d), 9.0, device="cuda").half()
            vp = kp.clone()
            engine.store_kv(prob, x, x, bt, sl, off, kp, vp)
        torch.cuda.synchronize()
        written = {}
        at = 0
        for row in range(5):
            for i in range(new[row]):
                p = lens[row] - new[row] + i
                if 0 <= lens[row] <= width * 16 and p >= 0 and 0 <= table[row, p // 16] < pages:
                    written[table[row, p // 16], p % 16] = at
                at += 1
        if kv4:
            got = [torch.full_like(x, 5.0) for _ in range(2)]
            cache.load(bt, sl, off, *got)
            back = set(written.values())
            for tok in range(n):
                untouched = bool((got[0][tok] == 5).all()) and bool((got[1][tok] == 5).all())
                assert untouched == (tok not in back), tok
            pool = cache.pool.cpu().numpy()
            for pg in range(pages):
                if not any(k[0] == pg for k in written):
                    assert (pool[pg] == 99).all(), pg
        else:
            for pg in range(pages):
                for slot in range(16):
                    tok = written.get((pg, slot))
                    want = torch.full_like(x[0], 9.0) if tok is None else x[tok]
                    assert torch.equal(kp[pg, :, slot], want) and torch.equal(vp[pg, :, slot], want)


# ---- decode steps --------------------------------------------------------------------

VIEWS = [(0, 0), (1, 0), (1, 1), (15, 4), (16, 16), (17, 40), (100, 5), (250, 0), (10 ** 6, 3),
         (64, 10 ** 6), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("d,dtype", [(128, "f16"), (128, "bf16"), (64, "f16"), (64, "bf16")])
@pytest.mark.parametrize("window,sinks", VIEWS)
def test_decode_view(window, sinks, d, dtype, kv4):
    seed = VIEWS.index((window, sinks))
    group, hkv = [(4, 2), (1, 3), (8, 1), (16, 1), (5, 2), (2, 8), (3, 1)][seed % 7]
    b = Batch(seed, LENS, hkv=hkv, group=group, d=d, dtype=dtype, window=window, sinks=sinks,
              kv4=kv4)
    ref = b.reference()
    w = b.device()
    for splits in (None, 1, 3, 100):
        say(f"[decode view] W={window} S={sinks} d={d} {dtype} kv4={kv4} G={group} Hkv={hkv} "
            f"splits={splits}")
        step = _step(b, splits)
        out, lse = step.run(w)
        torch.cuda.synchronize()
        check(out, lse, ref, dtype, d, b.vmax, False, f"splits {splits}")
        first = out.clone()
        step.run(w)
        torch.cuda.synchronize()
        assert _same(first, step.out)  # the workspace carries nothing over


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("group,hkv", [(1, 1), (2, 1), (3, 2), (6, 1), (7, 1), (9, 1), (13, 2), (16, 2)])
def test_decode_head_groups(group, hkv, kv4):
    for d in (64, 128):
        say(f"[groups] G={group} Hkv={hkv} d={d} kv4={kv4}")
        b = Batch(group, [37, 600, 0, 129], hkv=hkv, group=group, d=d, window=90, sinks=3, kv4=kv4)
        out, lse = _step(b).run(b.device())
        torch.cuda.synchronize()
        check(out, lse, b.reference(), "f16", d, b.vmax, False, "groups")


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_scales(kv4):
    """A negative scale, zero, and scores far apart."""
    for scale, spread in ((-0.2, 1.0), (0.0, 1.0), (1.0, 3.0), (1e-30, 1.0)):
        say(f"[scale] {scale} kv4={kv4}")
        b = Batch(5, [70, 300], scale=scale, spread=spread, kv4=kv4, dtype="bf16")
        out, lse = _step(b).run(b.device())
        torch.cuda.synchronize()
        check(out, lse, b.reference(), "bf16", 128, b.vmax, False, f"scale {scale}")


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_bad_rows_and_pages(kv4):
    """A length outside the table makes the row empty; a page outside the pool
    holds no tokens, also where it is all that a row has."""
    b = Batch(3, [100, 50, 20, 33, 16], kv4=kv4, window=60, sinks=2)
    pool = (b.pool4 if kv4 else b.kp).shape[0]
    cap = b.table.shape[1] * 16
    w = b.device()
    w["seq_lens"] = torch.tensor([100, -3, cap + 1, 33, 16], dtype=torch.int32).cuda()
    bt = b.table.copy()
    bt[0, 4], bt[3, 0], bt[4, 0] = -1, pool, 2 ** 31 - 1
    w["block_table"] = torch.from_numpy(bt).cuda()
    ref = b.reference(lens=[100, 0, 0, 33, 16],
                      present=lambda r, pg: 0 <= bt[r, pg] < pool)
    for splits in (1, 4):
        say(f"[bad pages] kv4={kv4} splits={splits}")
        out, lse = _step(b, splits).run(w)
        torch.cuda.synchronize()
        check(out, lse, ref, "f16", 128, b.vmax, False, "bad pages")
    assert not out[1].any() and not out[4].any()


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_long_row_many_splits(kv4):
    b = Batch(8, [20011, 17], hkv=1, group=4, dtype="bf16", kv4=kv4)
    ref = b.reference()
    w = b.device()
    for splits in (None, 2, 500):
        say(f"[long row] kv4={kv4} splits={splits}")
        out, lse = _step(b, splits).run(w)
        torch.cuda.synchronize()
        check(out, lse, ref, "bf16", 128, b.vmax, False, "long")


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_many_rows(kv4):
    """More rows than a wave has lanes, lengths 0..40."""
    b = Batch(9, np.random.default_rng(1).integers(0, 41, 150), hkv=1, group=2, d=64, kv4=kv4,
              window=20, sinks=1)
    ref = b.reference()
    for splits in (1, 2):
        say(f"[many rows] kv4={kv4} splits={splits}")
        out, lse = _step(b, splits).run(b.device())
        torch.cuda.synchronize()
        check(out, lse, ref, "f16", 64, b.vmax, False, "many rows")


def test_window_zero_agrees_with_the_engine_step():
    """Without a window the step computes what the self-planned step does."""
    b = Batch(4, [500, 3, 0, 129], hkv=2, group=4)
    w = b.device()
    out, lse = _step(b).run(w)
    other = engine.SelfPlannedStep(b.problem(), 4)
    other.run(w)
    torch.cuda.synchronize()
    assert (out.float() - other.out.float()).abs().max() <= 2e-3
    torch.testing.assert_close(lse, other.lse, rtol=0, atol=4e-4)


# ---- prompts ---------------------------------------------------------------------------

RUNS = [
    ([1], [1]),
    ([70], [70]),
    ([300, 0, 17, 45, 200], [300, 0, 1, 20, 7]),
    ([129, 64, 65, 16, 15], [129, 64, 65, 16, 15]),
    ([400, 600], [3, 150]),
]


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("d,dtype", [(128, "f16"), (128, "bf16"), (64, "f16"), (64, "bf16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (16, 4), (50, 33), (64, 0),
                                          (190, 17), (10 ** 6, 0)])
@pytest.mark.parametrize("run", range(len(RUNS)))
def test_prompt(run, window, sinks, d, dtype, kv4):
    lens, new = RUNS[run]
    group, hkv = [(4, 2), (1, 1), (8, 1), (5, 1), (16, 1)][(run + window) % 5]
    say(f"[prompt] lens={lens} new={new} W={window} S={sinks} d={d} {dtype} kv4={kv4} G={group} "
        f"Hkv={hkv}")
    b = Batch(run, lens, new, hkv=hkv, group=group, d=d, dtype=dtype, window=window, sinks=sinks,
              kv4=kv4)
    step = engine.PromptStep(b.problem(), int(b.new.sum()), window, sinks)
    out, lse = step.run(b.device())
    torch.cuda.synchronize()
    check(out, lse, b.reference(), dtype, d, b.vmax, True, "prompt")


def test_prompt_scales():
    for scale in (-0.3, 0.0, 1.0):
        say(f"[prompt scale] {scale}")
        b = Batch(2, [90, 40], [90, 10], scale=scale, dtype="bf16", spread=2.0)
        out, lse = engine.PromptStep(b.problem(), 100).run(b.device())
        torch.cuda.synchronize()
        check(out, lse, b.reference(), "bf16", 128, b.vmax, True, f"scale {scale}")


def test_prompt_one_token_per_row_without_offsets():
    b = Batch(6, LENS, window=40, sinks=2, group=8, hkv=2)
    w = b.device()
    del w["tok_offsets"]
    say("[prompt, no offsets]")
    out, lse = engine.PromptStep(b.problem(), len(LENS), 40, 2).run(w)
    torch.cuda.synchronize()
    check(out, lse, b.reference(), "f16", 128, b.vmax, True, "no offsets")


@pytest.mark.parametrize("kv4", [False, True])
def test_prompt_queries_outside_the_row_and_rows_behind_the_last(kv4):
    """Runs longer than their rows, invalid lengths, pages outside the pool;
    output rows behind the last offset stay as they were."""
    b = Batch(7, [30, 60, 20, 50], [45, 60, 5, 9], kv4=kv4, window=25, sinks=1, dtype="bf16")
    pool = (b.pool4 if kv4 else b.kp).shape[0]
    bt = b.table.copy()
    bt[1, 1], bt[3, 3] = -7, pool
    w = b.device()
    w["block_table"] = torch.from_numpy(bt).cuda()
    w["seq_lens"] = torch.tensor([30, 60, 10 ** 9, 50], dtype=torch.int32).cuda()
    ref = b.reference(lens=[30, 60, 0, 50], present=lambda r, pg: 0 <= bt[r, pg] < pool)
    n = int(b.new.sum())
    w["q"] = torch.cat([w["q"], torch.zeros_like(w["q"][:3])])
    step = engine.PromptStep(b.problem(), n + 3, 25, 1)
    step.out.fill_(3.0)
    step.lse.fill_(3.0)
    say(f"[prompt outside] kv4={kv4}")
    out, lse = step.run(w)
    torch.cuda.synchronize()
    check(out[:n], lse[:n], ref, "bf16", 128, b.vmax, True, "outside")
    assert (out[n:] == 3).all() and (lse[n:] == 3).all()


# ---- together, as they are used -----------------------------------------------------------

@pytest.mark.parametrize("kv4", [False, True])
def test_prompt_then_decode(kv4):
    """Two prompt chunks, then decode steps: store, attend, every call on a
    side stream, every output against the oracle over the cache's values."""
    rng = np.random.default_rng(11)
    hkv, group, d, dtype, window, sinks = 2, 4, 128, "f16", 48, 4
    final = [130, 61, 20]
    plan = [[100, 30, 0], [24, 27, 16]] + [[1, 1, 1]] * 4
    width = 10
    table = rng.permutation(40)[:3 * width].reshape(3, width).astype(np.int32)
    prob = engine.make_problem(3, hkv * group, hkv, d, 16, 40, width, dtype)
    bt = torch.from_numpy(table).cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        cache = engine.Kv4Cache(prob) if kv4 else None
        pools = {"kv4_pool": cache.pool} if kv4 else {
            n: torch.zeros(40, hkv, 16, d, dtype=TORCH[dtype], device="cuda")
            for n in ("k_pool", "v_pool")}
        decode = (engine.Kv4Step if kv4 else engine.WindowStep)(prob, window, sinks)
        lens = np.zeros(3, dtype=np.int64)
        history = [[np.zeros((0, hkv, d))] * 2 for _ in range(3)]
        for new in plan:
            say(f"[flow] kv4={kv4} lens={lens.tolist()} + {new}")
            n = sum(new)
            qkv = torch.from_numpy(rng.standard_normal((n, hkv * (group + 2), d),
                                                       dtype=np.float32)).to(TORCH[dtype])
            lens += new
            off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            dev = qkv.cuda()
            q, k, v = dev.split([hkv * group, hkv, hkv], 1)  # a fused projection's output
            sl, to = torch.from_numpy(lens.astype(np.int32)).cuda(), torch.from_numpy(off).cuda()
            one = all(m == 1 for m in new)
            if kv4:
                cache.store(k, v, bt, sl, None if one else to)
            else:
                engine.store_kv(prob, k, v, bt, sl, None if one else to, pools["k_pool"],
                                pools["v_pool"])
            w = dict(pools, q=q.contiguous(), block_table=bt, seq_lens=sl, tok_offsets=to)
            out, lse = (decode if one else engine.PromptStep(prob, n, window, sinks)).run(w)
            stream.synchronize()
            at = 0
            for r, m in enumerate(new):
                for x, t in enumerate((k, v)):
                    val = f64(t[at:at + m])
                    if kv4 and m:
                        val = oc.kv4_values(*oc.kv4_quantise(val, dtype))
                    history[r][x] = np.concatenate([history[r][x], val])
                kk, vv = history[r]
                if m:
                    ref = oc.attend_row(f64(q[at:at + m]), range(lens[r] - m, lens[r]), kk, vv,
                                        prob.sm_scale, window, sinks)
                    check(out[at:at + m], lse[at:at + m], ref, dtype, d, np.abs(vv).max(),
                          not one, f"row {r}")
                at += m
    assert lens.tolist() == [128, 61, 20] and final[1:] == lens.tolist()[1:]


@pytest.mark.parametrize("kv4", [False, True])
def test_graph_replays(kv4):
    """Store and decode captured once, replayed while lengths, queries and new
    tokens change on the device, with eager work of the same step between."""
    b = Batch(13, [200, 90, 33], hkv=2, group=4, kv4=kv4, window=70, sinks=3)
    prob, w = b.problem(), b.device()
    step, eager = _step(b), _step(b)
    rng = np.random.default_rng(3)
    kv = torch.zeros(3, 2, 2, 128, dtype=torch.float16, device="cuda")
    cache = engine.Kv4Cache(prob, pool=w["kv4_pool"]) if kv4 else None

    def store():
        if kv4:
            cache.store(kv[:, 0], kv[:, 1], w["block_table"], w["seq_lens"])
        else:
            engine.store_kv(prob, kv[:, 0], kv[:, 1], w["block_table"], w["seq_lens"], None,
                            w["k_pool"], w["v_pool"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        store()
        step.run(w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        store()
        step.run(w)
    for i in range(4):
        say(f"[graph] kv4={kv4} replay {i}")
        w["seq_lens"].copy_(torch.tensor([200 + i, 90 - 7 * i, 33 + i], dtype=torch.int32))
        w["q"].copy_(torch.from_numpy(rng.standard_normal(tuple(w["q"].shape), dtype=np.float32)))
        kv.copy_(torch.from_numpy(rng.standard_normal(tuple(kv.shape), dtype=np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        got = step.out.clone(), step.lse.clone()
        store()
        eager.run(w)
        torch.cuda.synchronize()
        assert _same(got[0], eager.out) and _same(got[1], eager.lse)


def test_two_streams_with_their_own_steps():
    """Two steps with workspaces of their own run at once on two streams."""
    a, b = (Batch(s, [900, 450, 77], hkv=2, group=4, window=300, sinks=4) for s in (1, 2))
    say("[two streams]")
    pairs = [(x, x.device(), _step(x, 16), torch.cuda.Stream()) for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, step, stream in pairs:
            step.run(w, stream)
    torch.cuda.synchronize()
    for x, w, step, stream in pairs:
        check(step.out, step.lse, x.reference(), "f16", 128, x.vmax, False, "stream")


def test_refusals_on_the_device():
    b = Batch(1, [20, 30])
    prob, w = b.problem(), b.device()
    step = _step(b)
    with pytest.raises(ValueError, match="q"):
        step.run(dict(w, q=w["q"].float()))
    with pytest.raises(ValueError, match="block_table"):
        step.run(dict(w, block_table=w["block_table"][:, :-1]))
    with pytest.raises(ValueError, match="cpu"):
        step.run(dict(w, seq_lens=w["seq_lens"].cpu()))
    with pytest.raises(ValueError, match="wrong kind"):
        engine.Kv4Step(prob).run(w)
    with pytest.raises(ValueError, match="tok_offsets"):
        engine.PromptStep(prob, 5).run(dict(w, q=w["q"].repeat(3, 1, 1)[:5], tok_offsets=None))
    with pytest.raises(_lib.PkvError):
        _context.pkv_attend_window(prob, step.view, w["seq_lens"], step.splits, w["q"],
                                   w["k_pool"], w["v_pool"], w["block_table"],
                                   step.workspace[:16], step.out)
    with pytest.raises(_lib.PkvError):
        engine.WindowStep(prob, window=-1).run(w)
    with pytest.raises(_lib.PkvError):
        engine.store_kv(prob, torch.zeros(2, 2, 132, dtype=torch.float16,
                                          device="cuda").as_strided((2, 2, 128), (260, 128, 1)),
                        torch.zeros(2, 2, 128, dtype=torch.float16, device="cuda"),
                        w["block_table"], w["seq_lens"], None, w["k_pool"], w["v_pool"])


# ---- larger sizes, shared buffers -----------------------------------------------------------

@pytest.mark.parametrize("rows", [63, 64, 65, 130])
def test_runs_of_many_rows(rows):
    """Rows around and beyond what a wave holds, some without new tokens: the
    prompt, the store and the read-back find every token's row."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, 40, rows)
    new = np.minimum(lens, rng.integers(0, 20, rows))
    new[rng.random(rows) < 0.3] = 0
    say(f"[many runs] rows={rows} tokens={new.sum()}")
    b = Batch(rows, lens, new, hkv=1, group=3, d=64, window=15, sinks=2, kv4=True)
    w = b.device()
    n = int(new.sum())
    out, lse = engine.PromptStep(b.problem(), n, 15, 2).run(w)
    torch.cuda.synchronize()
    check(out, lse, b.reference(), "f16", 64, b.vmax, True, "many runs")
    cache = engine.Kv4Cache(b.problem())
    x = torch.from_numpy(rng.standard_normal((n, 1, 64), dtype=np.float32)).half().cuda()
    cache.store(x, -x, w["block_table"], w["seq_lens"], w["tok_offsets"])
    k, v = torch.empty_like(x), torch.empty_like(x)
    cache.load(w["block_table"], w["seq_lens"], w["tok_offsets"], k, v)
    torch.cuda.synchronize()
    want = oc.kv4_values(*oc.kv4_quantise(f64(x), "f16"))
    np.testing.assert_array_equal(f64(k), want)
    np.testing.assert_array_equal(f64(v), -want)


@pytest.mark.parametrize("kv4", [False, True])
def test_pages_beyond_4_gib(kv4):
    """The same rows in a small pool and at the far end of a pool whose byte
    offsets pass 2^32: every call gives the same bits."""
    b = Batch(21, [300, 77], [40, 77], hkv=8, group=2, window=100, sinks=3, kv4=kv4, dtype="bf16")
    w = b.device()
    small = (w["kv4_pool"] if kv4 else w["k_pool"]).shape[0]
    page_bytes = 8 * (17 * 128 if kv4 else 16 * 128 * 2)
    big = (1 << 32) // page_bytes + 1000
    shift = big - small
    prob = b.problem(num_pool_pages=big)
    far = dict(w, block_table=w["block_table"] + shift)
    say(f"[far pages] kv4={kv4} pages={big}")
    for name in ("kv4_pool",) if kv4 else ("k_pool", "v_pool"):
        far[name] = torch.zeros(big, *w[name].shape[1:], dtype=w[name].dtype, device="cuda")
        far[name][shift:] = w[name]
    n = int(b.new.sum())
    qd = {"q": w["q"][:2].contiguous()}
    outs = []
    for pr, x in ((b.problem(), w), (prob, far)):
        got = [t.clone() for t in engine.PromptStep(pr, n, 100, 3).run(x)]
        cls = engine.Kv4Step if kv4 else engine.WindowStep
        got += [t.clone() for t in cls(pr, 100, 3).run(dict(x, **qd))]
        kv = torch.linspace(-3, 3, n * 8 * 128, device="cuda").to(torch.bfloat16).view(n, 8, 128)
        args = (x["block_table"], x["seq_lens"], x["tok_offsets"])
        if kv4:
            cache = engine.Kv4Cache(pr, pool=x["kv4_pool"])
            cache.store(kv, kv, *args)
            got += list(cache.load(*args, torch.empty_like(kv), torch.empty_like(kv)))
            got.append(x["kv4_pool"][-small:].clone())
        else:
            engine.store_kv(pr, kv, kv, *args, x["k_pool"], x["v_pool"])
            got += [x["k_pool"][-small:].clone(), x["v_pool"][-small:].clone()]
        torch.cuda.synchronize()
        outs.append(got)
    for a, c in zip(*outs):
        assert _same(a, c)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40])
def test_prompt_splits(splits):
    """Few queries over long contexts, the keys cut into ranges; twice on one
    workspace, with the same bits."""
    for kv4, d, dtype in ((False, 128, "bf16"), (False, 64, "f16"), (True, 128, "f16")):
        say(f"[prompt splits] {splits} kv4={kv4} d={d} {dtype}")
        b = Batch(splits, [1500, 0, 70, 900], [3, 0, 70, 33], hkv=2, group=4, d=d, dtype=dtype,
                  kv4=kv4, window=1200, sinks=20)
        step = engine.PromptStep(b.problem(), int(b.new.sum()), 1200, 20, splits)
        w = b.device()
        out, lse = step.run(w)
        torch.cuda.synchronize()
        check(out, lse, b.reference(), dtype, d, b.vmax, True, f"splits {splits}")
        first = out.clone(), lse.clone()
        step.run(w)
        torch.cuda.synchronize()
        assert _same(first[0], step.out) and _same(first[1], step.lse)


def test_two_graphs_of_one_step_replayed_in_turn():
    """Two captured graphs that share a step's workspace, one after the other."""
    b = Batch(17, [900, 450], hkv=2, group=4, window=0)
    step, w = _step(b, 16), b.device()
    other = dict(w, q=torch.randn_like(w["q"]))
    outs = [step.run(x)[0].clone() for x in (w, other)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run(w)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for x in (w, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step.run(x)
        graphs.append(g)
    for i in range(6):
        say(f"[two graphs] replay {i}")
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert _same(step.out, outs[i % 2])


def test_bound_calls_follow_their_buffers():
    b = Batch(18, [200, 33], window=50, sinks=2)
    step, w = _step(b), b.device()
    bound = step.bind(w)
    first = step.run_bound(bound)[0].clone()
    w["q"].mul_(-1)
    second = step.run_bound(bound)[0].clone()
    w["q"].mul_(-1)
    third = step.run_bound(bound)[0].clone()
    torch.cuda.synchronize()
    assert _same(first, third) and not _same(first, second)


def test_no_new_tokens_at_all():
    b = Batch(19, [20, 5], [0, 0], kv4=True)
    w, prob = b.device(), b.problem()
    empty = torch.empty(0, 2, 128, dtype=torch.float16, device="cuda")
    cache = engine.Kv4Cache(prob, pool=w["kv4_pool"])
    before = cache.pool.clone()
    args = (w["block_table"], w["seq_lens"], w["tok_offsets"])
    cache.store(empty, empty, *args)
    cache.load(*args, empty, empty.clone())
    out, lse = engine.PromptStep(prob, 0).run(dict(w, q=w["q"]))
    torch.cuda.synchronize()
    assert _same(before, cache.pool) and out.numel() == 0 and lse.numel() == 0


def test_unordered_offsets_stay_in_bounds():
    """Offsets that break the contract (decreasing, negative, beyond the token
    count) give rows that nobody promised, but touch nothing outside the
    buffers: guard rows around them keep their values."""
    b = Batch(20, [40, 40, 40, 40], [10, 10, 10, 10], kv4=True)
    w, prob = b.device(), b.problem()
    n = 40
    out = torch.full((n + 20, 8, 128), 5.0, dtype=torch.float16, device="cuda")
    kv = torch.ones(n, 2, 128, dtype=torch.float16, device="cuda")
    outs = [torch.full((n + 20, 2, 128), 5.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    cache = engine.Kv4Cache(prob, pool=w["kv4_pool"])
    for off in ([0, 30, 10, 35, 40], [-5, 10, 20, 90, 40], [40, 30, 20, 10, 0],
                [0, 2 ** 31 - 1, -2 ** 31, 7, 40]):
        say(f"[offsets] {off}")
        to = torch.tensor(off, dtype=torch.int32, device="cuda")
        _context.pkv_prompt_kv4(prob, None, to, n, w["seq_lens"], 1, w["q"], w["kv4_pool"],
                                w["block_table"], None, out[10:10 + n])
        _context.pkv_kv4_load(prob, to, n, w["seq_lens"], w["block_table"], w["kv4_pool"],
                              outs[0][10:10 + n], outs[1][10:10 + n])
        cache.store(kv, kv, w["block_table"], w["seq_lens"], to)
        torch.cuda.synchronize()
        for t in (out, *outs):
            assert (t[:10] == 5).all() and (t[10 + n:] == 5).all()


def test_one_workspace_for_problems_of_all_sizes():
    """Calls of different batches, splits and kinds use one workspace in turn,
    each finding its counters at zero."""
    shapes = [dict(lens=[900, 33], splits=40, hkv=2), dict(lens=[100] * 60, splits=3, hkv=8),
              dict(lens=[700], splits=100, hkv=1), dict(lens=[90, 300], new=[90, 40], splits=4, hkv=3)]
    steps = []
    for i, s in enumerate(shapes):
        b = Batch(i, s["lens"], s.get("new"), hkv=s["hkv"], group=2, d=64)
        step = (engine.PromptStep(b.problem(), int(b.new.sum()), 0, 0, s["splits"])
                if "new" in s else _step(b, s["splits"]))
        steps.append((b, step, b.device(), "new" in s))
    shared = torch.zeros(max(s.workspace.numel() for _, s, _, _ in steps), dtype=torch.uint8,
                         device="cuda")
    for _ in range(2):
        for b, step, w, many in steps + steps[::-1]:
            say(f"[shared workspace] B={len(b.lens)} Hkv={b.hkv} splits={step.splits}")
            head = (b.problem(), step.view)
            if many:
                _context.pkv_prompt_window(*head, w["tok_offsets"], step.num_tokens, w["seq_lens"],
                                           step.splits, w["q"], w["k_pool"], w["v_pool"],
                                           w["block_table"], shared, step.out, step.lse)
            else:
                _context.pkv_attend_window(*head, w["seq_lens"], step.splits, w["q"], w["k_pool"],
                                           w["v_pool"], w["block_table"], shared, step.out,
                                           step.lse)
            torch.cuda.synchronize()
            check(step.out, step.lse, b.reference(), "f16", 64, b.vmax, many, "shared workspace")
            assert not shared[:256 << 10].any()


@pytest.mark.parametrize("rows", [64, 65, 130, 300])
def test_prompt_splits_of_many_rows(rows):
    """The launch counts the tiles of any number of rows before it chooses the
    ranges; rows without new tokens between them."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, 400, rows)
    new = np.minimum(lens, rng.integers(0, 40, rows) * (rng.random(rows) < 0.6))
    say(f"[splits of many rows] {rows}")
    b = Batch(rows, lens, new, hkv=1, group=8, d=64, dtype="bf16", window=300, sinks=3)
    w = b.device()
    step = engine.PromptStep(b.problem(), int(new.sum()), 300, 3, splits=6)
    out, lse = step.run(w)
    torch.cuda.synchronize()
    check(out, lse, b.reference(), "bf16", 64, b.vmax, True, f"{rows} rows")


def test_prompt_split_replays_follow_the_offsets():
    """A captured prompt whose rows change: other tile counts, so other ranges,
    on one workspace; one token a row without offsets too."""
    b = Batch(31, [2000, 1500, 900, 60], [60, 1, 33, 60], hkv=1, group=4, d=128)
    w = b.device()
    n = int(b.new.sum())
    step = engine.PromptStep(b.problem(), n, 0, 0, splits=64)
    step.run(w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run(w)
    for new in ([60, 1, 33, 60], [0, 0, 154, 0], [100, 54, 0, 0], [1, 1, 1, 1], [0, 0, 0, 60]):
        say(f"[replay] new tokens {new}")
        off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        w["tok_offsets"].copy_(torch.from_numpy(off))
        step.out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = step.out.clone(), step.lse.clone()
        one = engine.PromptStep(b.problem(), n, 0, 0, splits=1)
        one.out.fill_(7)
        one.run(w)
        torch.cuda.synchronize()
        m = int(off[-1])
        assert (got[0][m:] == 7).all()
        # The same sums in another order: both within a rounding of P and of the output.
        err = (got[0][:m].double() - one.out[:m].double()).abs().max().item() if m else 0
        assert err <= 4 * 2.0 ** -11 * b.vmax, err
        assert not step.workspace[:256 << 10].any()
    with pytest.raises(ValueError):
        step.run(dict(w, tok_offsets=None))
    alone = engine.PromptStep(b.problem(), 4, 0, 0, splits=64)
    ones = Batch(31, [2000, 1500, 900, 60], [1, 1, 1, 1], hkv=1, group=4, d=128)
    x = ones.device()
    out, lse = alone.run(dict(x, tok_offsets=None))
    torch.cuda.synchronize()
    check(out, lse, ones.reference(), "f16", 128, ones.vmax, True, "one token a row")
