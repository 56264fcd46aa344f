"""GPU: the context operators at their edges: non-finite tokens, weights far
apart, steps built on one stream and run on another, ranges of every kind.
Bounds as derived in tests/context_cases.py."""
import numpy as np
import pytest
import torch

from oracle import context as oc
from paged_kv_gqa_block_amd import _context, engine
from tests.context_cases import TORCH, Batch, check, f64, lse_bound, out_bound
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


# ---- streams -----------------------------------------------------------------------------

def _busy(stream, ms=60):
    """Keep `stream` at work for a while: passes over 1 GiB of its own."""
    with torch.cuda.stream(stream):
        x = torch.zeros(1 << 28, dtype=torch.float32, device="cuda")
        for _ in range(2 * ms):
            x.add_(1)


def _litter(nbytes):
    """Leave set bits in the memory that the current stream's next buffers of
    these sizes get."""
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in nbytes]
    del junk


KINDS = ["window", "kv4", "prompt"]


def _of_kind(kind):
    b = Batch(51, [900, 450, 77], [1, 1, 1] if kind != "prompt" else [3, 40, 77], hkv=2, group=4,
              kv4=kind == "kv4")

    def make():
        if kind == "prompt":
            return engine.PromptStep(b.problem(), int(b.new.sum()), splits=8)
        return _step(b, 16)
    return b, b.device(), make


@pytest.mark.parametrize("given", ["argument", "number", "current", "bound"])
@pytest.mark.parametrize("kind", KINDS)
def test_step_built_on_a_busy_stream_runs_on_another(kind, given):
    """The workspace's counters are zero and its memory free before the first call
    on any stream, whatever still runs on the stream that it was built on."""
    b, w, make = _of_kind(kind)
    sizes = [t.numel() * t.element_size() for t in (lambda s: (s.workspace, s.out, s.lse))(make())]
    building, running = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    say(f"[built elsewhere] {kind} {given}")
    with torch.cuda.stream(building):
        _litter(sizes)
        _busy(building)
        step = make()
    if given == "current":
        with torch.cuda.stream(running):
            out, lse = step.run(w)
    elif given == "bound":
        out, lse = step.run_bound(step.bind(w, running))
    else:
        out, lse = step.run(w, running if given == "argument" else running.cuda_stream)
    running.synchronize()
    check(out, lse, b.reference(), "f16", 128, b.vmax, kind == "prompt", kind)
    torch.cuda.synchronize()
    assert not step.workspace[:256 << 10].any()


@pytest.mark.parametrize("kind", ["plan", "device", "selfplan"])
def test_engine_step_built_on_a_busy_stream_runs_on_another(kind):
    """The same of the steps over the whole context: plan, device plan and claim
    counter are not cleared behind a call."""
    b = Batch(53, [900, 450, 77], hkv=2, group=4)
    w, host = b.device(), b.lens.copy()

    def make():
        if kind == "plan":
            return engine.DecodeStep(b.problem(), "workqueue", 8)
        return {"device": engine.DeviceStep, "selfplan": engine.SelfPlannedStep}[kind](b.problem(), 8)
    first = make()
    zeros = {"plan": "plan_dev", "device": "plan_dev", "selfplan": "counter"}[kind]
    sizes = [t.numel() * t.element_size() for t in
             (first.out, first.lse, first.st_m, first.st_l, first.st_o, getattr(first, zeros))]
    building, running = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    say(f"[engine step built elsewhere] {kind}")
    with torch.cuda.stream(building):
        _litter(sizes)
        _busy(building)
        step = make()
    with torch.cuda.stream(running):
        if kind == "plan":
            step.plan(host, running)
        step.run(w, running)
    running.synchronize()
    check(step.out, step.lse, b.reference(), "f16", 128, b.vmax, True, kind)


@pytest.mark.parametrize("given", ["argument", "current"])
@pytest.mark.parametrize("kind", KINDS)
def test_dropped_step_keeps_its_memory_until_its_stream_is_done(kind, given):
    """A step that is dropped while its call waits on another stream: the memory
    of its workspace goes to nobody else before the call is done."""
    b, w, make = _of_kind(kind)
    running = torch.cuda.Stream()
    step = make()
    at, size = step.workspace.data_ptr(), step.workspace.numel()
    torch.cuda.synchronize()
    say(f"[dropped] {kind} {given}")
    _busy(running)
    if given == "argument":
        out, lse = step.run(w, running)
    else:
        with torch.cuda.stream(running):
            out, lse = step.run(w)
    del step
    other = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert all(t.data_ptr() != at for t in other)
    torch.cuda.synchronize()
    check(out, lse, b.reference(), "f16", 128, b.vmax, kind == "prompt", kind)


def test_new_cache_built_on_a_busy_stream_keeps_what_another_stores():
    """The zeros of a new 4-bit pool are there before anything is stored."""
    b = Batch(52, [100, 40], [100, 40], hkv=2, group=1, kv4=True)
    w, n = b.device(), 140
    x = torch.randn(n, 2, 128, generator=torch.Generator().manual_seed(1)).half().cuda()
    outs = []
    building, running = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    say("[new cache]")
    for _ in range(2):
        with torch.cuda.stream(building):
            _busy(building)
            cache = engine.Kv4Cache(b.problem())
        args = (w["block_table"], w["seq_lens"], w["tok_offsets"])
        cache.store(x, x, *args, stream=running)
        running.synchronize()
        building.synchronize()
        outs.append(cache.load(*args, torch.empty_like(x), torch.empty_like(x)))
    torch.cuda.synchronize()
    assert all(_same(a, c) for a, c in zip(*outs)) and outs[0][0].abs().sum() > 0
    assert _same(outs[0][0], outs[0][1])


def test_step_built_inside_a_capture():
    """A step whose buffers and zeros belong to the graph: every replay is right."""
    b, w, make = _of_kind("window")
    want = [t.clone() for t in make().run(w)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = make()
        step.run(w)
    for i in range(3):
        say(f"[built in a capture] replay {i}")
        graph.replay()
        torch.cuda.synchronize()
        assert _same(step.out, want[0]) and _same(step.lse, want[1])
        make().run(w)
        torch.cuda.synchronize()


# ---- weights far apart --------------------------------------------------------------------

def _one_row(q, k, v, scale, kv4, dtype):
    """A row of n tokens stored through the framework: (problem, call arguments,
    K and V as the cache holds them in fp64).  q [m][Hq][d] are its last m tokens."""
    n, hkv, d = k.shape
    pages = -(-n // 16)
    prob = engine.make_problem(1, q.shape[1], hkv, d, 16, pages, pages, dtype, scale)
    w = {"q": q.cuda(), "block_table": torch.randperm(
            pages, generator=torch.Generator().manual_seed(n)).int().view(1, -1).cuda(),
         "seq_lens": torch.tensor([n], dtype=torch.int32).cuda()}
    off = torch.tensor([0, n], dtype=torch.int32).cuda()
    if kv4:
        cache = engine.Kv4Cache(prob)
        cache.store(k.cuda(), v.cuda(), w["block_table"], w["seq_lens"], off)
        w["kv4_pool"] = cache.pool
        k, v = (oc.kv4_values(*oc.kv4_quantise(f64(x), dtype)) for x in (k, v))
    else:
        w["k_pool"], w["v_pool"] = (torch.zeros(pages, hkv, 16, d, dtype=TORCH[dtype],
                                                device="cuda") for _ in range(2))
        engine.store_kv(prob, k.cuda(), v.cuda(), w["block_table"], w["seq_lens"], off,
                        w["k_pool"], w["v_pool"])
        k, v = f64(k), f64(v)
    return prob, w, k, v


def _within(out, lse, ref, dtype, d, vmax, one_part, label):
    """The element bounds of tests/context_cases.py with the kernels' own share of
    f16 weights that are subnormal: the largest weight of a query is kept at 2^7
    or more (prompt) or 2^12 or more (decode), so a part of one is off by at most
    2^-25 / 2^7 or 2^-25 / 2^12 of the largest, n times."""
    want, want_lse, (mag, score_mag, count) = ref
    bound = out_bound(want, mag, score_mag, count, 0.0, d, dtype, one_part)
    if dtype == "f16":
        bound = bound + count.reshape(-1, 1, 1) * 2.0 ** (-32 if one_part else -37) * vmax
    over = np.abs(f64(out) - want) / bound
    assert np.isfinite(f64(out)).all() and over.max() <= 1, f"{label}: {over.max():.2f} of the bound"
    lo = np.abs(f64(lse) - want_lse) / lse_bound(want_lse, score_mag, count, d)
    assert lo.max() <= 1, f"{label}: lse {lo.max():.2f} of the bound"


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("d,dtype", [(128, "f16"), (64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("gap", [6, 10, 14, 16, 17.4, 20, 24])
def test_one_token_far_above_the_rest(gap, d, dtype, kv4, many):
    """A first token whose weight exceeds each other's by exp(gap) and whose V is
    zero, as a sink's often is: the output is what the others leave."""
    say(f"[sink] gap={gap} d={d} {dtype} kv4={kv4} prompt={many}")
    rng = np.random.default_rng(int(10 * gap))
    n, hkv, group = 1500, 2, 4
    t = TORCH[dtype]
    q = torch.zeros(5 if many else 1, hkv * group, d)
    q[..., 0] = 8.0
    q[..., 32:] = torch.from_numpy(rng.standard_normal((*q.shape[:2], d - 32)).astype(np.float32))
    k = torch.from_numpy(rng.standard_normal((n, hkv, d)).astype(np.float32)) * 0.05
    k[..., 0] = 0.0
    k[0] = 0.0
    k[0, :, 0] = 3.0  # exact in 4 bits
    v = 50 + 50 * torch.from_numpy(rng.standard_normal((n, hkv, d)).astype(np.float32))
    v[0] = 0.0
    scale = float(np.float32(gap / 24.0))
    prob, w, k64, v64 = _one_row(q.to(t), k.to(t), v.to(t), scale, kv4, dtype)
    m = q.shape[0]
    ref = oc.attend_row(f64(q.to(t)), range(n - m, n), k64, v64, scale)
    if many:
        w["tok_offsets"] = torch.tensor([0, m], dtype=torch.int32).cuda()
        steps = [engine.PromptStep(prob, m, splits=s) for s in (1, 4)]
    else:
        steps = [(engine.Kv4Step if kv4 else engine.WindowStep)(prob, splits=s) for s in (1, 5)]
    for step in steps:
        out, lse = step.run(w)
        torch.cuda.synchronize()
        _within(out, lse, ref, dtype, d, np.abs(v64).max(), many, f"splits {step.splits}")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale,spread", [(-0.2, 1.0), (0.0, 1.0), (1.0, 1.0), (1.0, 2.0),
                                          (1e-30, 1.0)])
def test_scales_of_every_type_and_kind(scale, spread, dtype, kv4, many):
    say(f"[scales] {scale} spread={spread} {dtype} kv4={kv4} prompt={many}")
    b = Batch(54, [90, 300, 40], [90, 20, 10] if many else None, scale=scale, spread=spread,
              dtype=dtype, kv4=kv4)
    step = engine.PromptStep(b.problem(), int(b.new.sum())) if many else _step(b)
    out, lse = step.run(b.device())
    torch.cuda.synchronize()
    _within(out, lse, b.reference(), dtype, 128, b.vmax, many, f"scale {scale}")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-38, -1e-38, 1e-39])
def test_smallest_scales_of_the_largest_products(scale, kv4, many):
    """bf16 products <q, k> near 2^124: a scale of zero weighs every token alike, and
    one about the smallest normal number keeps its value."""
    say(f"[smallest scales] {scale} kv4={kv4} prompt={many}")
    b = Batch(55, [90, 300, 40], [90, 20, 10] if many else None, scale=scale, spread=2.0 ** 60,
              dtype="bf16", kv4=kv4)
    b.q = b.q * 2.0 ** 60
    step = engine.PromptStep(b.problem(), int(b.new.sum())) if many else _step(b)
    out, lse = step.run(b.device())
    torch.cuda.synchronize()
    _within(out, lse, b.reference(), "bf16", 128, b.vmax, many, f"scale {scale}")


# ---- ranges ----------------------------------------------------------------------------------
# What the header says of them, in plain numbers: the caps, and which states a launch writes.

def _cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _decode_ranges(pages, pairs):
    fill = -(-_cus() // pairs)
    even = 1 if pairs >= 8 * _cus() else 20 * _cus() // pairs
    own = 1 if pages <= 40 else min(fill, -(-pages // 8))
    return max(own, min(even, pages // 96), 1)


def _decode_plan(pages, hkv, cap):
    """(ranges of every row, rounds of workgroups before evening out, whether the
    ranges were made longer to come out even)."""
    pages = np.asarray(pages)
    t_max, rows = int(pages.max()), len(pages)

    def ranges(per):
        return np.maximum(1, -(-pages // per))
    per = first = max(1, -(-t_max // min(cap, _decode_ranges(t_max, rows * hkv))))
    total = int(ranges(per).sum())
    rounds = -(-total * hkv // _cus())
    if 1 < rows <= 64 and 2 <= rounds <= 4 and cap > 1:
        even, t = (rounds - 1) * _cus() // hkv, total
        for _ in range(3):
            if t <= even or even < rows:
                break
            per = min(per + 1 + int(np.float32(per) * np.float32(t - even) / np.float32(even)), t_max)
            t = int(ranges(per).sum())
        if t > even or (rounds - 1) * (per + 8) >= rounds * (first + 8):
            per = first
    return ranges(per), rounds, per != first


def _decode_states(step, rows, hkv, group):
    """Ranges of every (row, KV head) whose state the last call wrote."""
    n = rows * hkv * step.splits * group * 2 * 4
    ml = step.workspace[256 << 10:(256 << 10) + n].view(torch.float32)
    return (~torch.isnan(ml.view(rows, hkv, step.splits, group * 2))).all(-1).sum(-1).cpu().numpy()


def _checked_decode(b, cap, wide=None):
    """Run, compare with the oracle and the expected ranges; (step, rounds, evened)."""
    w, prob = b.device(), b.problem()
    if wide:
        table = torch.zeros(len(b.lens), wide, dtype=torch.int32, device="cuda")
        table[:, :w["block_table"].shape[1]] = w["block_table"]
        w["block_table"], prob = table, b.problem(max_pages_per_row=wide)
    step = (engine.Kv4Step if b.kv4 else engine.WindowStep)(prob, b.window, b.sinks, cap)
    step.workspace[256 << 10:] = 255  # NaN, in every state
    out, lse = step.run(w)
    torch.cuda.synchronize()
    pages = [-(-int(n) // 16) for n in b.lens]
    want, rounds, evened = _decode_plan(pages, b.hkv, step.splits)
    got = _decode_states(step, len(b.lens), b.hkv, b.group)
    assert (got == np.where(want > 1, want, 0)[:, None]).all(), (got.tolist(), want.tolist())
    check(out, lse, b.reference(), b.dtype, b.d, b.vmax, False, "ranges")
    assert not step.workspace[:256 << 10].any()
    return step, rounds, evened


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("rows,length,hkv", [(1, 100, 2), (1, 640, 2), (1, 641, 2), (2, 1100, 1),
                                             (8, 384, 2), (8, 1300, 2), (3, 3300, 1)])
def test_short_rows_under_a_wide_table(rows, length, hkv, kv4):
    """Ranges follow the rows that there are: the bits of a table as wide as the
    rows, and rows of up to 40 pages whole."""
    say(f"[wide table] rows={rows} length={length} Hkv={hkv} kv4={kv4}")
    lens = [length - 5 * i for i in range(rows)]
    b = Batch(61, lens, hkv=hkv, group=4, kv4=kv4)
    tight, _, _ = _checked_decode(b, None)
    for wide in (2048, 8192):
        step, _, _ = _checked_decode(b, None, wide)
        assert step.splits > tight.splits
        assert _same(step.out, tight.out) and _same(step.lse, tight.lse)


EVENED = [(5, 900, 1000, 8, True), (9, 700, 720, 8, True), (20, 660, 700, 8, True),
          (40, 100, 700, 8, False), (60, 700, 900, 1, True), (30, 650, 1000, 2, True),
          (64, 641, 650, 3, True), (60, 3050, 3060, 5, False)]


@pytest.mark.parametrize("rows,low,high,hkv,evened,kv4",
                         [(*e, kv4) for e in EVENED for kv4 in (False, True)
                          if not kv4 or e[2] < 3000])
def test_ranges_evened_out(rows, low, high, hkv, evened, kv4):
    """Two to four rounds of workgroups: longer ranges where those come out even and
    cost less, the first ones otherwise."""
    lens = np.random.default_rng(rows).integers(low, high + 1, rows)
    lens[0] = high
    b = Batch(62, lens, hkv=hkv, group=1, d=64, kv4=kv4, dtype="bf16")
    say(f"[evened] rows={rows} {low}..{high} Hkv={hkv} kv4={kv4}")
    _, rounds, got = _checked_decode(b, 64)
    if _cus() == 256:  # the sizes above are chosen for a whole card
        assert 2 <= rounds <= 4 and got == evened, (rounds, got)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 9, 16])
def test_joins_of_every_group(group, kv4):
    """Sixteen ranges and more of one row, joined by every number of heads."""
    for d in (64, 128):
        say(f"[joins] G={group} d={d} kv4={kv4}")
        b = Batch(63, [2100], hkv=1, group=group, d=d, kv4=kv4)
        for cap in (None, 2, 5, 300):
            _checked_decode(b, cap, 200)


def _prompt_states(step, tiles, hkv, d):
    slot = 256 * (d // 2 + 2)
    st = step.workspace[256 << 10:].view(torch.float32)
    st = st[:tiles * hkv * step.splits * slot].view(tiles, hkv, step.splits, slot)
    return (~torch.isnan(st[..., -512:])).all(-1).sum(-1).cpu().numpy()


def _prompt_plan(b, cap, hkv):
    """Ranges of every tile, rows' last tiles first."""
    per_row = [-(-int(m) * b.group // 128) for m in b.new]
    longest = max([-(-int(n) // 64) for n, m in zip(b.lens, b.new) if m], default=0)
    slots = 2 * _cus() // hkv
    splits = min(cap, longest // 8 if longest >= 16 else 1, max(slots // max(sum(per_row), 1), 1))
    least = -(-longest // splits)
    out = []
    for n, m, tiles in zip(b.lens, b.new, per_row):
        for tile in reversed(range(tiles)):
            last = int(n) - int(m) + min((tile + 1) * 128 - 1, int(m) * b.group - 1) // b.group
            steps = -(-(last // 16 + 1) // 4)
            ns = -(-steps // max(least, -(-steps // splits)))
            out.append(ns if ns > 1 else 0)
    return out


@pytest.mark.parametrize("kv4,d,dtype", [(False, 128, "bf16"), (False, 64, "f16"), (True, 128, "f16")])
@pytest.mark.parametrize("lens,new", [
    ([5000], [1]), ([4000, 700, 100], [33, 5, 100]), ([1024], [1024]), ([200, 90], [20, 90]),
    ([1023, 2500, 0], [60, 70, 0])])
def test_prompt_ranges_follow_the_rows(lens, new, kv4, d, dtype):
    """Ranges of a prompt: eight steps or more each, in a table as wide as the rows
    and in a wide one, with the same bits."""
    b = Batch(64, lens, new, hkv=2, group=2, d=d, dtype=dtype, kv4=kv4)
    w, n = b.device(), int(b.new.sum())
    ref, outs = b.reference(), []
    for wide, cap in ((None, None), (8192, None), (8192, 3), (8192, 200)):
        say(f"[prompt ranges] {lens} {new} kv4={kv4} d={d} {dtype} wide={wide} cap={cap}")
        x, prob = w, b.problem()
        if wide:
            table = torch.zeros(len(lens), wide, dtype=torch.int32, device="cuda")
            table[:, :w["block_table"].shape[1]] = w["block_table"]
            x, prob = dict(w, block_table=table), b.problem(max_pages_per_row=wide)
        step = engine.PromptStep(prob, n, splits=cap)
        step.workspace[256 << 10:] = 255
        out, lse = step.run(x)
        torch.cuda.synchronize()
        check(out, lse, ref, dtype, d, b.vmax, True, f"wide {wide} cap {cap}")
        plan = _prompt_plan(b, step.splits, 2)
        if step.splits > 1:
            got = _prompt_states(step, len(plan), 2, d)
            assert (got == np.array(plan)[:, None]).all(), (got.tolist(), plan)
            assert not step.workspace[:256 << 10].any()
        outs.append((plan, out.clone(), lse.clone()))
    for plan, out, lse in outs[1:]:
        if plan == outs[0][0]:
            assert _same(out, outs[0][1]) and _same(lse, outs[0][2])


def test_prompt_ranges_behind_a_window():
    """A window over long rows: ranges of the pages that a tile sees, not of the row."""
    b = Batch(65, [6000, 3000], [40, 3], hkv=1, group=4, window=1500, sinks=20)
    w = b.device()
    for cap in (None, 2, 50):
        say(f"[prompt window ranges] cap={cap}")
        step = engine.PromptStep(b.problem(), 43, 1500, 20, cap)
        step.workspace[256 << 10:] = 255
        out, lse = step.run(w)
        torch.cuda.synchronize()
        check(out, lse, b.reference(), "f16", 128, b.vmax, True, f"cap {cap}")
        used = _prompt_states(step, 3, 1, 128)
        assert (used == (2 if cap == 2 else 3)).all(), used.tolist()


@pytest.mark.parametrize("rows", [64, 70])
def test_prompt_ranges_of_many_rows(rows):
    """Rows around and beyond what a wave holds, in ranges, one of them long."""
    rng = np.random.default_rng(rows)
    lens = rng.integers(0, 900, rows)
    lens[rows - 3] = 3500
    new = np.minimum(lens, rng.integers(0, 9, rows) * (rng.random(rows) < 0.5))
    new[rows - 3] = 20
    say(f"[prompt ranges of many rows] {rows}")
    b = Batch(66, lens, new, hkv=1, group=2, d=64, dtype="bf16")
    step = engine.PromptStep(b.problem(), int(new.sum()), splits=6)
    step.workspace[256 << 10:] = 255
    out, lse = step.run(b.device())
    torch.cuda.synchronize()
    check(out, lse, b.reference(), "bf16", 64, b.vmax, True, f"{rows} rows")
    plan = _prompt_plan(b, 6, 1)
    got = _prompt_states(step, len(plan), 1, 64)
    assert max(plan) > 1 and (got == np.array(plan)[:, None]).all(), (got.tolist(), plan)


def test_one_workspace_for_ranges_of_all_kinds():
    """Calls whose pairs and tiles are really cut share one workspace in turn."""
    steps = []
    for i, (lens, new, hkv, cap) in enumerate((
            ([900, 33], None, 2, 40), ([700] * 30, None, 2, 3), ([2000], None, 1, 100),
            ([1500, 2400], [90, 40], 3, 4), ([1100], [1], 8, 30))):
        b = Batch(70 + i, lens, new, hkv=hkv, group=2, d=64)
        step = (engine.PromptStep(b.problem(), int(b.new.sum()), splits=cap) if new
                else _step(b, cap))
        steps.append((b, step, b.device(), new is not None, b.reference()))
    shared = torch.zeros(max(x[1].workspace.numel() for x in steps), dtype=torch.uint8, device="cuda")
    for b, step, w, many, ref in steps + steps[::-1]:
        say(f"[shared ranges] B={len(b.lens)} Hkv={b.hkv} cap={step.splits} prompt={many}")
        head = (b.problem(), step.view)
        if many:
            _context.pkv_prompt_window(*head, w["tok_offsets"], step.num_tokens, w["seq_lens"],
                                       step.splits, w["q"], w["k_pool"], w["v_pool"],
                                       w["block_table"], shared, step.out, step.lse)
        else:
            _context.pkv_attend_window(*head, w["seq_lens"], step.splits, w["q"], w["k_pool"],
                                       w["v_pool"], w["block_table"], shared, step.out, step.lse)
        torch.cuda.synchronize()
        check(step.out, step.lse, ref, "f16", 64, b.vmax, many, "shared ranges")
        assert not shared[:256 << 10].any()


@pytest.mark.parametrize("kv4", [False, True])
def test_binding_and_engine_make_the_same_calls(kv4):
    """The plain binding of every entry point against the classes: the same bits."""
    b = Batch(80, [900, 0, 333], [40, 0, 333], hkv=2, group=4, kv4=kv4, window=500, sinks=4)
    w, prob = b.device(), b.problem()
    n = int(b.new.sum())
    x = torch.randn(n, 2, 2, 128, generator=torch.Generator().manual_seed(2)).half().cuda()
    k, v = x[:, 0], x[:, 1]
    run = (w["tok_offsets"], n, w["seq_lens"])
    say(f"[binding] kv4={kv4}")
    if kv4:
        mine, cache = w["kv4_pool"].clone(), engine.Kv4Cache(prob, pool=w["kv4_pool"])
        cache.store(k, v, w["block_table"], w["seq_lens"], w["tok_offsets"])
        _context.pkv_kv4_store(prob, *run, k, v, w["block_table"], mine)
        outs = [[torch.empty(n, 2, 128, dtype=torch.float16, device="cuda") for _ in range(2)]
                for _ in range(2)]
        cache.load(w["block_table"], w["seq_lens"], w["tok_offsets"], *outs[0])
        _context.pkv_kv4_load(prob, *run, w["block_table"], mine, *outs[1])
        torch.cuda.synchronize()
        assert _same(mine, w["kv4_pool"]) and all(_same(a, c) for a, c in zip(*outs))
        pools = (mine,)
    else:
        mine = w["k_pool"].clone(), w["v_pool"].clone()
        engine.store_kv(prob, k, v, w["block_table"], w["seq_lens"], w["tok_offsets"],
                        w["k_pool"], w["v_pool"])
        _context.pkv_store_kv(prob, *run, k, v, w["block_table"], *mine)
        torch.cuda.synchronize()
        assert _same(mine[0], w["k_pool"]) and _same(mine[1], w["v_pool"])
        pools = mine
    for step, q in ((_step(b), w["q"][:3].contiguous()),
                    (engine.PromptStep(prob, n, 500, 4, 3), w["q"])):
        out, lse = (t.clone() for t in step.run(dict(w, q=q)))
        got, got_lse = torch.zeros_like(out), torch.zeros_like(lse)
        many = isinstance(step, engine.PromptStep)
        fn = {(False, False): _context.pkv_attend_window, (False, True): _context.pkv_attend_kv4,
              (True, False): _context.pkv_prompt_window, (True, True): _context.pkv_prompt_kv4}
        head = (prob, step.view, *(run if many else (w["seq_lens"],)), step.splits, q)
        fn[many, kv4](*head, *pools, w["block_table"], step.workspace, got, got_lse)
        torch.cuda.synchronize()
        assert _same(out, got) and _same(lse, got_lse)
