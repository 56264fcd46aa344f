"""GPU: the context operators at their edges: non-finite tokens, weights far
apart, steps built on one stream and run on another, ranges of every kind.
Bounds as derived in tests/context_cases.py."""
import numpy as np
import pytest
import torch

from oracle import context as oc
from paged_kv_gqa_block_amd import engine
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


@pytest.mark.parametrize("kind", KINDS)
def test_step_built_on_a_busy_stream_runs_on_another(kind):
    """The workspace's counters are zero and its memory free when the constructor
    returns, whatever still runs on the stream that it was built on."""
    b, w, make = _of_kind(kind)
    sizes = [t.numel() * t.element_size() for t in (lambda s: (s.workspace, s.out, s.lse))(make())]
    building, running = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    say(f"[built elsewhere] {kind}")
    with torch.cuda.stream(building):
        _litter(sizes)
        _busy(building)
        step = make()
    out, lse = step.run(w, running)
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
