"""One decode step through libpkv: buffers from torch, work in the library.

``DecodeStep`` owns the per-step buffers (pinned host plan, device plan,
partial states, output) for one problem shape and one path, and calls the C
ABI in the documented order: pkv_plan -> pkv_decode -> pkv_merge.  torch only
allocates memory and supplies the stream.
"""
from __future__ import annotations

import ctypes
import json
import os

import numpy as np
import torch

from . import _context, _lib
from ._lib import (PATH_IDS, PATH_NAMES, PKV_NOSPLIT, PKV_WORKQUEUE, make_problem, pkv_decode,
                   pkv_decode_device, pkv_merge, pkv_merge_device, pkv_plan, pkv_plan_bytes,
                   pkv_plan_device, pkv_policy)

TORCH_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
POLICY_TABLE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "policy_table.json")
COST_MODEL_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cost_model.json")


def problem_from_workload(w: dict, kernel: str = "auto") -> _lib.pkv_problem:
    spec = w["spec"]
    return make_problem(spec.batch, spec.num_q_heads, spec.num_kv_heads, spec.head_dim,
                        spec.page_size, int(w["k_pool"].shape[0]),
                        int(w["block_table"].shape[1]), spec.dtype, w["scale"], kernel)


def to_device(w: dict, device="cuda") -> dict:
    """Copy a generated workload's tensors to the GPU (inputs resident in HBM)."""
    out = dict(w)
    for key in ("q", "k_pool", "v_pool", "block_table", "seq_lens"):
        out[key] = w[key].to(device).contiguous()
    out["seq_lens_host"] = w["seq_lens"].numpy().astype(np.int32).copy()
    return out


def _await_buffers(device: torch.device) -> None:
    """Wait until new buffers of `device` are ready: their zeros were filled, and
    earlier owners of their memory were done, in the order of the current stream
    alone, and a step may run on any.  Not inside a graph capture, where the
    fills become part of the graph."""
    if device.type == "cuda":
        with torch.cuda.device(device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()


class DecodeStep:
    """Buffers and calls for one (problem, path, split cap)."""

    def __init__(self, prob: _lib.pkv_problem, path, splits: int, device="cuda"):
        self.prob = prob
        self.path = PATH_IDS[path] if isinstance(path, str) else path
        self.splits = int(splits)
        self.device = torch.device(device)
        nbytes = pkv_plan_bytes(prob, self.path, self.splits)
        if nbytes == 0:
            raise _lib.PkvError("pkv_plan_bytes", _lib.PKV_EINVAL, "invalid problem")
        pin = self.device.type == "cuda"
        self.plan_host = torch.zeros(nbytes // 4, dtype=torch.int32, pin_memory=pin)
        self.plan_dev = torch.zeros(nbytes // 4, dtype=torch.int32, device=self.device)
        self.info = None
        g = prob.num_q_heads // prob.num_kv_heads
        d = prob.head_dim
        dt = torch.bfloat16 if prob.dtype == _lib.PKV_BF16 else torch.float16
        self.out = torch.empty(prob.batch, prob.num_q_heads, d, dtype=dt, device=self.device)
        self.lse = torch.empty(prob.batch, prob.num_q_heads, dtype=torch.float32,
                               device=self.device)
        # Upper bound of state slots: every row at the split cap.
        slots = prob.batch * prob.num_kv_heads * (1 if self.path == PKV_NOSPLIT else self.splits)
        self.st_m = torch.empty(max(slots, 1), g, dtype=torch.float32, device=self.device)
        self.st_l = torch.empty(max(slots, 1), g, dtype=torch.float32, device=self.device)
        self.st_o = torch.empty(max(slots, 1), g, d, dtype=torch.float32, device=self.device)
        _await_buffers(self.device)

    def plan(self, seq_lens_host: np.ndarray, stream=None) -> _lib.pkv_plan_info:
        self.info = pkv_plan(self.prob, np.ascontiguousarray(seq_lens_host, dtype=np.int32),
                             self.path, self.splits, self.plan_host, self.plan_dev, stream=stream)
        return self.info

    def decode(self, w: dict, stream=None) -> None:
        pkv_decode(self.prob, self.plan_host, self.plan_dev, w["q"], w["k_pool"], w["v_pool"],
                   w["block_table"], w["seq_lens"], self.st_m, self.st_l, self.st_o, self.out,
                   self.lse, stream=stream)

    def merge(self, stream=None) -> None:
        pkv_merge(self.prob, self.plan_host, self.plan_dev, self.st_m, self.st_l, self.st_o,
                  self.out, self.lse, stream=stream)

    def run(self, w: dict, stream=None):
        self.decode(w, stream)
        self.merge(stream)
        return self.out, self.lse

    def bind(self, w: dict, stream=None) -> tuple:
        """pkv_decode and pkv_merge of this step on workload buffers `w`, with
        their arguments marshalled once (see ``run_bound``)."""
        st = stream if stream is not None else torch.cuda.current_stream()
        dec = _lib.bind_call("pkv_decode", self.prob, self.plan_host, self.plan_dev, w["q"],
                             w["k_pool"], w["v_pool"], w["block_table"], w["seq_lens"],
                             self.st_m, self.st_l, self.st_o, self.out, self.lse, st)
        mrg = _lib.bind_call("pkv_merge", self.prob, self.plan_host, self.plan_dev, self.st_m,
                             self.st_l, self.st_o, self.out, self.lse, st)
        return dec, mrg

    def run_bound(self, bound: tuple) -> None:
        """The same two calls as ``run`` with pre-marshalled arguments: the
        host enqueues a step in a few microseconds, so timing loops of short
        steps measure the device, not the Python binding."""
        _lib.call_bound(bound[0])
        _lib.call_bound(bound[1])

    def decode_bound(self, bound: tuple) -> None:
        _lib.call_bound(bound[0])


class _PersistentStepBuffers:
    """Output and partial-state buffers of a persistent-grid workqueue step
    (room for B * Hkv * S states: the most any length mix can need)."""

    def __init__(self, prob: _lib.pkv_problem, splits: int, device="cuda"):
        self.prob = prob
        self.splits = int(splits)
        self.device = torch.device(device)
        g = prob.num_q_heads // prob.num_kv_heads
        d = prob.head_dim
        dt = torch.bfloat16 if prob.dtype == _lib.PKV_BF16 else torch.float16
        slots = prob.batch * prob.num_kv_heads * self.splits
        self.out = torch.empty(prob.batch, prob.num_q_heads, d, dtype=dt, device=self.device)
        self.lse = torch.empty(prob.batch, prob.num_q_heads, dtype=torch.float32,
                               device=self.device)
        self.st_m = torch.empty(slots, g, dtype=torch.float32, device=self.device)
        self.st_l = torch.empty(slots, g, dtype=torch.float32, device=self.device)
        self.st_o = torch.empty(slots, g, d, dtype=torch.float32, device=self.device)


class DeviceStep(_PersistentStepBuffers):
    """Device-planned workqueue step: plan, split and merge all on the GPU.

    ``run`` enqueues pkv_plan_device -> pkv_decode_device -> pkv_merge_device on
    one stream with no host work, so the three launches can be captured once in
    a HIP graph and replayed while the device lengths change.
    """

    def __init__(self, prob: _lib.pkv_problem, splits: int, device="cuda"):
        super().__init__(prob, splits, device)
        nbytes = pkv_plan_bytes(prob, PKV_WORKQUEUE, self.splits)
        if nbytes == 0:
            raise _lib.PkvError("pkv_plan_bytes", _lib.PKV_EINVAL, "invalid problem")
        self.plan_dev = torch.zeros(nbytes // 4, dtype=torch.int32, device=self.device)
        self.bad_rows = torch.zeros(1, dtype=torch.int32, device=self.device)
        _await_buffers(self.device)

    def run(self, w: dict, stream=None):
        pkv_plan_device(self.prob, w["seq_lens"], self.splits, self.plan_dev,
                        bad_rows_dev=self.bad_rows, stream=stream)
        pkv_decode_device(self.prob, self.plan_dev, self.splits, w["q"], w["k_pool"],
                          w["v_pool"], w["block_table"], self.st_m, self.st_l, self.st_o,
                          stream=stream)
        pkv_merge_device(self.prob, self.plan_dev, self.st_m, self.st_l, self.st_o, self.out,
                         self.lse, stream=stream)
        return self.out, self.lse


class SelfPlannedStep(_PersistentStepBuffers):
    """Self-planned workqueue step: the device-planned step in two launches.

    ``run`` enqueues pkv_decode_selfplan -> pkv_merge_selfplan: the split and
    merge kernels derive the workqueue of the device lengths themselves, so
    there is no planner launch and no plan buffer, only a one-word claim
    counter (zeroed here once; the merge leaves it zeroed).
    """

    def __init__(self, prob: _lib.pkv_problem, splits: int, device="cuda"):
        super().__init__(prob, splits, device)
        self.counter = torch.zeros(1, dtype=torch.int32, device=self.device)
        _await_buffers(self.device)

    def run(self, w: dict, stream=None):
        _lib.pkv_decode_selfplan(self.prob, w["seq_lens"], self.splits, self.counter, w["q"],
                                 w["k_pool"], w["v_pool"], w["block_table"], self.st_m,
                                 self.st_l, self.st_o, stream=stream)
        _lib.pkv_merge_selfplan(self.prob, w["seq_lens"], self.splits, self.counter, self.st_m,
                                self.st_l, self.st_o, self.out, self.lse, stream=stream)
        return self.out, self.lse


class _ContextCalls:
    """Argument checks and stream choice shared by the context operators
    (include/pkv_context.h).  They run on the device of their buffers, on the
    given stream or that device's current one.

    The first call on a stream waits for the fills of what the object allocated,
    and its memory is not reused before work on the torch streams that it was
    given is done.  A stream given as a number is not torch's to watch: keep the
    object until work on it is done.  A stream that is being captured cannot
    wait: build the object inside the capture, or let the device finish first
    (torch.cuda.graph does).  The caller's buffers have to be
    ready on the stream of a call and live until its work is done, as with every
    torch call.  A bound form and a captured graph hold addresses alone: keep the
    object and the buffers as long as those are used."""

    def __init__(self, prob: _lib.pkv_problem, device):
        self.prob = prob
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError(f"the context operators run on a GPU, not on {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self.dtype = torch.bfloat16 if prob.dtype == _lib.PKV_BF16 else torch.float16
        self.kv4_page_bytes = _context.pkv_kv4_page_bytes(prob.head_dim)

        p = prob
        self._shapes = {"block_table": (p.batch, p.max_pages_per_row), "seq_lens": (p.batch,),
                        "tok_offsets": (p.batch + 1,),
                        "kv4_pool": (p.num_pool_pages, p.num_kv_heads, self.kv4_page_bytes),
                        "pool": (p.num_pool_pages, p.num_kv_heads, p.page_size, p.head_dim),
                        "token": (p.num_kv_heads, p.head_dim),
                        "q": (p.batch, p.num_q_heads, p.head_dim)}
        self._prob_ref = ctypes.byref(prob)
        self._buffers, self._ready = (), None
        self._waited, self._known = set(), set()  # streams: ordered, and recorded too

    def _own_buffers(self, *buffers: torch.Tensor) -> None:
        """Take charge of buffers just allocated and filled on the current stream."""
        self._buffers = buffers
        with torch.cuda.device(self.device):
            if not torch.cuda.is_current_stream_capturing():
                self._ready = torch.cuda.Event()
                self._ready.record()
            home = torch.cuda.current_stream().cuda_stream
        self._waited, self._known = {home}, {home}

    def _meet(self, handle: int, stream) -> None:
        """Order a stream behind the fills of the object's buffers, and have their
        memory wait for it."""
        number = isinstance(stream, int)
        if handle not in self._waited and self._ready is not None:  # None: built in a capture
            with torch.cuda.device(self.device):
                if torch.cuda.is_current_stream_capturing():
                    return
                at = (torch.cuda.ExternalStream(handle) if number
                      else torch.cuda.current_stream() if stream is None else stream)
                at.wait_event(self._ready)
        self._waited.add(handle)
        if not number:  # of a number nobody knows how long its stream lives
            at = torch.cuda.current_stream(self.device) if stream is None else stream
            for t in self._buffers:
                t.record_stream(at)
            self._known.add(handle)

    def _stream(self, stream) -> int:
        if stream is None:
            handle = torch._C._cuda_getCurrentRawStream(self._index)
        else:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
        if self._buffers and handle not in self._known:
            self._meet(handle, stream)
        return handle

    def _expect(self, name: str, t: torch.Tensor, shape: tuple, dtype) -> int:
        """The address of `t`, after its checks."""
        if t.shape != shape or t.dtype != dtype or t.device != self.device:
            raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}, expected {shape} "
                             f"{dtype} on {self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def _tables(self, block_table, seq_lens) -> tuple:
        s = self._shapes
        return (self._expect("block_table", block_table, s["block_table"], torch.int32),
                self._expect("seq_lens", seq_lens, s["seq_lens"], torch.int32))

    def _offsets(self, tok_offsets, num_tokens: int):
        if tok_offsets is not None:
            return self._expect("tok_offsets", tok_offsets, self._shapes["tok_offsets"],
                                torch.int32)
        if num_tokens != self.prob.batch:
            raise ValueError(f"{num_tokens} tokens of {self.prob.batch} rows need tok_offsets")
        return None

    def _kv4_pool(self, pool) -> int:
        return self._expect("kv4_pool", pool, self._shapes["kv4_pool"], torch.uint8)

    def _pools(self, w: dict) -> tuple:
        """The cache of `w`: (its 4-bit pool,) or (its two 16-bit pools)."""
        if "kv4_pool" in w:
            return (self._kv4_pool(w["kv4_pool"]),)
        shape = self._shapes["pool"]
        return (self._expect("k_pool", w["k_pool"], shape, self.dtype),
                self._expect("v_pool", w["v_pool"], shape, self.dtype))

    def _new_tokens(self, name: str, t: torch.Tensor, n: int) -> tuple:
        """Address and token stride of new keys or values."""
        heads, d = self._shapes["token"]
        if t.shape != (n, heads, d) or t.dtype != self.dtype or t.device != self.device:
            raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} on {t.device}")
        stride = t.stride()
        if n > 1 and stride[1] == d and stride[2] == 1:
            return t.data_ptr(), stride[0]
        return t.data_ptr(), _context.token_stride(t)

    def _launch(self, fn: str, *args) -> None:
        """Call an entry point (every argument a number or a reference) with
        the buffers' device current."""
        call = getattr(_lib.LIB, fn)
        if torch._C._cuda_getDevice() == self._index:
            status = call(self._prob_ref, *args)
        else:
            with torch.cuda.device(self.device):
                status = call(self._prob_ref, *args)
        if status != _lib.PKV_OK:
            raise _lib.PkvError(fn, status, _lib.pkv_status_str(status))


class Kv4Cache(_ContextCalls):
    """The paged cache held in 4 bits: K and V of one layer in one byte pool.

    ``store`` quantises a run of new tokens as it writes them and ``load``
    reads a run back; ``Kv4Step`` and ``PromptStep`` attend over ``pool``.
    """

    def __init__(self, prob: _lib.pkv_problem, pool: torch.Tensor | None = None, device="cuda"):
        super().__init__(prob, pool.device if pool is not None else device)
        own = pool is None
        if own:
            pool = torch.zeros(prob.num_pool_pages, prob.num_kv_heads, self.kv4_page_bytes,
                               dtype=torch.uint8, device=self.device)
        self._kv4_pool(pool)
        self.pool = pool
        if own:
            self._own_buffers(pool)

    def store(self, k_new, v_new, block_table, seq_lens, tok_offsets=None, stream=None) -> None:
        """k_new, v_new: [tokens][Hkv][d], heads contiguous, any token stride
        that is a multiple of 8; seq_lens: the lengths after them; tok_offsets:
        [B + 1], or None for one token per row."""
        n = k_new.shape[0]
        table, lens = self._tables(block_table, seq_lens)
        self._launch("pkv_kv4_store", self._offsets(tok_offsets, n), n, lens,
                     *self._new_tokens("k_new", k_new, n), *self._new_tokens("v_new", v_new, n),
                     table, self.pool.data_ptr(), self._stream(stream))

    def load(self, block_table, seq_lens, tok_offsets, k_out, v_out, stream=None) -> tuple:
        """The values the cache stands for, into k_out, v_out [tokens][Hkv][d]."""
        n = k_out.shape[0]
        shape = (n, *self._shapes["token"])
        table, lens = self._tables(block_table, seq_lens)
        self._launch("pkv_kv4_load", self._offsets(tok_offsets, n), n, lens, table,
                     self.pool.data_ptr(), self._expect("k_out", k_out, shape, self.dtype),
                     self._expect("v_out", v_out, shape, self.dtype), self._stream(stream))
        return k_out, v_out


def store_kv(prob: _lib.pkv_problem, k_new, v_new, block_table, seq_lens, tok_offsets, k_pool,
             v_pool, stream=None) -> None:
    """Write a run of new tokens into the 16-bit pools (arguments as
    ``Kv4Cache.store``)."""
    calls, n = _ContextCalls(prob, k_pool.device), k_new.shape[0]
    table, lens = calls._tables(block_table, seq_lens)
    calls._launch("pkv_store_kv", calls._offsets(tok_offsets, n), n, lens,
                  *calls._new_tokens("k_new", k_new, n), *calls._new_tokens("v_new", v_new, n),
                  table, *calls._pools({"k_pool": k_pool, "v_pool": v_pool}),
                  calls._stream(stream))


class WindowStep(_ContextCalls):
    """One decode step over the visible part of a 16-bit cache: the last
    `window` tokens (0: all) and the first `sinks`.

    Owns the output and the workspace, so calls of one step must not overlap.
    ``run`` takes the dict of ``DecodeStep.run`` (q, k_pool, v_pool,
    block_table, seq_lens); ``bind`` / ``run_bound`` are its form with the
    arguments checked and marshalled once, for loops over fixed buffers.
    """

    _call, _num_pools = "pkv_attend_window", 2

    def __init__(self, prob: _lib.pkv_problem, window: int = 0, sinks: int = 0,
                 splits: int | None = None, device="cuda"):
        super().__init__(prob, device)
        self.view = _context.make_view(window, sinks)
        if splits is None:
            splits = _context.pkv_attend_splits(
                prob, self.view, torch.cuda.get_device_properties(
                    self.device).multi_processor_count)
        self.splits = splits
        nbytes = _context.pkv_attend_workspace_bytes(prob, splits)
        if nbytes == 0:
            raise _lib.PkvError("pkv_attend_workspace_bytes", _lib.PKV_EINVAL, "invalid problem")
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self.out = torch.empty(prob.batch, prob.num_q_heads, prob.head_dim, dtype=self.dtype,
                               device=self.device)
        self.lse = torch.empty(prob.batch, prob.num_q_heads, dtype=torch.float32,
                               device=self.device)
        self._own_buffers(self.workspace, self.out, self.lse)
        self._view_ref = ctypes.byref(self.view)
        self._own = (self.workspace.data_ptr(), nbytes, self.out.data_ptr(), self.lse.data_ptr())

    def bind(self, w: dict, stream=None) -> tuple:
        q = self._expect("q", w["q"], self._shapes["q"], self.dtype)
        table, lens = self._tables(w["block_table"], w["seq_lens"])
        pools = self._pools(w)
        if len(pools) != self._num_pools:
            raise ValueError(f"{type(self).__name__} over the wrong kind of cache")
        return (self._view_ref, lens, self.splits, q, *pools, table, *self._own,
                self._stream(stream))

    def run(self, w: dict, stream=None) -> tuple:
        return self.run_bound(self.bind(w, stream))

    def run_bound(self, bound: tuple) -> tuple:
        self._launch(self._call, *bound)
        return self.out, self.lse


class Kv4Step(WindowStep):
    """One decode step over the 4-bit cache (q, kv4_pool, block_table,
    seq_lens), with the view of ``WindowStep``."""

    _call, _num_pools = "pkv_attend_kv4", 1


class PromptStep(_ContextCalls):
    """Causal attention of up to `num_tokens` new tokens, all rows together,
    over a 16-bit or 4-bit cache that already holds them.  Owns the output and
    the workspace, as ``WindowStep``.

    ``run`` takes q [num_tokens][Hq][d], tok_offsets [B + 1] (or None for one
    token per row), block_table, seq_lens and k_pool, v_pool or kv4_pool.
    """

    def __init__(self, prob: _lib.pkv_problem, num_tokens: int, window: int = 0, sinks: int = 0,
                 splits: int | None = None, device="cuda"):
        super().__init__(prob, device)
        self.view = _context.make_view(window, sinks)
        self.num_tokens = num_tokens
        if splits is None:
            splits = _context.pkv_prompt_splits(
                prob, self.view, num_tokens, False, torch.cuda.get_device_properties(
                    self.device).multi_processor_count)
        self.splits = splits
        nbytes = _context.pkv_prompt_workspace_bytes(prob, num_tokens, False, splits)
        if num_tokens == prob.batch:  # room for calls without tok_offsets too
            nbytes = max(nbytes, _context.pkv_prompt_workspace_bytes(prob, num_tokens, True,
                                                                     splits))
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self.out = torch.empty(num_tokens, prob.num_q_heads, prob.head_dim, dtype=self.dtype,
                               device=self.device)
        self.lse = torch.empty(num_tokens, prob.num_q_heads, dtype=torch.float32,
                               device=self.device)
        self._own_buffers(self.workspace, self.out, self.lse)
        self._view_ref = ctypes.byref(self.view)
        self._own = (self.workspace.data_ptr(), nbytes, self.out.data_ptr(), self.lse.data_ptr())

    def bind(self, w: dict, stream=None) -> tuple:
        n = self.num_tokens
        q = self._expect("q", w["q"], self.out.shape, self.dtype)
        table, lens = self._tables(w["block_table"], w["seq_lens"])
        pools = self._pools(w)
        return ("pkv_prompt_kv4" if len(pools) == 1 else "pkv_prompt_window", self._view_ref,
                self._offsets(w.get("tok_offsets"), n), n, lens, self.splits, q, *pools, table,
                *self._own,
                self._stream(stream))

    def run(self, w: dict, stream=None) -> tuple:
        return self.run_bound(self.bind(w, stream))

    def run_bound(self, bound: tuple) -> tuple:
        self._launch(*bound)
        return self.out, self.lse


def load_policy_table(path: str = POLICY_TABLE_PATH):
    """Rules [(b_lo, b_hi, nmax_lo, nmax_hi, path_id, splits)] from the JSON table."""
    with open(path) as f:
        doc = json.load(f)
    return [(r["b_lo"], r["b_hi"], r["nmax_lo"], r["nmax_hi"], PATH_IDS[r["path"]], r["splits"])
            for r in doc["rules"]]


def choose(rules, batch: int, max_len: int):
    """Path name and split cap from the calibrated table (C-ABI pkv_policy)."""
    path, splits = pkv_policy(rules, batch, max_len)
    return PATH_NAMES[path], splits


def split_kernel_of(prob: _lib.pkv_problem) -> str:
    """The split-kernel variant pkv_decode runs for this problem: the explicit
    choice, else the library's AUTO rule (matrix cores for d = 128, vector ALU
    for 64).  The matrix-core kernel for G > 8 is a variant of its own (two
    resident workgroups per CU instead of three, deeper prefetch), with its
    own cost model."""
    if prob.kernel == _lib.PKV_KERNEL_VALU or (prob.kernel == _lib.PKV_KERNEL_AUTO
                                               and prob.head_dim != 128):
        return "valu"
    return "mfma" if prob.num_q_heads // prob.num_kv_heads <= 8 else "mfma_g16"


def load_cost_model(path: str = COST_MODEL_PATH):
    """(candidates [(path_id, splits)], {split kernel: weights [4][PKV_COST_FEATURES]},
    num_cus).  The model has one weight matrix per split kernel."""
    with open(path) as f:
        doc = json.load(f)
    cands = [(PATH_IDS[c["path"]], c["splits"]) for c in doc["candidates"]]
    weights = {}
    for kernel, rows in doc["weights"].items():
        w = np.zeros((4, _lib.PKV_COST_FEATURES), dtype=np.float32)
        for name, row in rows.items():
            w[PATH_IDS[name]] = np.asarray(row, dtype=np.float32)
        weights[kernel] = w
    return cands, weights, int(doc["num_cus"])


def choose_model(model, prob: _lib.pkv_problem, seq_lens_host):
    """Path name, split cap and predicted µs from the learned cost model
    (C-ABI pkv_policy_model, with the weights of the problem's split kernel)."""
    cands, weights, num_cus = model
    path, splits, pred = _lib.pkv_policy_model(prob, cands, weights[split_kernel_of(prob)],
                                               num_cus, seq_lens_host)
    return PATH_NAMES[path], splits, pred


# Candidates of the default policy's cost-model leg (B >= 2): the compact
# workqueue at each split cap, and the single-pass kernel.  On the calibration
# and held-out draws of every sweep and trace workload the full candidate list
# picks the same (path, split cap) at B >= 2, at a third of the host time.
DEFAULT_MODEL_PATHS = (PKV_WORKQUEUE, PKV_NOSPLIT)


def choose_default(rules, model, prob: _lib.pkv_problem, seq_lens_host):
    """Path name and split cap of the engine's default policy
    (pkv_policy_default): the calibrated table for one row, the learned cost
    model (workqueue and no-split candidates, and the CU-balanced workqueue
    caps the library adds) for several."""
    cands, weights, num_cus = model
    cands = [c for c in cands if c[0] in DEFAULT_MODEL_PATHS]
    path, splits = _lib.pkv_policy_default(rules, prob, cands, weights[split_kernel_of(prob)],
                                           num_cus, seq_lens_host)
    return PATH_NAMES[path], splits


def validate_inputs(w: dict) -> None:
    """Host-side checks that the tensors match what the kernels assume.

    Shapes, dtypes and contiguity of q / pools / block table / lengths, every
    length within the table's capacity, and every block-table entry that a
    row uses inside [0, num_pool_pages).  Raises ValueError.
    """
    spec = w["spec"]
    q, kp, vp, bt, sl = w["q"], w["k_pool"], w["v_pool"], w["block_table"], w["seq_lens"]
    dt = TORCH_DTYPE[spec.dtype]
    b, hq, hkv, d, p = (spec.batch, spec.num_q_heads, spec.num_kv_heads, spec.head_dim,
                        spec.page_size)
    if tuple(q.shape) != (b, hq, d) or q.dtype != dt:
        raise ValueError(f"q: {tuple(q.shape)} {q.dtype}")
    for name, t in (("k_pool", kp), ("v_pool", vp)):
        if t.dim() != 4 or tuple(t.shape[1:]) != (hkv, p, d) or t.dtype != dt:
            raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype}")
    if kp.shape[0] != vp.shape[0]:
        raise ValueError("K and V pools differ in page count")
    if bt.dim() != 2 or bt.shape[0] != b or bt.dtype != torch.int32:
        raise ValueError(f"block_table: {tuple(bt.shape)} {bt.dtype}")
    if tuple(sl.shape) != (b,) or sl.dtype != torch.int32:
        raise ValueError(f"seq_lens: {tuple(sl.shape)} {sl.dtype}")
    for t in (q, kp, vp, bt, sl):
        if not t.is_contiguous():
            raise ValueError("inputs must be contiguous")
    lens = sl.cpu().numpy()
    btn = bt.cpu().numpy()
    cap = btn.shape[1] * p
    pool = kp.shape[0]
    for i, n in enumerate(lens):
        if n < 0 or n > cap:
            raise ValueError(f"row {i}: length {n} outside [0, {cap}]")
        used = btn[i, :(int(n) + p - 1) // p]
        if used.size and (used.min() < 0 or used.max() >= pool):
            raise ValueError(f"row {i}: block-table entry outside [0, {pool})")
