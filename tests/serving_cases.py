"""Inputs of the serving-operator tests (not a test module).  Bounds are those of
tests/context_cases.py: the kernels multiply the values that the codes stand for,
which are exact in 16 bits."""
from __future__ import annotations

import numpy as np
import torch

from oracle import serving as sv
from tests.context_cases import Batch, f64


class Batch8(Batch):
    """``Batch`` over the 8-bit cache: tokens that no query of their row sees and pages
    that no row uses hold NaN codes, unused pages a scale byte of all ones too.  Rows
    are quantised page by page, as stored at once."""

    def __init__(self, seed, lens, new=None, *, everything=False, **kw):
        window, sinks = kw.get("window", 0), kw.get("sinks", 0)
        super().__init__(seed, lens, new, **kw)
        pool, hkv, _, d = self.kp.shape
        self.cache = sv.Cache8(pool, hkv, d, self.dtype)
        self.cache.codes[:] = np.where(np.arange(d) % 2, 0x7f, 0xff)
        self.cache.scales[:] = 255
        self.vmax = 0.0
        from oracle.context import sees
        for i, n in enumerate(self.lens):
            if n == 0:
                continue
            x = np.stack(self.kv[i], 1)  # [n][2][hkv][d]
            y = np.zeros_like(x)
            first = max(int(n - self.new[i]), 0)
            for at in range(0, n, 16):
                page, m = int(self.table[i, at // 16]), min(16, n - at)
                self.cache.store(page, 0, x[at:at + m])
                for s in range(m):
                    y[at + s] = self.cache.values(page, s)
                    t = at + s
                    if not everything and not any(sees(p, t, window, sinks)
                                                  for p in {first, max(t, first)} if p < n):
                        self.cache.codes[page, :, :, s] = 0x7f
            self.kv[i] = (y[:, 0], y[:, 1])
            self.vmax = max(self.vmax, float(np.abs(y[:, 1]).max()))
        self.pool8, self.scales8 = self.cache.bytes(), self.cache.scales.copy()

    def device(self):
        w = super().device()
        del w["k_pool"], w["v_pool"]
        w["kv8_pool"] = torch.from_numpy(self.pool8.copy()).cuda()
        w["kv8_scales"] = torch.from_numpy(self.scales8.copy()).cuda()
        return w


def make_cross(kind, seed, lens, queries, *, hkv=2, group=4, d=128, dtype="f16", scale=None,
               spread=1.0):
    """A batch of encoder states, `lens` of them, in pages of `kind` (16, 4 or 8 bits),
    with `queries` of each row.  Poison behind a row's states and in unused pages."""
    cls = Batch8 if kind == 8 else Batch
    lens = np.asarray(lens)
    # Every state is visible: the batch is built as if all were queries, then gets its own.
    b = cls(seed, lens, lens, hkv=hkv, group=group, d=d, dtype=dtype, kv4=kind == 4, scale=scale,
            spread=spread)
    rng = np.random.default_rng(seed + 1)
    b.new = np.asarray(queries, dtype=np.int64)
    b.q = torch.from_numpy(rng.standard_normal(
        (int(b.new.sum()), hkv * group, d), dtype=np.float32)).to(b.q.dtype)
    return b


def cross_reference(b, lens=None, present=None):
    """Oracle outputs of ``make_cross``'s batch, token-major, as Batch.reference."""
    lens = b.lens if lens is None else lens
    parts, at = [], 0
    for i, n in enumerate(lens):
        m = int(b.new[i])
        q = f64(b.q[at:at + m])
        at += m
        k, v = b.kv[i]
        here = None
        if present is not None:
            here = np.array([present(i, t // 16) for t in range(n)], dtype=bool)
        parts.append(sv.cross_row(q, k[:n], v[:n], b.scale, here))
    return (np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts]),
            tuple(np.concatenate([p[2][j] for p in parts]) for j in range(3)))
