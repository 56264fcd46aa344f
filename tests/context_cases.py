"""Inputs, oracle outputs and error bounds of the context-operator tests (not a
test module).

Bounds.  With u = half a step of the output type (finfo.eps / 2), A = sum_t w_t
|v_t| over the softmax weights, S = the largest sum_c |scale q_c k_c| of a seen
token and n the seen tokens:
* a score is a sum of d products in fp32, off by at most (d + 4) 2^-24 S (the
  four: the scale, its product, the running maximum's subtraction, and the
  change of units);
* exp2 adds 2^-22, so a weight is off by a relative e_w = 2 ((d + 4) 2^-24 S) +
  2^-21 (numerator's exponent and the common maximum's), and the same again
  through the sum L;
* the weights enter P V with a relative u_p: two 16-bit parts in the decode
  kernels (u^2, at most 2^-16), one in the prompt kernel (u);
* sums of n terms in fp32: n 2^-24 worst case, twice (numerator and L);
* f16 parts of a weight below 2^-14 are subnormal: an absolute 2^-25 of the
  largest weight, n times, relative to L >= 1 and |v| <= V;
* the output is rounded once: u |out| plus half of f16's smallest subnormal.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import context as oc

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def out_bound(ref, mag, score_mag, count, vmax, d, dtype, one_part):
    u = U[dtype]
    e_w = 2 * (d + 4) * 2.0 ** -24 * score_mag + 2.0 ** -21
    u_p = u if one_part else u * u
    n = count.reshape(-1, 1, 1)
    rel = 2 * e_w[..., None] + u_p + 2 * n * 2.0 ** -24
    sub = n * 2.0 ** -25 * vmax if dtype == "f16" else 0.0
    return u * np.abs(ref) + 1.01 * rel * mag + sub + 2.0 ** -25


def lse_bound(ref, score_mag, count, d):
    fin = np.where(np.isfinite(ref), np.abs(ref), 0)
    return (d + 4) * 2.0 ** -24 * score_mag * 2 + 2.0 ** -20 + count.reshape(-1, 1) * 2.0 ** -24 + \
        2.0 ** -22 * fin


def check(got_out, got_lse, ref, dtype, d, vmax, one_part, label):
    out, lse, (mag, score_mag, count) = ref
    g, gl = f64(got_out), f64(got_lse)
    assert np.isfinite(g).all(), f"{label}: non-finite output"
    bound = out_bound(out, mag, score_mag, count, vmax, d, dtype, one_part)
    over = np.abs(g - out) / bound
    assert over.max(initial=0) <= 1, f"{label}: {over.max():.2f} of the bound"
    assert np.array_equal(np.isneginf(gl), np.isneginf(lse)), f"{label}: rows that see nothing"
    fin = np.isfinite(lse)
    if fin.any():
        lo = np.abs(gl[fin] - lse[fin]) / lse_bound(lse, score_mag, count, d)[fin]
        assert lo.max() <= 1, f"{label}: lse {lo.max():.2f} of the bound"
    norm = np.linalg.norm(out)
    if norm > 0:  # the rounding of outputs (and of P) averages out: well below a half step
        rel = np.linalg.norm(g - out) / norm
        assert rel <= U[dtype] * (1.5 if one_part else 1.0), f"{label}: rel-L2 {rel:.2e}"


class Batch:
    """A batch with a paged cache: row lengths `lens` after `new` tokens each.
    Every token that no query of its row sees, every page that no row uses and
    the table entries behind a row's pages hold poison (NaN, infinities; 4-bit:
    codes and scale bytes of all ones)."""

    def __init__(self, seed, lens, new=None, *, hkv=2, group=4, d=128, dtype="f16", window=0,
                 sinks=0, kv4=False, extra_pages=5, scale=None, spread=1.0):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        b = len(self.lens)
        self.new = np.ones(b, dtype=np.int64) if new is None else np.asarray(new, dtype=np.int64)
        self.hkv, self.group, self.d, self.dtype = hkv, group, d, dtype
        self.window, self.sinks, self.kv4 = window, sinks, kv4
        self.scale = float(np.float32(1 / np.sqrt(d) if scale is None else scale))
        t = TORCH[dtype]
        pages = -(-self.lens.astype(np.int64) // 16)
        width = max(1, int(pages.max(initial=0))) + 1
        pool = int(pages.sum()) + extra_pages
        perm = rng.permutation(pool)
        self.table = np.full((b, width), int(perm[-1]), dtype=np.int32)  # unused: poison
        at = 0
        for i, n in enumerate(pages):
            self.table[i, :n] = perm[at:at + n]
            at += n
        self.q = torch.from_numpy(rng.standard_normal(
            (int(self.new.sum()), hkv * group, d), dtype=np.float32)).to(t)
        self.kv = []  # per row: k, v [n][hkv][d] as fp64 values of the cache
        poison = np.array([np.nan, np.inf, -np.inf], dtype=np.float32)
        shape = (pool, hkv, 16, d)
        if kv4:
            self.pool4 = np.full((pool, hkv, 17 * d), 255, dtype=np.uint8)
        else:
            fill = torch.from_numpy(poison[rng.integers(0, 3, size=shape)]).to(t)
            self.kp, self.vp = fill.clone(), fill.clone()
        self.vmax = 0.0
        for i, n in enumerate(self.lens):
            k, v = (torch.from_numpy((rng.standard_normal((n, hkv, d), dtype=np.float32) * spread))
                    .to(t) for _ in range(2))
            if kv4:
                kc, ks = self._quick(f64(k))
                vc, vs = self._quick(f64(v))
                k64, v64 = oc.kv4_values(kc, ks), oc.kv4_values(vc, vs)
            else:
                k64, v64 = f64(k), f64(v)
            self.kv.append((k64, v64))
            if v64.size:
                self.vmax = max(self.vmax, float(np.abs(v64).max()))
            for tok in range(n):
                first = max(int(n - self.new[i]), 0)
                if not any(oc.sees(p, tok, window, sinks) for p in {first, max(tok, first)} if p < n):
                    continue  # unseen by every query: stays poison
                pg, slot = self.table[i, tok // 16], tok % 16
                if not kv4:
                    self.kp[pg, :, slot], self.vp[pg, :, slot] = k[tok], v[tok]
                    continue
                for h in range(hkv):
                    self._put(self.pool4[pg, h], slot, kc[tok, h], ks[tok, h], vc[tok, h],
                              vs[tok, h])

    _maps = {}

    def _quick(self, x):
        """oc.kv4_quantise for finite values, vectorised (pinned to it by a CPU
        test)."""
        z = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
        top = np.abs(z).max(-1)
        _, ex = np.frexp(top)
        e = ex - 3
        e = np.where(top > 7 * np.ldexp(1.0, e), e + 1, e)
        lo, hi = oc.EXP[self.dtype]
        e = np.clip(np.where(top > 0, e, lo), lo, hi)
        y = np.abs(z) / np.ldexp(1.0, e)[..., None]
        code = np.zeros(z.shape, dtype=np.uint8)
        for c in range(1, 8):
            mid = (oc.E2M1[c - 1] + oc.E2M1[c]) / 2
            code[(y > mid) | ((y == mid) & (c % 2 == 0))] = c
        return ((code | (np.signbit(z).astype(np.uint8) << 3)).reshape(x.shape),
                (e + 127).astype(np.uint8))

    def _put(self, page, slot, kc, ks, vc, vs):
        d = self.d
        if d not in self._maps:
            k, v, s, w = oc.kv4_places(d)
            self._maps[d] = [
                (np.array([[at[t, c][0] for c in range(0, d, 2)] for t in range(16)]),
                 np.array([[sc[t, b] for b in range(d // 32)] for t in range(16)]))
                for at, sc in ((k, s), (v, w))]
        for (at, sc), codes, scales in zip(self._maps[d], (kc, vc), (ks, vs)):
            page[at[slot]] = codes[0::2] | (codes[1::2] << 4)
            page[sc[slot]] = scales

    def problem(self, **over):
        from paged_kv_gqa_block_amd import engine

        pool = (self.pool4 if self.kv4 else self.kp).shape[0]
        a = dict(batch=len(self.lens), num_q_heads=self.hkv * self.group, num_kv_heads=self.hkv,
                 head_dim=self.d, page_size=16, num_pool_pages=pool,
                 max_pages_per_row=self.table.shape[1], dtype=self.dtype, sm_scale=self.scale)
        a.update(over)
        return engine.make_problem(**a)

    def device(self):
        w = {"q": self.q.cuda(), "block_table": torch.from_numpy(self.table.copy()).cuda(),
             "seq_lens": torch.from_numpy(self.lens.copy()).cuda(),
             "tok_offsets": torch.from_numpy(
                 np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)).cuda()}
        if self.kv4:
            w["kv4_pool"] = torch.from_numpy(self.pool4.copy()).cuda()
        else:
            w["k_pool"], w["v_pool"] = self.kp.cuda(), self.vp.cuda()
        return w

    def reference(self, lens=None, present=None):
        """Oracle outputs, token-major.  `lens` replaces the rows' lengths;
        present(row, page index) says whether a page exists."""
        lens = self.lens if lens is None else lens
        parts, at = [], 0
        for i, n in enumerate(lens):
            m = int(self.new[i])
            q = f64(self.q[at:at + m])
            at += m
            k, v = self.kv[i]
            here = None
            if present is not None:
                here = np.array([present(i, t // 16) for t in range(n)], dtype=bool)
            parts.append(oc.attend_row(q, range(n - m, n), k[:n], v[:n], self.scale, self.window,
                                       self.sinks, here))
        return (np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts]),
                tuple(np.concatenate([p[2][j] for p in parts]) for j in range(3)))
