"""Windowed and prompt attention and the 4-bit cache, in fp64 numpy.

Written from the definitions in include/pkv_context.h: a query at position p
sees token t when t <= p and (window == 0 or t > p - window or t < sinks); a
4-bit block is 32 channels of one token and KV head, a power-of-two scale and
e2m1 elements.  Unseen tokens are left out of every sum, so they may hold
anything.
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EXP = {"f16": (-23, 13), "bf16": (-120, 125)}


def sees(p: int, t, window: int, sinks: int):
    """Whether the query at position p sees token(s) t."""
    t = np.asarray(t)
    return (t <= p) & ((window == 0) | (t > p - window) | (t < sinks))


def attend_row(q, positions, k, v, scale, window=0, sinks=0, present=None):
    """One row: q [m][Hq][d] at `positions`, k, v [n][Hkv][d]; `present` [n]
    marks tokens that exist (all by default).  Returns out [m][Hq][d], lse
    [m][Hq] and, per query, (sum of softmax weight times |v|, largest
    sum_c |q_c k_c| of a seen token, seen tokens): the scales of its rounding
    errors."""
    m, hq, d = q.shape
    n, hkv = k.shape[0], k.shape[1]
    grp = hq // hkv
    out = np.zeros((m, hq, d))
    lse = np.full((m, hq), -np.inf)
    mag = np.zeros((m, hq, d))
    score_mag = np.zeros((m, hq))
    count = np.zeros(m, dtype=np.int64)
    for i, p in enumerate(positions):
        seen = sees(p, np.arange(n), window, sinks)
        if present is not None:
            seen &= present
        idx = np.flatnonzero(seen)
        count[i] = idx.size
        if not idx.size:
            continue
        for g in range(hkv):
            kk, vv = k[idx, g], v[idx, g]
            for h in range(g * grp, (g + 1) * grp):
                x = (kk @ q[i, h]) * scale
                top = x.max()
                w = np.exp(x - top)
                l = w.sum()
                out[i, h] = (w @ vv) / l
                lse[i, h] = top + math.log(l)
                mag[i, h] = (w @ np.abs(vv)) / l
                score_mag[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, (mag, score_mag, count)


def kv4_quantise(x, dtype: str):
    """x [..., d] (fp64 values of the 16-bit type) -> (codes uint8 [..., d],
    scale bytes uint8 [..., d/32])."""
    z = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    codes = np.zeros(z.shape, dtype=np.uint8)
    scales = np.zeros(z.shape[:-1], dtype=np.uint8)
    for i in np.ndindex(*z.shape[:-1]):
        b = z[i]
        if not np.isfinite(b).all():
            scales[i] = 255
            continue
        top = np.abs(b).max()
        e = EXP[dtype][0]
        if top > 0:
            _, ex = math.frexp(top)  # top = f * 2^ex with f in [0.5, 1)
            own = ex - 1 - 2
            if top > 7 * 2.0 ** own:
                own += 1
            e = min(max(e, own), EXP[dtype][1])
        scales[i] = e + 127
        y = np.abs(b) / 2.0 ** e
        best = np.zeros(32, dtype=np.uint8)
        for c in range(1, 8):
            mid = (E2M1[c - 1] + E2M1[c]) / 2
            up = (y > mid) | ((y == mid) & (c % 2 == 0))  # ties to the even code
            best[up] = c
        codes[i] = best | (np.signbit(b).astype(np.uint8) << 3)
    return codes.reshape(x.shape), scales


def kv4_values(codes, scales):
    """The values that codes [..., d] and scale bytes [..., d/32] stand for, in
    fp64."""
    mag = np.array(E2M1)[codes & 7]
    val = np.where(codes & 8, -mag, mag).reshape(*scales.shape, 32)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (val * s[..., None]).reshape(codes.shape)


def kv4_places(d: int):
    """Where a page of one KV head (17 d bytes) keeps token t, channel ch:
    dicts (t, ch) -> (byte, nibble) for K and V, (t, block) -> byte for their
    scales."""
    k, v, ks, vs = {}, {}, {}, {}
    for t in range(16):
        for ch in range(d):
            block, kg, j = ch // 32, ch % 32 // 8, ch % 8
            lane = 16 * kg + t
            k[t, ch] = (lane * (d // 8) + 4 * block + j // 2, j % 2)
            col, j = ch // (d // 16), ch % (d // 16)
            lane = 16 * (t // 4) + col
            v[t, ch] = (8 * d + lane * (d // 8) + t % 4 * (d // 32) + j // 2, j % 2)
        for block in range(d // 32):
            ks[t, block] = 16 * d + t * (d // 32) + block
            vs[t, block] = 16 * d + d // 2 + t // 4 * (d // 8) + block * 4 + t % 4
    return k, v, ks, vs


def kv4_write(page, t: int, codes, scales, which: str):
    """Put token t's codes [d] and scale bytes [d/32] of K or V into a page's
    bytes, in place."""
    d = codes.shape[0]
    k, v, ks, vs = kv4_places(d)
    at, sc = (k, ks) if which == "k" else (v, vs)
    for ch in range(d):
        b, nib = at[t, ch]
        page[b] = (page[b] & (0x0F if nib else 0xF0)) | (int(codes[ch]) << (4 * nib))
    for block in range(d // 32):
        page[sc[t, block]] = scales[block]


def kv4_read(page, which: str):
    """Codes [16][d] and scale bytes [16][d/32] of K or V of a page's bytes."""
    d = page.shape[0] // 17
    k, v, ks, vs = kv4_places(d)
    at, sc = (k, ks) if which == "k" else (v, vs)
    codes = np.zeros((16, d), dtype=np.uint8)
    scales = np.zeros((16, d // 32), dtype=np.uint8)
    for (t, ch), (b, nib) in at.items():
        codes[t, ch] = (page[b] >> (4 * nib)) & 15
    for (t, block), b in sc.items():
        scales[t, block] = page[b]
    return codes, scales
