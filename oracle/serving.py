"""The 8-bit cache, cross attention and page tables, in fp64 numpy and plain
Python.

Written from the definitions in include/pkv_serving.h: a block is 16 tokens (one
page) by d channels of one KV head, K and V apart, e4m3 codes and one
power-of-two scale; page tables take from and give back to a stack of free pages.
"""
from __future__ import annotations

import math

import numpy as np

EXP8 = {"f16": (-15, 7), "bf16": (-117, 119)}
TOP8 = 448.0


def _e4m3(code: int) -> float:
    sign = -1.0 if code & 128 else 1.0
    exp, mant = (code >> 3) & 15, code & 7
    if exp == 15 and mant == 7:
        return math.nan
    if exp == 0:
        return sign * mant * 2.0 ** -9
    return sign * (1 + mant / 8) * 2.0 ** (exp - 7)


E4M3 = np.array([_e4m3(c) for c in range(256)])


def exponent_for(top: float, dtype: str) -> int:
    """The smallest exponent e with top <= 448 * 2^e, kept in the type's range."""
    lo, hi = EXP8[dtype]
    e = lo
    while e < hi and top > TOP8 * 2.0 ** e:
        e += 1
    return e


def e4m3_round(y):
    """Codes of |y| and signs: nearest, ties to the even code, 448 at most; what is
    not finite becomes 127 (a NaN)."""
    y = np.asarray(y, dtype=np.float64)
    mag = np.abs(y)
    grid = E4M3[:127]  # 0 .. 448, increasing
    mids = (grid[1:] + grid[:-1]) / 2
    fine = np.isfinite(mag)
    m = np.where(fine, mag, 0)
    code = np.searchsorted(mids, m, side="left")  # mids below m
    at_tie = np.isin(m, mids)
    tie = np.searchsorted(mids, m, side="left")  # m == mids[tie]: codes tie, tie + 1
    code = np.where(at_tie, tie + tie % 2, code)
    code = np.where(fine, code, 127)
    return (code | (np.signbit(y) << 7)).astype(np.uint8)


def kv8_values(codes, exponents):
    """What codes [..., 16, d] at block exponents [...] stand for."""
    return E4M3[codes] * np.ldexp(1.0, np.asarray(exponents, dtype=np.int64))[..., None, None]


class Cache8:
    """Logical contents of an 8-bit cache: codes [pages][Hkv][2][16][d] and scale bytes
    [pages][Hkv][2]."""

    def __init__(self, pages, hkv, d, dtype):
        self.codes = np.zeros((pages, hkv, 2, 16, d), dtype=np.uint8)
        self.scales = np.zeros((pages, hkv, 2), dtype=np.uint8)
        self.dtype = dtype

    def store(self, page: int, slot: int, x):
        """Tokens x [n][2][Hkv][d] of one run into the page's slots from `slot` on."""
        n, _, hkv, _ = x.shape
        for h in range(hkv):
            for kv in range(2):
                z = x[:, kv, h]
                fine = np.abs(z[np.isfinite(z)])
                e = exponent_for(fine.max(initial=0.0), self.dtype)
                if slot:
                    was = int(self.scales[page, h, kv]) - 127
                    if was > e:
                        e = was
                    if e > was:
                        old = self.codes[page, h, kv, :slot]
                        self.codes[page, h, kv, :slot] = e4m3_round(
                            E4M3[old] * 2.0 ** (was - e))
                self.codes[page, h, kv, slot:slot + n] = e4m3_round(z / 2.0 ** e)
                self.scales[page, h, kv] = e + 127

    def values(self, page: int, slot: int):
        """What the page's token `slot` stands for, [2][Hkv][d]."""
        e = self.scales[page].astype(np.int64) - 127
        return np.moveaxis(E4M3[self.codes[page, :, :, slot]] * np.ldexp(1.0, e)[..., None], 1, 0)

    def bytes(self):
        """The pool's bytes [pages][Hkv][32 d]."""
        pages, hkv, _, _, d = self.codes.shape
        out = np.zeros((pages, hkv, 32 * d), dtype=np.uint8)
        for kv, at in enumerate(kv8_places(d)):
            out[..., at] = self.codes[:, :, kv]
        return out


def kv8_places(d: int):
    """Where a page of one KV head (32 d bytes) keeps token t, channel ch: int arrays
    [16][d] of bytes for K and for V."""
    k, v = np.zeros((16, d), dtype=np.int64), np.zeros((16, d), dtype=np.int64)
    per = 256 // d  # V tokens in a lane's 16 bytes
    for t in range(16):
        for ch in range(d):
            block, kg, j = ch // 32, ch % 32 // 8, ch % 8
            lane = 16 * kg + t
            k[t, ch] = block // 2 * 1024 + lane * 16 + block % 2 * 8 + j
            col, j = ch // (d // 16), ch % (d // 16)
            lane = 16 * (t // 4) + col
            v[t, ch] = 16 * d + t % 4 // per * 1024 + lane * 16 + t % 4 % per * (d // 16) + j
    return k, v


def cross_row(q, k, v, scale, present=None):
    """Every query of q [m][Hq][d] over all of k, v [n][Hkv][d]: as
    oracle.context.attend_row."""
    from .context import attend_row

    n = k.shape[0]
    if n == 0:
        m, hq, d = q.shape
        return (np.zeros((m, hq, d)), np.full((m, hq), -np.inf),
                (np.zeros((m, hq, d)), np.zeros((m, hq)), np.zeros(m, dtype=np.int64)))
    return attend_row(q, [n - 1] * q.shape[0], k, v, scale, 0, 0, present)


class Pages:
    """Page tables: lens, table [B][width] and the stack of free pages, as Python
    lists."""

    def __init__(self, lens, table, free, pool, width):
        self.lens = [int(x) for x in lens]
        self.table = [[int(x) for x in row] for row in table]
        self.free = [int(x) for x in free]  # the last is on top
        self.pool, self.width = pool, width

    def take(self, counts, num_tokens):
        """(seq_lens, tok_offsets, slots, positions, rows turned down) of a step; slots
        and positions of its tokens alone."""
        cap = self.width * 16
        seq, off, slots, positions, denied = [], [0], {}, {}, 0
        total, asked, have = 0, 0, len(self.free)
        for r, c in enumerate(max(int(c), 0) for c in counts):
            first, total = total, total + c
            off.append(min(total, num_tokens))
            n = self.lens[r]
            ok = 0 <= n <= cap and n + c <= cap and (c == 0 or total <= num_tokens)
            need = -(-(n + c) // 16) + -n // 16 if ok else 0
            asked += need
            ok = ok and (need == 0 or asked <= have)
            if ok:
                for i in range(need):
                    self.table[r][-(-n // 16) + i] = self.free.pop()
                self.lens[r] = n + c
            elif c:
                denied += 1
            seq.append(n + c if ok else 0)
            for j in range(min(c, max(0, num_tokens - first))):
                page = self.table[r][(n + j) // 16] if ok else -1
                slots[first + j] = page * 16 + (n + j) % 16 if 0 <= page < self.pool else -1
                positions[first + j] = n + j if ok else -1
        return seq, off, slots, positions, denied

    def release(self, keep):
        room = self.pool - len(self.free)  # taken by numbers outside the pool too
        for r in reversed(range(len(self.lens))):
            n, k = self.lens[r], int(keep[r])
            if not 0 <= n <= self.width * 16 or k < 0 or k >= n:
                continue
            for e in reversed(range(-(-k // 16), -(-n // 16))):
                if room > 0 and 0 <= self.table[r][e] < self.pool:
                    self.free.append(self.table[r][e])
                self.table[r][e] = -1
                room -= 1
            self.lens[r] = k
