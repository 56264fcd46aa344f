"""CPU: the context operators' C ABI: exports, sizes, and every refusal; nothing
is launched."""
import ctypes
import os
import re

import pytest

from paged_kv_gqa_block_amd import _context, _lib
from paged_kv_gqa_block_amd._lib import (PKV_EDTYPE, PKV_EINVAL, PKV_ENOSPC, PKV_ERANGE, PKV_ESHAPE,
                                         PKV_OK)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "pkv_context.h")
pytestmark = pytest.mark.skipif(not hasattr(_lib.LIB, "pkv_attend_kv4"),
                                reason="this build holds the decode engine's host code only")
P = 4096  # any aligned address: refused calls read nothing


def _prob(**over):
    a = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
             num_pool_pages=64, max_pages_per_row=32, dtype="f16")
    a.update(over)
    return _lib.make_problem(**a)


def test_every_declared_symbol_is_exported_and_bound():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\b(pkv_\w+)\s*\(", text))
    assert declared == set(_context.EXPORTED)
    for name in declared:
        assert hasattr(_lib.LIB, name) and getattr(_lib.LIB, name).argtypes is not None, name


def test_page_bytes():
    assert _context.pkv_kv4_page_bytes(128) == 2176 and _context.pkv_kv4_page_bytes(64) == 1088
    assert all(_context.pkv_kv4_page_bytes(d) == 0 for d in (0, -64, 32, 96, 256))


def test_workspace_and_splits():
    p = _prob()
    one, four = (_context.pkv_attend_workspace_bytes(p, s) for s in (1, 4))
    slots = 2 * 2 * 4
    assert four >= slots * 4 * (128 + 2) * 4 and one < four
    for bad in (0, -1, 65536):
        assert _context.pkv_attend_workspace_bytes(p, bad) == 0
    assert _context.pkv_attend_workspace_bytes(_prob(head_dim=96), 1) == 0
    assert _context.pkv_attend_workspace_bytes(_prob(batch=65536), 1) == 0
    assert _context.pkv_attend_workspace_bytes(_prob(batch=65535), 65535) == 0
    # More rows, fewer ranges each; a narrow view needs no splitting at all.
    s = [_context.pkv_attend_splits(_prob(batch=b, max_pages_per_row=2048), None, 256)
         for b in (1, 8, 64, 1024)]
    assert s == sorted(s, reverse=True) and s[0] > 1 and s[-1] == 1
    narrow = _context.make_view(16, 0)
    assert _context.pkv_attend_splits(_prob(max_pages_per_row=2048), narrow, 256) == 1
    assert _context.pkv_attend_splits(_prob(), None, 0) == 0
    assert _context.pkv_attend_splits(_prob(), _context.make_view(-1, 0), 256) == 0


def test_prompt_workspace_and_splits():
    ws, sp = _context.pkv_prompt_workspace_bytes, _context.pkv_prompt_splits
    p = _prob(max_pages_per_row=2048)
    tiles = 10 * 4 // 128 + 2
    assert ws(p, 10, False, 1) == 0
    assert ws(p, 10, False, 3) >= tiles * 2 * 3 * 128 * (128 + 2) * 4
    assert ws(p, 2, True, 3) >= 2 * 2 * 3 * 128 * (128 + 2) * 4
    assert ws(p, 3, True, 3) == 0 and ws(p, -1, False, 3) == 0 and ws(p, 10, False, 0) == 0
    assert ws(p, 2 ** 31 - 1, False, 2) == 0
    s = [sp(p, None, n, False, 256) for n in (1, 100, 10000, 100000)]
    assert s == sorted(s, reverse=True) and s[0] > 1 and s[-1] == 1
    assert sp(p, _context.make_view(16, 0), 10, False, 256) == 1
    assert sp(p, None, 0, False, 256) >= 1 and sp(p, None, 10, False, 0) == 0
    assert sp(p, _context.make_view(-1, 0), 10, False, 256) == 0 and sp(p, None, 3, True, 256) == 0


def _attend(kv4=False, prob=None, view=None, lens=P, splits=4, q=P, k=P, v=P, bt=P, ws=P,
            ws_bytes=1 << 30, out=P, lse=None):
    prob = prob or _prob()
    view = None if view is None else ctypes.byref(_context.make_view(*view))
    head = (ctypes.byref(prob), view, lens, splits, q)
    tail = (bt, ws, ws_bytes, out, lse, None)
    if kv4:
        return _lib.LIB.pkv_attend_kv4(*head, k, *tail)
    return _lib.LIB.pkv_attend_window(*head, k, v, *tail)


@pytest.mark.parametrize("kv4", [False, True])
def test_attend_refusals(kv4):
    for name in ("lens", "q", "k", "bt", "ws", "out"):
        assert _attend(kv4, **{name: None}) == PKV_EINVAL, name
    if not kv4:
        assert _attend(v=None) == PKV_EINVAL
        assert _attend(v=P + 8) == PKV_ESHAPE
    for name in ("q", "k", "ws", "out"):
        assert _attend(kv4, **{name: P + 8}) == PKV_ESHAPE, name
    assert _attend(kv4, view=(-1, 0)) == PKV_EINVAL
    assert _attend(kv4, view=(4, -1)) == PKV_EINVAL
    for s in (0, -4, 65536):
        assert _attend(kv4, splits=s) == PKV_EINVAL
    assert _attend(kv4, ws_bytes=64) == PKV_ENOSPC
    need = _context.pkv_attend_workspace_bytes(_prob(), 4)
    assert _attend(kv4, ws_bytes=need - 1) == PKV_ENOSPC
    assert _attend(kv4, prob=_prob(batch=65536)) == PKV_ERANGE
    assert _attend(kv4, prob=_prob(batch=65535), splits=65535) == PKV_ERANGE
    assert _attend(kv4, prob=_prob(num_q_heads=65536, num_kv_heads=8192)) == PKV_ERANGE
    assert _attend(kv4, prob=_prob(head_dim=96)) == PKV_ESHAPE
    assert _attend(kv4, prob=_prob(num_q_heads=34)) == PKV_ESHAPE  # G = 17
    assert _attend(kv4, prob=_prob(page_size=32)) == PKV_ESHAPE
    assert _attend(kv4, prob=_prob(dtype=7)) == PKV_EDTYPE
    assert _attend(kv4, prob=_prob(batch=0)) == PKV_EINVAL


def _prompt(kv4=False, prob=None, view=None, off=P, n=10, lens=P, splits=1, q=P, k=P, v=P, bt=P,
            ws=None, ws_bytes=0, out=P):
    prob = prob or _prob()
    view = None if view is None else ctypes.byref(_context.make_view(*view))
    head, tail = (ctypes.byref(prob), view, off, n, lens, splits, q), (ws, ws_bytes, out, None, None)
    if kv4:
        return _lib.LIB.pkv_prompt_kv4(*head, k, bt, *tail)
    return _lib.LIB.pkv_prompt_window(*head, k, v, bt, *tail)


@pytest.mark.parametrize("kv4", [False, True])
def test_prompt_refusals(kv4):
    for name in ("lens", "q", "k", "bt", "out"):
        assert _prompt(kv4, **{name: None}) == PKV_EINVAL, name
    assert _prompt(kv4, n=-1) == PKV_EINVAL
    assert _prompt(kv4, off=None) == PKV_EINVAL  # ten tokens of two rows
    assert _prompt(kv4, view=(-1, 0)) == PKV_EINVAL
    assert _prompt(kv4, view=(0, -1)) == PKV_EINVAL
    for name in ("q", "k", "out"):
        assert _prompt(kv4, **{name: P + 2}) == PKV_ESHAPE, name
    assert _prompt(kv4, n=2 ** 31 - 1) == PKV_ERANGE
    for s in (0, -1, 65536):
        assert _prompt(kv4, splits=s) == PKV_EINVAL
    assert _prompt(kv4, splits=2) == PKV_EINVAL  # needs a workspace
    assert _prompt(kv4, splits=2, ws=P + 8, ws_bytes=1 << 30) == PKV_ESHAPE
    need = _context.pkv_prompt_workspace_bytes(_prob(), 10, False, 2)
    assert need > 0 and _prompt(kv4, splits=2, ws=P, ws_bytes=need - 1) == PKV_ENOSPC
    assert _prompt(kv4, splits=65535, n=8000, ws=P, ws_bytes=1 << 60) == PKV_ERANGE
    assert _prompt(kv4, n=0) == PKV_OK
    assert _prompt(kv4, n=0, prob=_prob(head_dim=80)) == PKV_ESHAPE


def _store(kv4=True, prob=None, off=P, n=10, lens=P, k=P, ks=256, v=P, vs=256, bt=P, pool=P,
           vpool=P):
    prob = prob or _prob()
    head = (ctypes.byref(prob), off, n, lens, k, ks, v, vs, bt, pool)
    return _lib.LIB.pkv_kv4_store(*head, None) if kv4 else _lib.LIB.pkv_store_kv(*head, vpool, None)


@pytest.mark.parametrize("kv4", [False, True])
def test_store_refusals(kv4):
    for name in ("lens", "k", "v", "bt", "pool"):
        assert _store(kv4, **{name: None}) == PKV_EINVAL, name
    if not kv4:
        assert _store(False, vpool=None) == PKV_EINVAL
    assert _store(kv4, n=-1) == PKV_EINVAL
    assert _store(kv4, off=None) == PKV_EINVAL
    for stride in (255, 248, 260, 0, -256):
        assert _store(kv4, ks=stride) == PKV_ESHAPE, stride
        assert _store(kv4, vs=stride) == PKV_ESHAPE, stride
    for name in ("k", "v", "pool"):
        assert _store(kv4, **{name: P + 4}) == PKV_ESHAPE, name
    big = _prob(num_q_heads=512, num_kv_heads=512)
    assert _store(kv4, prob=big, ks=1 << 16, vs=1 << 16, n=2 ** 31 - 1) == PKV_ERANGE
    assert _store(kv4, n=0) == PKV_OK


def test_load_refusals():
    def load(prob=None, off=P, n=10, lens=P, bt=P, pool=P, k=P, v=P):
        prob = prob or _prob()
        return _lib.LIB.pkv_kv4_load(ctypes.byref(prob), off, n, lens, bt, pool, k, v, None)

    for name in ("lens", "bt", "pool", "k", "v"):
        assert load(**{name: None}) == PKV_EINVAL, name
    for name in ("pool", "k", "v"):
        assert load(**{name: P + 8}) == PKV_ESHAPE, name
    assert load(n=-2) == PKV_EINVAL and load(off=None) == PKV_EINVAL
    assert load(prob=_prob(num_q_heads=512, num_kv_heads=512), n=2 ** 31 - 1) == PKV_ERANGE
    assert load(n=0) == PKV_OK


def test_token_strides_are_checked_by_the_binding():
    import torch

    x = torch.zeros(4, 2, 3, 64)
    assert _context.token_stride(x[:, 0]) == 2 * 3 * 64
    assert _context.token_stride(torch.zeros(1, 3, 64)) == 192
    with pytest.raises(ValueError):
        _context.token_stride(x.transpose(1, 2)[:, 0])
    with pytest.raises(ValueError):
        _context.token_stride(x[..., ::2][:, 0])


@pytest.mark.parametrize("kv4", [False, True])
def test_counters_of_split_calls(kv4):
    """Pairs of row (or tile) and KV head in splits: one counter each, 65536 of
    them, at one place for every problem; one split takes none."""
    many = _prob(batch=9000, num_q_heads=8, num_kv_heads=8)
    assert _attend(kv4, prob=many, ws_bytes=1 << 60) == PKV_ERANGE
    assert _context.pkv_attend_workspace_bytes(many, 4) == 0
    assert _context.pkv_attend_workspace_bytes(many, 1) > 0
    assert _prompt(kv4, splits=2, n=1 << 20, ws=P, ws_bytes=1 << 60,
                   prob=_prob(num_q_heads=8, num_kv_heads=8)) == PKV_ERANGE  # 65552 pairs
    assert _context.pkv_attend_workspace_bytes(_prob(), 4) >= (256 << 10) + 16 * 4 * 130 * 4
    assert (_context.pkv_prompt_workspace_bytes(_prob(), 10, False, 3)
            >= (256 << 10) + 2 * 2 * 3 * 128 * 130 * 4)


def test_split_caps_over_the_whole_range():
    """No sizes, zero tokens and one row among them, end in anything but a cap
    that the call accepts."""
    for b in (1, 2, 3, 65, 65535):
        for hq, hkv in ((1, 1), (16, 1), (8, 8), (64, 8), (4096, 4096)):
            for pages in (1, 7, 41, 2048, (2 ** 31 - 1) // 16):
                p = _prob(batch=b, num_q_heads=hq, num_kv_heads=hkv, max_pages_per_row=pages)
                for view in (None, _context.make_view(1, 0), _context.make_view(2 ** 31 - 1, 5)):
                    for cus in (1, 256, 1024):
                        s = _context.pkv_attend_splits(p, view, cus)
                        assert 1 <= s <= 1024
                        assert s == 1 or b * hkv <= 65536
                        for n in (0, 1, 2, 127, 129, 5000):
                            s = _context.pkv_prompt_splits(p, view, n, False, cus)
                            assert 1 <= s <= 2048
                            assert s == 1 or _context.pkv_prompt_workspace_bytes(p, n, False, s)
                        assert _context.pkv_prompt_splits(p, view, b, True, cus) >= 1
