"""CPU: the serving operators' C ABI: exports, sizes, and every refusal; nothing
is launched."""
import ctypes
import os
import re

import pytest

from paged_kv_gqa_block_amd import _lib, _serving
from paged_kv_gqa_block_amd._lib import (PKV_EDTYPE, PKV_EINVAL, PKV_ENOSPC, PKV_ERANGE, PKV_ESHAPE,
                                         PKV_OK)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "pkv_serving.h")
pytestmark = pytest.mark.skipif(not hasattr(_lib.LIB, "pkv_attend_kv8"),
                                reason="this build holds other host code only")
P = 4096  # any aligned address: refused calls read nothing
KINDS = [16, 4, 8]


def _prob(**over):
    a = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16,
             num_pool_pages=64, max_pages_per_row=32, dtype="f16")
    a.update(over)
    return _lib.make_problem(**a)


BAD_PROBLEMS = [(dict(head_dim=96), PKV_ESHAPE), (dict(num_q_heads=34), PKV_ESHAPE),
                (dict(page_size=32), PKV_ESHAPE), (dict(dtype=7), PKV_EDTYPE),
                (dict(batch=0), PKV_EINVAL)]


def test_every_declared_symbol_is_exported_and_bound():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = set(re.findall(r"\b(pkv_\w+)\s*\(", text))
    assert declared == set(_serving.EXPORTED)
    for name in declared:
        assert hasattr(_lib.LIB, name) and getattr(_lib.LIB, name).argtypes is not None, name


def test_page_bytes():
    assert _serving.pkv_kv8_page_bytes(128) == 4096 and _serving.pkv_kv8_page_bytes(64) == 2048
    assert all(_serving.pkv_kv8_page_bytes(d) == 0 for d in (0, -64, 32, 96, 256))


def _store(prob=None, off=P, n=10, lens=P, k=P, ks=256, v=P, vs=256, bt=P, pool=P, scales=P):
    return _lib.LIB.pkv_kv8_store(ctypes.byref(prob or _prob()), off, n, lens, k, ks, v, vs, bt,
                                  pool, scales, None)


def test_store_refusals():
    for name in ("lens", "k", "v", "bt", "pool", "scales"):
        assert _store(**{name: None}) == PKV_EINVAL, name
    assert _store(n=-1) == PKV_EINVAL and _store(off=None) == PKV_EINVAL
    for stride in (255, 248, 260, 0, -256):
        assert _store(ks=stride) == PKV_ESHAPE and _store(vs=stride) == PKV_ESHAPE, stride
    for name in ("k", "v", "pool"):
        assert _store(**{name: P + 8}) == PKV_ESHAPE, name
    assert _store(scales=P + 1) == PKV_ESHAPE
    big = _prob(num_q_heads=512, num_kv_heads=512)
    assert _store(prob=big, ks=1 << 16, vs=1 << 16, n=2 ** 31 - 1) == PKV_ERANGE
    for over, want in BAD_PROBLEMS:
        assert _store(prob=_prob(**over)) == want, over
    assert _store(n=0) == PKV_OK


def test_load_refusals():
    def load(prob=None, off=P, n=10, lens=P, bt=P, pool=P, scales=P, k=P, v=P):
        return _lib.LIB.pkv_kv8_load(ctypes.byref(prob or _prob()), off, n, lens, bt, pool, scales,
                                     k, v, None)

    for name in ("lens", "bt", "pool", "scales", "k", "v"):
        assert load(**{name: None}) == PKV_EINVAL, name
    for name in ("pool", "k", "v"):
        assert load(**{name: P + 8}) == PKV_ESHAPE, name
    assert load(scales=P + 1) == PKV_ESHAPE
    assert load(n=-2) == PKV_EINVAL and load(off=None) == PKV_EINVAL
    assert load(prob=_prob(num_q_heads=512, num_kv_heads=512), n=2 ** 31 - 1) == PKV_ERANGE
    assert load(n=0) == PKV_OK


def _attend(prob=None, view=None, lens=P, splits=4, q=P, k=P, scales=P, bt=P, ws=P,
            ws_bytes=1 << 30, out=P, lse=None):
    from paged_kv_gqa_block_amd import _context
    view = None if view is None else ctypes.byref(_context.make_view(*view))
    return _lib.LIB.pkv_attend_kv8(ctypes.byref(prob or _prob()), view, lens, splits, q, k, scales,
                                   bt, ws, ws_bytes, out, lse, None)


def test_attend_refusals():
    from paged_kv_gqa_block_amd import _context
    for name in ("lens", "q", "k", "scales", "bt", "ws", "out"):
        assert _attend(**{name: None}) == PKV_EINVAL, name
    for name in ("q", "k", "ws", "out"):
        assert _attend(**{name: P + 8}) == PKV_ESHAPE, name
    assert _attend(scales=P + 1) == PKV_ESHAPE
    assert _attend(view=(-1, 0)) == PKV_EINVAL and _attend(view=(4, -1)) == PKV_EINVAL
    for s in (0, -4, 65536):
        assert _attend(splits=s) == PKV_EINVAL
    need = _context.pkv_attend_workspace_bytes(_prob(), 4)
    assert _attend(ws_bytes=need - 1) == PKV_ENOSPC
    assert _attend(prob=_prob(batch=65536)) == PKV_ERANGE
    assert _attend(prob=_prob(batch=9000, num_kv_heads=8), ws_bytes=1 << 60) == PKV_ERANGE
    for over, want in BAD_PROBLEMS:
        assert _attend(prob=_prob(**over)) == want, over


def _prompt(prob=None, view=None, off=P, n=10, lens=P, splits=1, q=P, k=P, scales=P, bt=P, ws=None,
            ws_bytes=0, out=P):
    from paged_kv_gqa_block_amd import _context
    view = None if view is None else ctypes.byref(_context.make_view(*view))
    return _lib.LIB.pkv_prompt_kv8(ctypes.byref(prob or _prob()), view, off, n, lens, splits, q, k,
                                   scales, bt, ws, ws_bytes, out, None, None)


def test_prompt_refusals():
    for name in ("lens", "q", "k", "scales", "bt", "out"):
        assert _prompt(**{name: None}) == PKV_EINVAL, name
    assert _prompt(n=-1) == PKV_EINVAL and _prompt(off=None) == PKV_EINVAL
    assert _prompt(view=(-1, 0)) == PKV_EINVAL and _prompt(view=(0, -1)) == PKV_EINVAL
    for name in ("q", "k", "out"):
        assert _prompt(**{name: P + 2}) == PKV_ESHAPE, name
    assert _prompt(scales=P + 1) == PKV_ESHAPE
    assert _prompt(n=2 ** 31 - 1) == PKV_ERANGE
    assert _prompt(splits=2) == PKV_EINVAL  # needs a workspace
    assert _prompt(splits=2, ws=P, ws_bytes=1 << 10) == PKV_ENOSPC
    for over, want in BAD_PROBLEMS:
        assert _prompt(prob=_prob(**over)) == want, over
    assert _prompt(n=0) == PKV_OK


def test_prompt_shares():
    """Caps and workspaces of a prompt's even shares, over the whole range."""
    from paged_kv_gqa_block_amd import _context
    ws, sp = _serving.pkv_prompt_kv8_workspace_bytes, _serving.pkv_prompt_kv8_splits
    for b in (1, 2, 65, 65535):
        for hq, hkv in ((1, 1), (16, 1), (8, 8), (64, 8), (4096, 4096)):
            for pages in (1, 41, 2048, (2 ** 31 - 1) // 16):
                p = _prob(batch=b, num_q_heads=hq, num_kv_heads=hkv, max_pages_per_row=pages)
                for view in (None, _context.make_view(1, 0), _context.make_view(2 ** 31 - 1, 5)):
                    for n in (0, 1, 2, 129, 5000, 10 ** 6):
                        s = sp(p, view, n, False, 256)
                        assert 1 <= s <= 512 and (s == 1 or ws(p, n, False, s) > 0)
                    assert sp(p, view, b, True, 256) >= 1
    p = _prob(max_pages_per_row=2048)
    state = 256 * (128 // 2 + 2) * 4
    assert ws(p, 10, False, 3) == (256 << 10) + (2 + 3 - 1) * 2 * state
    assert ws(p, 2, True, 3) == (256 << 10) + (2 + 3 - 1) * 2 * state
    assert ws(p, 10, False, 1) == 0 and ws(p, 3, True, 3) == 0 and ws(p, -1, False, 3) == 0
    assert sp(p, None, 10, False, 0) == 0 and sp(p, _context.make_view(-1, 0), 10, False, 256) == 0


def _cross(kind, prob=None, off=P, n=10, lens=P, splits=1, q=P, k=P, v=P, bt=P, ws=None,
           ws_bytes=0, out=P):
    head = (ctypes.byref(prob or _prob()), off, n, lens, splits, q)
    tail = (bt, ws, ws_bytes, out, None, None)
    if kind == 4:
        return _lib.LIB.pkv_cross_kv4(*head, k, *tail)
    return (_lib.LIB.pkv_cross if kind == 16 else _lib.LIB.pkv_cross_kv8)(*head, k, v, *tail)


@pytest.mark.parametrize("n", [10, 1000])  # tiles of 16 queries, and of 128
@pytest.mark.parametrize("kind", KINDS)
def test_cross_refusals(kind, n):
    for name in ("lens", "q", "k", "bt", "out"):
        assert _cross(kind, n=n, **{name: None}) == PKV_EINVAL, name
    if kind != 4:
        assert _cross(kind, n=n, v=None) == PKV_EINVAL
        assert _cross(kind, n=n, v=P + 1) == PKV_ESHAPE
    for name in ("q", "k", "out"):
        assert _cross(kind, n=n, **{name: P + 8}) == PKV_ESHAPE, name
    assert _cross(kind, n=-1) == PKV_EINVAL and _cross(kind, n=n, off=None) == PKV_EINVAL
    for s in (0, -1, 65536):
        assert _cross(kind, n=n, splits=s) == PKV_EINVAL
    assert _cross(kind, n=n, splits=2) == PKV_EINVAL  # needs a workspace
    assert _cross(kind, n=n, splits=2, ws=P + 8, ws_bytes=1 << 40) == PKV_ESHAPE
    need = _serving.pkv_cross_workspace_bytes(_prob(), n, False, 2)
    assert need > 0 and _cross(kind, n=n, splits=2, ws=P, ws_bytes=need - 1) == PKV_ENOSPC
    assert _cross(kind, n=2 ** 31 - 1) == PKV_ERANGE
    assert _cross(kind, n=n, splits=65535, ws=P, ws_bytes=1 << 60,
                  prob=_prob(num_q_heads=2048, num_kv_heads=1024)) == PKV_ERANGE
    for over, want in BAD_PROBLEMS:
        assert _cross(kind, n=n, prob=_prob(**over)) == want, over
    assert _cross(kind, n=0) == PKV_OK


def test_cross_sizes_over_the_whole_range():
    """No sizes end in anything but a split cap and a workspace that the call accepts."""
    ws, sp = _serving.pkv_cross_workspace_bytes, _serving.pkv_cross_splits
    for b in (1, 2, 65, 30000, 65535, 10 ** 6):
        for hq, hkv in ((1, 1), (16, 1), (8, 8), (64, 8), (4096, 4096)):
            for pages in (1, 41, 2048, (2 ** 31 - 1) // 16):
                p = _prob(batch=b, num_q_heads=hq, num_kv_heads=hkv, max_pages_per_row=pages)
                for n in (0, 1, 2, 33, 5000, 10 ** 6):
                    for cus in (1, 256, 1024):
                        s = sp(p, n, False, cus)
                        assert 1 <= s <= 2048
                        assert s == 1 or ws(p, n, False, s) > 0
                s = sp(p, b, True, 256)
                assert s >= 1 and (s == 1 or ws(p, b, True, s) > 0)
                assert sp(p, b + 1, True, 256) == 0
    p = _prob(max_pages_per_row=2048)
    assert ws(p, 10, False, 1) == 0 and ws(p, -1, False, 2) == 0 and ws(p, 3, True, 2) == 0
    assert ws(p, 10, False, 65536) == 0 and ws(_prob(head_dim=96), 10, False, 2) == 0
    assert sp(p, 10, False, 0) == 0 and sp(p, -1, False, 256) == 0
    assert sp(p, 10, False, 1025) == 0
    # Four queries of two rows over two KV heads: tiles of sixteen, a state for each query.
    assert ws(p, 4, False, 3) >= (256 << 10) + (4 * 4 // 16 + 2) * 2 * 3 * 16 * (128 + 2) * 4


# PKV_EHIP: every check is passed and there is no GPU to launch on.  (With one, nothing
# may be launched over these addresses: sizes alone are compared there.)
GPU = os.path.exists("/dev/kfd")


@pytest.mark.parametrize("kind", KINDS)
def test_a_workspace_does_for_every_smaller_step(kind):
    """Calls of any number of queries over the workspace of the largest, around the border
    between few and many, at fixed splits and at each step's own."""
    ws, sp = _serving.pkv_cross_workspace_bytes, _serving.pkv_cross_splits
    fell = 0
    for b, hq, hkv, d in ((8, 32, 8, 128), (1, 16, 1, 64), (5, 15, 5, 128), (40, 64, 8, 64)):
        p = _prob(batch=b, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, max_pages_per_row=2048)
        few = (64 if b * hkv <= 64 else 32) * b * hkv // hq  # the last call of few queries
        for splits in (2, 3, 17, 64):
            for most in (few - 1, few, few + 1, 2 * few, 40 * few):
                room = ws(p, most, False, splits)
                for n in {1, 2, b, few // 2, few - 1, few, few + 1, most}:
                    if n > most:
                        continue
                    fell += ws(p, n, False, splits) > room
                    for s in {2, splits, max(sp(p, n, False, 256), 2)} if n <= few else {splits}:
                        if not GPU:
                            got = _cross(kind, p, n=n, splits=s, ws=P, ws_bytes=room)
                            assert got == _lib.PKV_EHIP, (b, hq, n, s, most, splits)
                            got = _cross(kind, p, n=n, splits=s, ws=P,
                                         ws_bytes=min(ws(p, n, False, 2), room) - 1)
                            assert got == PKV_ENOSPC or n > few, (b, hq, n, s, most, splits)
    assert fell  # sizes that are not the largest step's


def test_pages_refusals():
    def take(prob=None, counts=P, n=10, lens=P, bt=P, free=P, state=P, seq=P, off=P):
        return _lib.LIB.pkv_pages_take(ctypes.byref(prob or _prob()), counts, n, lens, bt, free,
                                       state, seq, off, None, None, None)

    def release(prob=None, keep=P, lens=P, bt=P, free=P, state=P):
        return _lib.LIB.pkv_pages_release(ctypes.byref(prob or _prob()), keep, lens, bt, free,
                                          state, None)

    for name in ("counts", "lens", "bt", "free", "state", "seq", "off"):
        assert take(**{name: None}) == PKV_EINVAL, name
    for name in ("keep", "lens", "bt", "free", "state"):
        assert release(**{name: None}) == PKV_EINVAL, name
    assert take(n=-1) == PKV_EINVAL and take(n=2 ** 30 + 1) == PKV_ERANGE
    for over, want in BAD_PROBLEMS:
        assert take(prob=_prob(**over)) == want and release(prob=_prob(**over)) == want, over
