"""Measured cases of the 8-bit cache, cross attention and page tables.

Five operators over paged K/V (pages of 16 tokens, read through a block table,
grouped-query heads):

* ``cache8``: a run of new tokens is quantised into the 8-bit cache as it is
  written, and the pages that it touched are read back;
* ``kv8``: one query token per row attends over the 8-bit cache;
* ``prompt8``: many query tokens per row, causal, over the 8-bit cache;
* ``cross``: every query token of a row attends over all of the row's encoder
  states, whose length is its own (16-bit or 8-bit pages);
* ``pages``: pages are taken from the free list for a step's new tokens, with
  the slots, positions, lengths and offsets that the step's calls read, and
  given back.

``own`` false computes them in plain torch operations; ``own`` true makes the
calls of ``paged_kv_gqa_block_amd``.  Row lengths follow from the case alone
(``len_seed``), values and page order from ``prepare``'s seed.

The 8-bit cache: a block is one page of one KV head, K and V apart: 16 tokens by
d channels of e4m3 codes (no infinities, 448 the largest) and one scale, a power
of two 2^e held as the byte e + 127.  Writing a run gives a block the smallest e
with max |x| <= 448 * 2^e over the run's tokens in it, kept in [-15, 7] (f16) or
[-117, 119] (bf16); where the block holds earlier tokens of the row its e does
not shrink, and where it grows they are rounded again.  Bytes of a block are
ordered as the layout functions below say.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# Smallest and largest block exponent: every value stays exact in the 16-bit type.
EXP8 = {"f16": (-15, 7), "bf16": (-117, 119)}
TOP8 = 448.0


# ---- cases -------------------------------------------------------------------

def _case(name, op, dtype, heads, kv_heads, d, batch, lo, hi, new_lo=1, new_hi=1, window=0,
          sinks=0, bits=8, len_seed=0, mix="uniform", spare=150):
    """Row lengths lo..hi (cache tokens after the pass; cross: encoder states;
    pages: tokens held before), of which new_lo..new_hi are new (cross: queries
    of the row); window 0 sees everything; new_hi 0 makes every token new.
    spare: free pages for every hundred that the step asks for."""
    return {"name": name, "op": op, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "d": d,
            "batch": batch, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi,
            "window": window, "sinks": sinks, "bits": bits, "len_seed": len_seed, "mix": mix,
            "spare": spare}


def listed():
    return [
        # One decode step's keys and values of 64 requests: latency counts, and
        # most pages hold earlier tokens.
        _case("cache8_step_b64", "cache8", "bf16", 64, 8, 128, 64, 1024, 32768, len_seed=1),
        # Eight ragged prompts written at once, short and long ones.
        _case("cache8_prompts_b8", "cache8", "f16", 32, 8, 128, 8, 128, 32768, new_hi=0,
              len_seed=2, mix="bimodal"),
        # The smallest step: one request, small heads.
        _case("kv8_tiny", "kv8", "f16", 8, 2, 64, 1, 2048, 2048, len_seed=3),
        # One long request.
        _case("kv8_long", "kv8", "f16", 32, 8, 128, 1, 32768, 32768, len_seed=4),
        # A full serving batch.
        _case("kv8_b64", "kv8", "bf16", 64, 8, 128, 64, 1024, 32768, len_seed=5),
        # Short chunks after long cached contexts (a few tokens each, ragged).
        _case("prompt8_chunks_b8", "prompt8", "bf16", 64, 8, 128, 8, 1024, 32768, 1, 64,
              window=4096, sinks=4, len_seed=6),
        # Ragged prompts from scratch, the whole context visible.
        _case("prompt8_ragged_b8", "prompt8", "f16", 32, 8, 128, 8, 300, 4096, new_hi=0,
              len_seed=7),
        # Beam search of 16 utterances: four beams of one row read its states once.
        _case("cross_beams_b16", "cross", "f16", 16, 16, 64, 16, 200, 1500, 4, 4, bits=16,
              len_seed=8),
        # Ragged decoder prompts over documents of other lengths.
        _case("cross_prompts_b8", "cross", "bf16", 32, 8, 128, 8, 1024, 8192, 1, 448, bits=16,
              len_seed=9),
        # One to four tokens a row of a large batch, states held in 8 bits.
        _case("cross_step8_b64", "cross", "bf16", 32, 8, 128, 64, 500, 8000, 1, 4, bits=8,
              len_seed=10),
        # One new token of 64 requests, a few of which start a page.
        _case("pages_step_b64", "pages", "bf16", 64, 8, 128, 64, 1024, 32768, len_seed=11),
        # Prompt chunks of 256 requests, more than the free pages can hold.
        _case("pages_chunks_b256", "pages", "bf16", 64, 8, 128, 256, 0, 4096, 0, 1024,
              len_seed=12, spare=90),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:  # a draw without anything to do is no case
        case = _draw(rng)
        n, new = _lengths(case)
        if case["op"] == "pages":
            if new.sum() > 0 and _page_count(n).sum() + _free_pages(case, n, new) >= 32:
                return case
        elif (n * (1 if case["op"] == "kv8" else new)).sum() > 0:
            return case


def _draw(rng):
    op = rng.choice(["cache8", "kv8", "prompt8", "cross", "pages"])
    d = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 8])
    group = rng.choice([1, 2, 4, 5, 8, 16])
    dtype = rng.choice(["f16", "bf16"])
    window, sinks = 0, 0
    if op in ("kv8", "prompt8") and rng.random() < 0.5:
        window, sinks = _log(rng, 1, 8192), rng.choice([0, 1, 4, rng.randint(0, 64)])
    len_seed = rng.randrange(1 << 30)
    if op == "pages":
        batch = _log(rng, 1, 512)
        new_hi = rng.choice([1, 1, _log(rng, 2, max(3, 131072 // batch))])
        return _case("", op, dtype, kv_heads * group, kv_heads, d, batch, 0, _log(rng, 1, 8192),
                     rng.choice([0, 1]), new_hi, len_seed=len_seed,
                     spare=rng.choice([40, 100, 150, 300]))
    if op in ("prompt8", "cross"):
        batch = _log(rng, 1, 8 if op == "prompt8" else 32)
        hi = _log(rng, 16, max(17, (4096 if op == "prompt8" else 32768) // batch))
        if op == "prompt8":
            new = rng.choice([0, 0, 1, rng.randint(1, 128)])
        else:
            new = rng.choice([1, rng.randint(1, 8), _log(rng, 4, 256)])
        return _case("", op, dtype, kv_heads * group, kv_heads, d, batch,
                     rng.choice([0, hi // 3, hi]), hi, rng.choice([0, new]), new, window, sinks,
                     8 if op == "prompt8" else rng.choice([8, 16]), len_seed)
    batch = _log(rng, 1, 64)
    hi = _log(rng, 1, 131072 // batch)
    new_hi = 1 if op != "cache8" else rng.choice([0, 1, rng.randint(1, 300)])
    return _case("", op, dtype, kv_heads * group, kv_heads, d, batch,
                 rng.choice([0, hi // 8, hi]), hi,
                 rng.choice([0, new_hi]) if op == "cache8" else 1, new_hi, window, sinks,
                 len_seed=len_seed)


def _lengths(case):
    """(cache tokens, new tokens) of every row; a row may be empty.  cross:
    (encoder states, queries); pages: (tokens held before, new tokens)."""
    rng = np.random.default_rng(case["len_seed"])
    b = case["batch"]
    if case["mix"] == "bimodal":
        n = np.concatenate([rng.integers(case["lo"], case["hi"] // 16, b // 2, endpoint=True),
                            rng.integers(case["hi"] // 2, case["hi"], b - b // 2, endpoint=True)])
        rng.shuffle(n)
    else:
        n = rng.integers(case["lo"], case["hi"], b, endpoint=True)
    if case["new_hi"] == 0:
        return n, n.copy()
    new = rng.integers(case["new_lo"], case["new_hi"], b, endpoint=True)
    if case["op"] in ("cross", "pages"):
        return n, new
    return n, np.minimum(n, new)


def _page_count(n):
    return -(-n // PAGE)


def _free_pages(case, n, new):
    """Free pages before a step of a pages case."""
    return int((_page_count(n + new) - _page_count(n)).sum()) * case["spare"] // 100


def _first_seen(case, n, new):
    """First token of the window of a row's first new token."""
    w = case["window"]
    return np.maximum(n - new + 1 - w, 0) if w else np.zeros_like(n)


def work(case):
    n, new = _lengths(case)
    d, hkv, hq, s = case["d"], case["kv_heads"], case["heads"], case["sinks"]
    if case["op"] == "pages":
        # Counts, lengths and offsets of a row; a slot and a position a token; a
        # page's number from the list to the table and back.
        taken = min(int((_page_count(n + new) - _page_count(n)).sum()), _free_pages(case, n, new))
        return {"bytes": float(24 * len(n) + 12 * int(new.sum()) + 16 * taken), "flops": 0.0}
    if case["op"] == "cache8":
        # 16 bits in, 8 bits out, the touched pages' 8 bits in and 16 out.
        back = np.where(new > 0, n - (n - new) // PAGE * PAGE, 0)
        return {"bytes": float(new.sum()) * hkv * 2 * 3 * d + float(back.sum()) * hkv * 2 * 3 * d,
                "flops": 0.0}
    token = 2 * d * case["bits"] // 8
    rows = np.ones_like(n) if case["op"] == "kv8" else new
    io = float(rows.sum()) * hq * (2 * d * 2 + 4)
    if case["op"] == "cross":
        return {"bytes": float(n[new > 0].sum()) * hkv * token + io,
                "flops": 4.0 * d * hq * float((n * new).sum())}
    first = _first_seen(case, n, new)
    seen = n - first + np.minimum(s, first)
    pairs = 0.0
    for ni, mi in zip(n.tolist(), new.tolist()):
        p = np.arange(ni - mi, ni, dtype=np.float64)
        f = np.maximum(p + 1 - case["window"], 0) if case["window"] else np.zeros_like(p)
        pairs += float((p + 1 - f + np.minimum(s, f)).sum())
    return {"bytes": float(seen.sum()) * hkv * token + io, "flops": 4.0 * d * hq * pairs}


# ---- the 8-bit cache's layout ----------------------------------------------------

def _pack8(k, v):
    """Codes uint8 [..., 16, d] of K and of V to the cache's bytes [..., 32 d]."""
    lead, d = k.shape[:-2], k.shape[-1]
    half, tok = d // 64, 256 // d  # 16-byte pieces of a lane; its V tokens in each
    k = k.reshape(-1, 16, half, 2, 4, 8).permute(0, 2, 4, 1, 3, 5)  # [half, kg, token, block, 8]
    v = v.reshape(-1, 4, half, tok, 16, d // 16).permute(0, 2, 1, 4, 3, 5)
    return torch.cat([k.reshape(-1, 16 * d), v.reshape(-1, 16 * d)], -1).view(*lead, 32 * d)


def _unpack8(b):
    """The cache's bytes [..., 32 d] to codes uint8 [..., 16, d] of K and of V."""
    lead, d = b.shape[:-1], b.shape[-1] // 32
    half, tok = d // 64, 256 // d
    k, v = b.reshape(-1, 32 * d).split(16 * d, -1)
    k = k.reshape(-1, half, 4, 16, 2, 8).permute(0, 3, 1, 4, 2, 5)
    v = v.reshape(-1, half, 4, 16, tok, d // 16).permute(0, 2, 1, 4, 3, 5)
    return k.reshape(*lead, 16, d), v.reshape(*lead, 16, d)


def _two_to(e):
    """2^e in float32, |e| < 127, exactly (a power function may round)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _value8(code, scale):
    """What codes [..., 16, d] with scale bytes [...] stand for, float32."""
    return code.view(torch.float8_e4m3fn).float() * _two_to(scale.int() - 127)[..., None, None]


def _need8(top, dtype):
    """Smallest block exponents for maxima `top`."""
    mant, exp = torch.frexp(top)
    lo, hi = EXP8[dtype]
    return torch.where(top == 0, lo, exp - 9 + (mant > 0.875)).clamp(lo, hi)


def _code8(x, e):
    """Codes of values x [..., 16, d] at block exponents e [...]."""
    y = x * _two_to(-e)[..., None, None]
    y = torch.where(torch.isfinite(x), y.clamp(-TOP8, TOP8), math.nan)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


# ---- inputs ----------------------------------------------------------------------

def _random_pool8(pages, hkv, d, dtype, normal):
    """An 8-bit pool of quantised random pages and its scales."""
    pool = torch.empty(pages, hkv, 32 * d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, hkv, 2, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (hkv * 32 * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = normal(n, hkv, 2, PAGE, d).float()
        e = _need8(x.abs().amax((-1, -2)), dtype)
        c = _code8(x, e)
        pool[a:a + n] = _pack8(c[:, :, 0], c[:, :, 1])
        scales[a:a + n] = (e + 127).byte()
    return pool, scales


def _prepare_pages(case, g):
    n, new = _lengths(case)
    b = case["batch"]
    held = _page_count(n)
    width = int(_page_count(n + new).max()) + 1
    free = _free_pages(case, n, new)
    total = max(int(held.sum()) + free, 1)
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    at = torch.from_numpy(np.concatenate([[0], np.cumsum(held)[:-1]])).cuda()
    j = torch.arange(width, device="cuda")[None]
    mine = j < torch.from_numpy(held).cuda()[:, None]
    table = torch.where(mine, order[torch.where(mine, at[:, None] + j, 0)], table)
    free_list = torch.cat([order[int(held.sum()):], order[:int(held.sum())]])
    s = {"case": case, "tokens": int(new.sum()), "pool": total, "block_table": table,
         "lens": torch.from_numpy(n.astype(np.int32)).cuda(),
         "counts": torch.from_numpy(new.astype(np.int32)).cuda(),
         "free": free_list, "num_free": free}
    # Where the rows are when their step's tokens have gone again.
    s["keep"] = s["lens"].clone()
    if own:
        from paged_kv_gqa_block_amd import engine
        prob = engine.make_problem(b, case["heads"], case["kv_heads"], case["d"], PAGE, total,
                                   width, case["dtype"])
        t = engine.PageTable(prob, s["tokens"])
        t.block_table.copy_(table)
        t.lens.copy_(s["lens"])
        t.free_pages.copy_(free_list)
        t.state[0] = free
        s["table"] = t
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "pages":
        return _prepare_pages(case, g)
    n, new = _lengths(case)
    b, hq, hkv, d = case["batch"], case["heads"], case["kv_heads"], case["d"]
    dt = TYPES[case["dtype"]]
    pages = np.maximum(_page_count(n), 1)
    width = int(pages.max())
    total = int(pages.sum())
    order = torch.randperm(total + total // 2 + 1, generator=g, device="cuda").int()
    at = torch.from_numpy(np.concatenate([[0], np.cumsum(pages)[:-1]])).cuda()
    j = torch.arange(width, device="cuda")
    j = at[:, None] + torch.minimum(j[None], torch.from_numpy(pages).cuda()[:, None] - 1)
    tokens = int(new.sum())

    def offsets(counts):
        return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dt)
    s = {"case": case, "block_table": order[j].contiguous(), "tokens": tokens,
         "seq_lens": torch.from_numpy(n.astype(np.int32)).cuda(), "tok_offsets": offsets(new),
         "new_max": int(new.max()), "scale": float(np.float32(1 / math.sqrt(d)))}
    pool = order.numel()
    if case["op"] == "cache8":
        # Keys and values as a fused projection leaves them: one row per token.
        s["kv_new"] = normal(max(tokens, 1), 2, hkv, d)[:tokens]
        first = (n - new) // PAGE * PAGE
        back = np.where(new > 0, n - first, 0)
        s["back_offsets"], s["back"] = offsets(back), int(back.sum())
        s["blocks"] = int(np.where(new > 0, _page_count(n) - first // PAGE, 0).sum())
        s["kv8_pool"] = torch.zeros(pool, hkv, 32 * d, dtype=torch.uint8, device="cuda")
        s["kv8_scales"] = torch.zeros(pool, hkv, 2, dtype=torch.uint8, device="cuda")
        # The earlier tokens of the first page that a row's run touches.
        mine, rows = _random_pool8(b, hkv, d, case["dtype"], normal), np.flatnonzero(new > 0)
        rows = torch.from_numpy(rows).cuda()
        page = s["block_table"].long()[rows, torch.from_numpy(first // PAGE).cuda()[rows]]
        s["kv8_pool"][page], s["kv8_scales"][page] = mine[0][rows], mine[1][rows]
    else:
        many = case["op"] != "kv8"
        s["q"] = normal(max(tokens, 1) if many else b, hq, d)
        if many:
            s["q"] = s["q"][:tokens]
        if case["bits"] == 8:
            s["kv8_pool"], s["kv8_scales"] = _random_pool8(pool, hkv, d, case["dtype"], normal)
        else:
            s["k_pool"], s["v_pool"] = normal(pool, hkv, PAGE, d), normal(pool, hkv, PAGE, d)
        first = _first_seen(case, n, new)
        last, begin = _page_count(n), first // PAGE
        s["seen_pages"] = max(1, int((last - begin + np.minimum(_page_count(case["sinks"]),
                                                                begin)).max()))
    if own:
        from paged_kv_gqa_block_amd import engine
        prob = engine.make_problem(b, hq, hkv, d, PAGE, pool, width, case["dtype"], s["scale"])
        if case["op"] == "cache8":
            s["cache"] = engine.Kv8Cache(prob, pool=s["kv8_pool"], scales=s["kv8_scales"])
            s["k_out"] = torch.empty(s["back"], hkv, d, dtype=dt, device="cuda")
            s["v_out"] = torch.empty_like(s["k_out"])
        elif case["op"] == "kv8":
            s["step"] = engine.Kv8Step(prob, case["window"], case["sinks"])
        elif case["op"] == "prompt8":
            s["step"] = engine.PromptStep(prob, tokens, case["window"], case["sinks"])
        else:
            s["step"] = engine.CrossStep(prob, tokens)
    return s


# ---- one pass ------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return (_plain_pages if op == "pages" else _plain_cache if op == "cache8"
                else _plain_attention)(s)
    if op == "pages":
        t = s["table"]
        w = t.take(s["counts"])
        t.release(s["keep"])
        return (w["seq_lens"], w["tok_offsets"], w["slots"], w["positions"], t.lens,
                t.block_table, t.free_pages)
    if op == "cache8":
        s["cache"].store(s["kv_new"][:, 0], s["kv_new"][:, 1], s["block_table"], s["seq_lens"],
                         s["tok_offsets"])
        k, v = s["cache"].load(s["block_table"], s["seq_lens"], s["back_offsets"], s["k_out"],
                               s["v_out"])
        return k, v, s["cache"].scales
    return s["step"].run(s)


def _plain_pages(s):
    held, cnt, table = s["lens"].long(), s["counts"].long(), s["block_table"]
    free, nfree, dev = s["free"], s["num_free"], s["lens"].device
    cap = table.shape[1] * PAGE
    upto = cnt.cumsum(0)
    offsets = torch.cat([upto.new_zeros(1), upto])
    fits = (upto <= s["tokens"]) & (held + cnt <= cap)
    had = (held + PAGE - 1) // PAGE
    need = torch.where(fits, (held + cnt + PAGE - 1) // PAGE - had, 0)
    asked = need.cumsum(0)
    served = fits & ((asked <= nfree) | (need == 0))
    lens = torch.where(served, held + cnt, 0)
    # Every new token's place; a token at the start of a page brings the page.
    t = torch.arange(s["tokens"], device=dev)
    row = torch.searchsorted(upto, t, right=True)
    p = held[row] + t - offsets[row]
    rank = (asked - need)[row] + p // PAGE - had[row]
    fresh = p // PAGE >= had[row]
    page = torch.where(fresh, free[(nfree - 1 - rank).clamp(0, free.numel() - 1)],
                       table[row, (p // PAGE).clamp_max(table.shape[1] - 1)]).long()
    ok = served[row]
    slots = torch.where(ok, page * PAGE + p % PAGE, -1)
    positions = torch.where(ok, p, -1).int()
    flat = torch.cat([table.flatten(), table.new_zeros(1)])  # the last takes what is not written
    at = torch.where(ok & fresh & (p % PAGE == 0), row * table.shape[1] + p // PAGE,
                     table.numel())
    flat[at] = page.int()
    table = flat[:-1].view_as(table)
    nfree -= torch.where(served, need, 0).sum()
    # Back: what lies behind the tokens to keep, the first row's pages on top.
    now = torch.where(served, held + cnt, held)
    keep = torch.minimum(now, s["keep"].long())
    j = torch.arange(table.shape[1], device=dev)[None]
    gone = (j >= ((keep + PAGE - 1) // PAGE)[:, None]) & (j < ((now + PAGE - 1) // PAGE)[:, None])
    rank = gone.flatten().cumsum(0)
    at = torch.where(gone.flatten(), nfree + rank[-1] - rank, free.numel())
    free = torch.cat([free, free.new_zeros(1)])
    free[at] = table.flatten()
    table = torch.where(gone, -1, table)
    return (lens.int(), offsets.int(), slots, positions, keep.int(), table, free[:-1])


def _plain_cache(s):
    c = s["case"]
    n, off = s["seq_lens"].long(), s["tok_offsets"].long()
    new = off[1:] - off[:-1]
    first = (n - new) // PAGE
    count = torch.where(new > 0, (n + PAGE - 1) // PAGE - first, 0).cumsum(0)
    blk = torch.arange(s["blocks"], device=n.device)
    row = torch.searchsorted(count, blk, right=True)
    entry = first[row] + blk - torch.cat([count.new_zeros(1), count])[row]
    page = s["block_table"][row, entry].long()
    pos = entry[:, None] * PAGE + torch.arange(PAGE, device=n.device)
    begin = (n - new)[row][:, None]
    fresh = (pos >= begin) & (pos < n[row][:, None])
    if s["tokens"] == 0:
        z = torch.zeros(0, c["kv_heads"], c["d"], dtype=s["kv_new"].dtype, device=n.device)
        return z, z.clone(), s["kv8_scales"].clone()
    tok = torch.where(fresh, off[row][:, None] + pos - begin, 0)
    x = s["kv_new"].float()[tok].permute(0, 2, 3, 1, 4)  # [blocks, 2, heads, 16, d]
    x = torch.where(fresh[:, None, None, :, None], x, 0)
    top = torch.where(torch.isfinite(x), x, 0).abs().amax((-1, -2))
    e = _need8(top, c["dtype"])
    old = torch.stack(_unpack8(s["kv8_pool"][page]), 1)
    old_scale = s["kv8_scales"][page].transpose(1, 2)
    e = torch.where((pos[:, :1] < begin)[..., None], torch.maximum(e, old_scale.int() - 127), e)
    x = torch.where(fresh[:, None, None, :, None], x, _value8(old, old_scale))
    x = _value8(_code8(x, e), e + 127).to(s["kv_new"].dtype)
    scales = s["kv8_scales"].clone()
    scales[page] = (e + 127).byte().transpose(1, 2)
    # The touched pages' tokens, row after row.
    back = s["back_offsets"].long()
    t = torch.arange(s["back"], device=n.device)
    row = torch.searchsorted(back[1:].contiguous(), t, right=True)
    t = t - back[row]
    blk = torch.cat([count.new_zeros(1), count])[row] + t // PAGE
    x = x.permute(0, 3, 1, 2, 4)[blk, t % PAGE]
    return x[:, 0].contiguous(), x[:, 1].contiguous(), scales


def _plain_attention(s):
    c = s["case"]
    hq, hkv, d, w, sinks = c["heads"], c["kv_heads"], c["d"], c["window"], c["sinks"]
    many, cross = c["op"] != "kv8", c["op"] == "cross"
    grp = hq // hkv
    n = s["seq_lens"].long()[:, None]
    b = n.shape[0]
    dev = n.device
    # Queries, padded to the longest run: [b, m, hq, d] at positions p (negative: none).
    if many:
        off = s["tok_offsets"].long()
        new = (off[1:] - off[:-1])[:, None]
        m = max(1, s["new_max"])
        t = torch.arange(m, device=dev)[None]
        p = torch.where(t < new, n - 1 if cross else n - new + t, -1)
        if s["tokens"] == 0:
            return s["q"].clone(), torch.empty(0, hq, device=dev)
        q = s["q"][(off[:-1, None] + t).clamp_max(s["tokens"] - 1)]
    else:
        new, m, p, q = n.clamp_max(1), 1, n - 1, s["q"][:, None]
    # The pages that some query of the row sees: the sinks', then the window's.
    first = (n - new + 1 - w).clamp_min(0) if w else torch.zeros_like(n)
    last, begin = (n + PAGE - 1) // PAGE, first // PAGE
    ahead = begin.clamp_max((sinks + PAGE - 1) // PAGE)
    j = torch.arange(s["seen_pages"], device=dev)[None]
    page = torch.where(j < ahead, j, begin + j - ahead)
    page = torch.where(page < last, page, -1)
    at = s["block_table"].long().gather(1, page.clamp_min(0))
    if "kv8_pool" in s:
        scale = s["kv8_scales"][at]
        k, v = _unpack8(s["kv8_pool"][at])
        k, v = _value8(k, scale[..., 0]), _value8(v, scale[..., 1])
    else:
        k, v = s["k_pool"][at].float(), s["v_pool"][at].float()
    pos = (page[:, :, None] * PAGE + torch.arange(PAGE, device=dev)).masked_fill(
        page[:, :, None] < 0, 1 << 40).view(b, 1, -1)
    seen = pos <= p[:, :, None]
    if w:
        seen &= (pos > p[:, :, None] - w) | (pos < sinks)
    k, v = (x.permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d) for x in (k, v))
    q = q.float().view(b, m, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, m * grp, d)
    x = torch.matmul(q, k.transpose(-1, -2).contiguous()) * s["scale"]
    x = x.view(b, hkv, m, grp, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x.sub_(top.clamp_min(-1e38)))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hkv, m * grp, -1), v).view(b, hkv, m, grp, d)
    o = torch.where(total > 0, o / total, 0)
    lse = (top + total.log())[..., 0]
    o, lse = o.permute(0, 2, 1, 3, 4).reshape(b, m, hq, d), lse.permute(0, 2, 1, 3).reshape(b, m, hq)
    if not many:
        return o[:, 0].to(s["q"].dtype), lse[:, 0].contiguous()
    token = torch.arange(s["tokens"], device=dev)
    row = torch.searchsorted(off[1:].contiguous(), token, right=True)
    return o[row, token - off[row]].to(s["q"].dtype), lse[row, token - off[row]]


# ---- the definition, in 64 bits -------------------------------------------------------

def _power(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _stands_for(code, scale):
    """e4m3 codes [...] to 64-bit values: sign, four bits of exponent, three of
    mantissa, subnormals in steps of 2^-9."""
    c = code.int()
    exp, mant = ((c >> 3) & 15).double(), (c & 7).double()
    x = torch.where(exp == 0, mant * 2.0 ** -9, (8 + mant) * _power(exp - 10))
    x = torch.where((c & 127) == 127, math.nan, torch.where(c > 127, -x, x))
    return x * _power(scale.int() - 127)


def _e4m3(x, e):
    """Values x rounded to the nearest code at exponent e, ties to even, and
    back, in 64 bits."""
    y = x.abs() / _power(e)
    step = _power(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    step = torch.where(y / step >= 16, step * 2, step)  # log2 of a value just below a power
    step = torch.where((y / step < 8) & (step > 2.0 ** -9), step / 2, step)
    return torch.sign(x) * torch.clamp(torch.round(y / step) * step, max=TOP8) * _power(e)


def _exact_pages(case, s):
    n, new = _lengths(case)
    table, free = s["block_table"].cpu().numpy(), s["free"].cpu().numpy()[:s["num_free"]].tolist()
    order, left = [], s["num_free"]
    lens, slots, positions = [], [], []
    for r, (held, m) in enumerate(zip(n.tolist(), new.tolist())):
        pages = [int(x) for x in table[r, :_page_count(held)]]
        want = _page_count(held + m) - len(pages)
        ok = held + m <= table.shape[1] * PAGE and (want == 0 or 0 <= want <= left)
        if want:  # once a row has to wait, those behind it that need pages do too
            left = left - want if ok else -1
        if ok:
            for _ in range(want):
                pages.append(free.pop())
                order.append(pages[-1])
        lens.append(held + m if ok else 0)
        for p in range(held, held + m):
            slots.append(pages[p // PAGE] * PAGE + p % PAGE if ok else -1)
            positions.append(p if ok else -1)

    def back(x, like):
        return torch.tensor(x, dtype=like, device="cuda")
    # Given back in the reverse order, so that lists and tables are as they were.
    return (back(lens, torch.int32), back(np.concatenate([[0], np.cumsum(new)]), torch.int32),
            back(slots, torch.int64), back(positions, torch.int32), s["lens"], s["block_table"],
            back(free + order[::-1] + s["free"].cpu().numpy()[s["num_free"]:].tolist(),
                 torch.int32))


def _exact_cache(case, s):
    n, new = _lengths(case)
    lo, hi = EXP8[case["dtype"]]
    outs, scales = ([], []), s["kv8_scales"].clone()
    at = 0
    for i, (ni, mi) in enumerate(zip(n.tolist(), new.tolist())):
        if mi == 0:
            continue
        p0 = (ni - mi) // PAGE * PAGE
        old = ni - mi - p0
        ids = s["block_table"][i, p0 // PAGE:_page_count(ni)].long()
        for x, out in enumerate(outs):
            z = s["kv_new"][at:at + mi, x].double()
            z = torch.cat([z.new_zeros(old, *z.shape[1:]), z,
                           z.new_zeros(-(ni - p0) % PAGE, *z.shape[1:])])
            z = z.view(-1, PAGE, *z.shape[1:])  # [pages, 16, heads, d]
            top = z.abs().amax((1, 3))
            e = torch.full_like(top, lo)
            for k in range(lo, hi):
                e = torch.where(top > TOP8 * 2.0 ** k, k + 1, e)
            if old:
                was = s["kv8_scales"][ids[0], :, x]
                e[0] = torch.maximum(e[0], was.double() - 127)
                codes = _unpack8(s["kv8_pool"][ids[0]])[x]  # [heads, 16, d]
                z[0, :old] = _stands_for(codes, was[:, None, None]).transpose(0, 1)[:old]
            out.append(_e4m3(z, e[:, None, :, None]).flatten(0, 1)[:ni - p0])
            scales[ids, :, x] = (e + 127).byte()
        at += mi
    if not outs[0]:
        z = torch.zeros(0, case["kv_heads"], case["d"], dtype=torch.float64, device="cuda")
        return z, z.clone(), scales
    return torch.cat(outs[0]), torch.cat(outs[1]), scales


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "pages":
        return _exact_pages(case, s)
    if case["op"] == "cache8":
        return _exact_cache(case, s)
    n, new = _lengths(case)
    d, hkv, w = case["d"], case["kv_heads"], case["window"]
    many = case["op"] != "kv8"
    outs, lses = [], []
    at = 0
    for i, (ni, mi) in enumerate(zip(n.tolist(), new.tolist())):
        mi = mi if many else 1
        q = s["q"][at:at + mi].double().view(mi, hkv, case["heads"] // hkv, d)
        at += mi
        ids = s["block_table"][i, :_page_count(ni)].long()
        if case["bits"] == 8:
            scale = s["kv8_scales"][ids][..., None, None]
            k, v = (_stands_for(x, scale[:, :, j])
                    for j, x in enumerate(_unpack8(s["kv8_pool"][ids])))
        else:
            k, v = s["k_pool"][ids].double(), s["v_pool"][ids].double()
        k, v = (x.transpose(1, 2).reshape(-1, hkv, d)[:ni] for x in (k, v))
        t = torch.arange(ni, device=k.device)
        step = max(1, (1 << 27) // max(1, ni * q.shape[2]))
        for a in range(0, mi, step):
            p = torch.arange(ni - mi + a, min(ni, ni - mi + a + step), device=k.device)[:, None]
            if case["op"] == "cross":
                p = torch.full((min(step, mi - a), 1), ni - 1, device=k.device)
            if ni == 0:
                outs.append(torch.zeros(mi, case["heads"], d, dtype=torch.float64, device=k.device))
                lses.append(torch.full((mi, case["heads"]), -math.inf, dtype=torch.float64,
                                       device=k.device))
                break
            ok = t <= p
            if w:
                ok &= (p - t < w) | (t < case["sinks"])
            o_h, l_h = [], []
            for h in range(hkv):
                qh = q[a:a + step, h].reshape(-1, d)
                z = (qh @ k[:, h].t().contiguous()).view(p.shape[0], q.shape[2], ni) * s["scale"]
                z = z.masked_fill(~ok[:, None], -math.inf)
                l_h.append(torch.logsumexp(z, -1))
                o_h.append((torch.exp(z - l_h[-1][..., None]).view(-1, ni) @ v[:, h]).view(
                    p.shape[0], -1, d))
            outs.append(torch.cat(o_h, 1))
            lses.append(torch.cat(l_h, 1))
    if not outs:
        return (torch.zeros(0, case["heads"], d, dtype=torch.float64, device="cuda"),
                torch.zeros(0, case["heads"], dtype=torch.float64, device="cuda"))
    return torch.cat(outs), torch.cat(lses)
