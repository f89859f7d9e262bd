"""Cases of the operators that surround the MoE reader in a decode step.

Five kinds: ``plan`` (page tables and slot maps from request lengths),
``append`` (new key/value rows into a paged cache, with page summaries),
``attend`` (one new token per request over the paged cache), ``sparse`` (the
same over pages chosen by their summaries' score) and ``norm`` (post-norm,
gate, scaled residual and pre-norm in one pass).

``run`` computes a case with plain torch operations in 32 bits when ``own`` is
false, and through ``calibration_free_sparse_gb300.block`` when it is true.
"""

import json
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _plan(requests, longest, new, page, width):
    return {"kind": "plan", "requests": requests, "longest": longest, "new": new, "page": page,
            "width": width}


def _append(requests, longest, new, page, kv_heads, dim, cache, rows):
    return {"kind": "append", "requests": requests, "longest": longest, "new": new, "page": page,
            "kv_heads": kv_heads, "dim": dim, "cache": cache, "rows": rows}


def _attend(requests, longest, heads, kv_heads, dim, page, cache, q, window=0, sinks=False):
    return {"kind": "attend", "requests": requests, "longest": longest, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "cache": cache, "q": q,
            "window": window, "sinks": sinks}


def _sparse(requests, longest, heads, kv_heads, dim, page, keep, cache, q):
    return {"kind": "sparse", "requests": requests, "longest": longest, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "keep": keep, "cache": cache, "q": q}


def _norm(tokens, hidden, h, y, x, post, gate, scale):
    return {"kind": "norm", "tokens": tokens, "hidden": hidden, "h": h, "y": y, "x": x,
            "post": post, "gate": gate, "scale": scale}


def listed():
    def named(name, case):
        return dict(case, name=name)

    return [
        # every decode step of a batch of 16 begins with this
        named("plan_decode_16", _plan(16, 4096, 1, 16, 512)),
        # admitting 256 ragged prompts of up to 1024 tokens at once
        named("plan_prompts_256", _plan(256, 1024, 1024, 16, 192)),
        # one new token of 16 requests, once a layer and step
        named("append_decode_16", _append(16, 4096, 1, 16, 4, 128, "bf16", "bf16")),
        # prompts of up to 2000 tokens into an 8-bit cache
        named("append_prompts_8", _append(8, 700, 2000, 64, 8, 64, "e4m3", "bf16")),
        # the latency of one request early in its answer
        named("attend_1_short", _attend(1, 301, 32, 4, 128, 16, "bf16", "bf16")),
        # a large batch of long conversations
        named("attend_128", _attend(128, 8192, 64, 4, 128, 64, "bf16", "bf16")),
        # an ordinary serving batch: heads of 64 with learned sinks and a sliding window
        named("attend_16_window", _attend(16, 4001, 64, 8, 64, 32, "f16", "f16", 1000, True)),
        # one very long document in an 8-bit cache
        named("attend_1_long_e4m3", _attend(1, 131071, 32, 8, 128, 64, "e4m3", "bf16")),
        # one very long document, 2048 of its tokens read
        named("sparse_1_long", _sparse(1, 131071, 32, 4, 128, 16, 128, "bf16", "bf16")),
        # a batch of long contexts, an eighth of them read
        named("sparse_16", _sparse(16, 32768, 64, 8, 64, 64, 64, "f16", "f16")),
        # a decode step's norm before the reader
        named("norm_16", _norm(16, 2048, "f32", "bf16", "f32", False, "none", 1.0)),
        # a prompt's rows through a gated sandwich norm
        named("norm_prompt", _norm(8191, 2880, "bf16", "bf16", "bf16", True, "full", 0.5)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "append", "attend", "attend", "sparse", "norm"])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "plan":
        longest, new = _log(rng, 1, 8192), rng.choice([1, 1, _log(rng, 1, 1024)])
        requests = _log(rng, 1, 1024 if new == 1 else 256)
        return _plan(requests, longest, new, page, -(-(longest + new) // page) + rng.randrange(8))
    if kind == "append":
        longest, new = _log(rng, 1, 4096), rng.choice([1, 1, _log(rng, 1, 2000)])
        requests = _log(rng, 1, 128 if new == 1 else 8)
        cache = rng.choice(["bf16", "f16", "e4m3"])
        rows = rng.choice(["bf16", "f16"]) if cache == "e4m3" else cache
        return _append(requests, longest, new, page, rng.choice([1, 2, 4, 8]),
                       rng.choice([64, 128]), cache, rows)
    cache = rng.choice(["bf16", "f16", "e4m3"])
    q = rng.choice(["bf16", "f16"]) if cache == "e4m3" else cache
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    heads = kv_heads * rng.choice([1, 2, 4, 7, 8, 16])
    if kind == "attend":
        requests = _log(rng, 1, 128)
        most = 128 * 8192 * 4 * 128 // (requests * kv_heads * dim)
        longest = _log(rng, 1, min(131072, most))
        return _attend(requests, longest, heads, kv_heads, dim, page, cache, q,
                       rng.choice([0, 0, 128, 777]), rng.choice([False, False, True]))
    if kind == "sparse":
        requests = _log(rng, 1, 32)
        most = 32 * 32768 * 4 * 128 // (requests * kv_heads * dim)
        longest = _log(rng, 1000, min(131072, most))
        keep = max(2, _log(rng, 128, 4096) // page)
        return _sparse(requests, longest, heads, kv_heads, dim, page, keep, cache, q)
    hidden = rng.choice([256, 2048, 2880, 4096, 8 * rng.randrange(1, 1024)])
    if hidden == 24 * 128:
        hidden += 8
    tokens = _log(rng, 1, max(1, min(16384, 8191 * 2880 // (2 * hidden))))
    h = rng.choice(["f32", "bf16", "f16"])
    return _norm(tokens, hidden, h, rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16", h]),
                 rng.choice([False, True]), rng.choice(["none", "channel", "token", "full"]),
                 rng.choice([1.0, 0.5, 0.22]))


def _lengths(case, longest, requests):
    """Ragged lengths of a case, from its fields alone: the longest, then
    anything from a quarter of it; in larger batches an empty and a
    one-token request."""
    r = random.Random(json.dumps({k: v for k, v in case.items() if k != "name"}, sort_keys=True))
    out = [longest] + [r.randint(max(1, longest // 4), longest) for _ in range(requests - 1)]
    if requests >= 8:
        out[3], out[5] = 0, 1
    return out


def _new(case):
    if case["new"] == 1:
        return [1] * case["requests"]
    return _lengths(dict(case, which="new"), case["new"], case["requests"])


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pages(g, held, width, spare=0):
    """A page table for requests that hold `held` pages each, pages in random
    order, and the number of pages of the pool."""
    total = sum(held)
    order = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(held, device="cuda")
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(n, 0) - n)[:, None] + col[None, :]
    mine = col[None, :] < n[:, None]
    table = torch.where(mine, order[at.clamp(max=max(0, total + spare - 1))], -1).to(torch.int32)
    return table.contiguous(), order[total:].contiguous(), total + spare


def _draw_cache(g, pages, kv_heads, page, dim, cache, scale, drift):
    """One of the cache's two arrays: rows around a direction of their page."""
    out = torch.empty((pages, kv_heads, page, dim), device="cuda", dtype=DTYPES[cache])
    chunk = max(1, (1 << 27) // (kv_heads * page * dim))
    for a in range(0, pages, chunk):
        n = min(chunk, pages - a)
        v = _randn(g, (n, kv_heads, page, dim))
        if drift:
            v = 0.8 * v + 0.6 * _randn(g, (n, kv_heads, 1, dim))
        if cache == "e4m3":
            v = (v / scale[:, None, None]).clamp(-448.0, 448.0)
        out[a:a + n] = v.to(DTYPES[cache])
    return out


def _with_cache(g, case, table, held, lens, drift=False):
    s = {"table": table, "page": case["page"]}
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.012 + 0.004 * torch.rand(case["kv_heads"], generator=g, device="cuda")
        s["v_scale"] = 0.012 + 0.004 * torch.rand(case["kv_heads"], generator=g, device="cuda")
    else:
        s["k_scale"] = s["v_scale"] = None
    pool = max(1, held)
    s["k"] = _draw_cache(g, pool, case["kv_heads"], case["page"], case["dim"], case["cache"],
                         s["k_scale"], drift)
    s["v"] = _draw_cache(g, pool, case["kv_heads"], case["page"], case["dim"], case["cache"],
                         s["v_scale"], False)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return s


def _all_summaries(s, pool):
    """Summaries of every page that a request holds, over its written rows."""
    k, table, lens, page = s["k"], s["table"], s["lens"], s["page"]
    cols = torch.arange(table.shape[1], device="cuda")
    rows = (lens[:, None] - cols[None, :] * page).clamp(0, page)
    filled = torch.zeros(max(1, pool), dtype=torch.long, device="cuda")
    mine = (table >= 0) & (rows > 0)
    filled[table[mine].long()] = rows[mine].long()
    codes = torch.zeros((k.shape[0], k.shape[1], 2, k.shape[3]), dtype=torch.int8, device="cuda")
    steps = torch.zeros((k.shape[0], k.shape[1]), device="cuda")
    chunk = max(1, (1 << 26) // (k.shape[1] * page * k.shape[3]))
    for a in range(0, k.shape[0], chunk):
        codes[a:a + chunk], steps[a:a + chunk] = _summary(k[a:a + chunk].float(),
                                                           filled[a:a + chunk])
    s["codes"], s["steps"] = codes, steps


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    if kind == "norm":
        T, H = case["tokens"], case["hidden"]
        s = {"h": _randn(g, (T, H), DTYPES[case["h"]]), "y": _randn(g, (T, H), DTYPES[case["y"]]),
             "post": None, "gate": None, "scale": case["scale"]}
        s["pre"] = 1.0 + 0.1 * _randn(g, (H,))
        if case["post"]:
            s["post"] = 1.0 + 0.1 * _randn(g, (H,))
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
        if shape is not None:
            s["gate"] = torch.sigmoid(_randn(g, shape)).to(DTYPES[case["y"]])
        s["h_out"] = torch.empty_like(s["h"])
        s["x"] = torch.empty((T, H), device="cuda", dtype=DTYPES[case["x"]])
        return dict(s, case=case)
    page, R = case["page"], case["requests"]
    if kind in ("plan", "append"):
        prev, new = _lengths(case, case["longest"], R), _new(case)
        held = [-(-n // page) for n in prev]
        need = [-(-(a + b) // page) - c for a, b, c in zip(prev, new, held)]
        width = case["width"] if kind == "plan" else max(a + b for a, b in zip(held, need)) + 1
        width = max(width, max(a + b for a, b in zip(held, need)))
        table, free, pool = _pages(g, held, width, sum(need) + 8)
        s = {"prev": torch.tensor(prev, dtype=torch.int32, device="cuda"),
             "new": torch.tensor(new, dtype=torch.int32, device="cuda"), "free": free,
             "table": table, "tokens": sum(new), "page": page}
        if kind == "plan":
            if own:
                from calibration_free_sparse_gb300 import block

                kv = torch.zeros((pool, 1, page, 64), device="cuda", dtype=torch.bfloat16)
                s["cache"] = block.PagedCache(kv, kv.clone(), 1, max_requests=R)
                s["plan"] = s["cache"].plan(table, sum(new))
            return dict(s, case=case)
        s["table"], _, _, slots, _, _, _ = _plan_plain(s)
        s.update(_with_cache(g, case, s["table"], pool, [a + b for a, b in zip(prev, new)]))
        s["slots"] = slots
        s["codes"] = torch.zeros((pool, case["kv_heads"], 2, case["dim"]), dtype=torch.int8,
                                 device="cuda")
        s["steps"] = torch.zeros((pool, case["kv_heads"]), device="cuda")
        # the new rows are slices of a joint projection's output
        qkv = _randn(g, (sum(new), 3 * case["kv_heads"], case["dim"]), DTYPES[case["rows"]])
        s["k_new"] = qkv[:, case["kv_heads"]:2 * case["kv_heads"]]
        s["v_new"] = qkv[:, 2 * case["kv_heads"]:]
        if own:
            from calibration_free_sparse_gb300 import block

            s["cache"] = block.PagedCache(s["k"], s["v"], case["kv_heads"], max_requests=R,
                                          codes=s["codes"], steps=s["steps"],
                                          k_scale=s["k_scale"], v_scale=s["v_scale"])
        return dict(s, case=case)
    lens = _lengths(case, case["longest"], R)
    held = [-(-n // page) for n in lens]
    table, _, pool = _pages(g, held, max(1, max(held)))
    s = _with_cache(g, case, table, pool, lens, drift=kind == "sparse")
    s["q"] = 1.5 * _randn(g, (R, case["heads"], case["dim"]))
    s["q"] = s["q"].to(DTYPES[case["q"]])
    s["out"] = torch.empty_like(s["q"])
    s["sinks"], s["window"] = None, 0
    if kind == "attend":
        s["lse"] = torch.empty((R, case["heads"]), device="cuda")
        s["window"] = case["window"]
        if case["sinks"]:
            s["sinks"] = _randn(g, (case["heads"],))
        s["codes"] = s["steps"] = None
    else:
        s["keep"] = case["keep"]
        s["pages"] = torch.empty((R, case["kv_heads"], case["keep"]), dtype=torch.int32,
                                 device="cuda")
        _all_summaries(s, pool)
    if own:
        from calibration_free_sparse_gb300 import block

        s["cache"] = block.PagedCache(s["k"], s["v"], case["heads"], max_requests=R,
                                      codes=s["codes"], steps=s["steps"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"])
    return dict(s, case=case)


# --------------------------------------------------------------------------
# the operators, plainly
# --------------------------------------------------------------------------
def _two_to(e):
    """2^e as float32, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _floor_log2(a):
    """floor(log2 a) of a > 0 (clamped to 2^-100 .. 2^100), from its bits."""
    return (a.clamp(2.0 ** -100, 2.0 ** 100).contiguous().view(torch.int32) >> 23) - 127


def _take(cache, *at):
    """Rows of a cache by index, as float32 (8-bit floats are indexed as bytes)."""
    if cache.element_size() > 1:
        return cache[at].float()
    return cache.view(torch.uint8)[at].view(cache.dtype).float()


def _put(cache, rows, *at):
    if cache.element_size() > 1:
        cache[at] = rows.to(cache.dtype)
    else:
        cache.view(torch.uint8)[at] = rows.to(cache.dtype).view(torch.uint8)


def _summary(rows, filled):
    """int8 codes [n][heads][2][dim] and steps [n][heads] of pages' keys
    (float32 [n][heads][page][dim]), over each page's first `filled` rows."""
    used = torch.arange(rows.shape[2], device=rows.device)[None, :] < filled[:, None]
    used = used[:, None, :, None]
    hi = torch.where(used, rows, -math.inf).amax(2)
    lo = torch.where(used, rows, math.inf).amin(2)
    empty = (filled == 0)[:, None, None]
    hi, lo = torch.where(empty, 0.0, hi), torch.where(empty, 0.0, lo)
    a = torch.maximum(hi.abs(), lo.abs()).amax(-1).clamp(2.0 ** -100, 2.0 ** 100)
    step = _two_to(_floor_log2(a) - 6)
    step = torch.where(a > 127.0 * step, 2.0 * step, step)
    hi = torch.ceil(hi / step[..., None]).clamp(-127, 127)
    lo = torch.floor(lo / step[..., None]).clamp(-127, 127)
    return torch.stack([hi, lo], 2).to(torch.int8), step


def _plan_plain(s):
    prev, new, page = s["prev"].long(), s["new"].long(), s["page"]
    lens = prev + new
    have = (prev + page - 1) // page
    need = (lens + page - 1) // page - have
    ends = torch.cumsum(new, 0)
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), ends])
    first = torch.cumsum(need, 0) - need
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free"].shape[0] - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    t = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(ends, t, right=True).clamp(max=prev.shape[0] - 1)
    pos = prev[r] + t - starts[r]
    slots = table[r, pos // page] * page + pos % page
    i32 = torch.int32
    return (table, lens.to(i32), starts.to(i32), slots.to(i32), pos.to(i32), r.to(i32),
            need.sum().reshape(1).to(i32))


def _append_plain(s):
    k, v, page, slots = s["k"], s["v"], s["page"], s["slots"].long()
    k_rows, v_rows = s["k_new"].float(), s["v_new"].float()
    if s["k_scale"] is not None:
        k_rows = (k_rows / s["k_scale"][:, None]).clamp(-448.0, 448.0)
        v_rows = (v_rows / s["v_scale"][:, None]).clamp(-448.0, 448.0)
    every = slice(None)
    _put(k, k_rows, slots // page, every, slots % page)
    _put(v, v_rows, slots // page, every, slots % page)
    # the last new row of each page sums the page up
    follows = torch.cat([slots[1:] == slots[:-1] + 1, slots.new_zeros(1, dtype=torch.bool)])
    last = slots[~follows | (slots % page == page - 1)]
    pages = last // page
    codes, steps = _summary(_take(k, pages), last % page + 1)
    s["codes"][pages], s["steps"][pages] = codes, steps
    return {"k": k, "v": v, "codes": s["codes"], "steps": s["steps"]}


def _softmax_over(q, k, v, seen, scale, sinks):
    """q [R][kv][G][D], k and v [R][kv][L][D], seen [R or 1][kv or 1][1][L]."""
    logits = torch.matmul(q, k.transpose(-1, -2)) * scale
    logits = torch.where(seen, logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    if sinks is not None:
        top = torch.maximum(top, sinks)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    if sinks is not None:
        total = total + torch.exp(sinks - top)
    out = torch.matmul(p, torch.where(seen.transpose(-1, -2), v, 0.0))
    out = torch.where(total > 0, out / total, 0.0)
    return out, torch.log(total) + top


def _grouped(s):
    R, heads, dim = s["q"].shape
    kv = s["k"].shape[1]
    return s["q"].float().reshape(R, kv, heads // kv, dim)


def _scaled(x, scale):
    return x if scale is None else x * scale[:, None, None]


def _attend_plain(s):
    q, (R, heads, dim) = _grouped(s), s["q"].shape
    kv, page = s["k"].shape[1], s["page"]
    width, lens = s["table"].shape[1], s["lens"].long()[:, None]
    lo, count = torch.zeros_like(lens), width
    if s["window"]:
        lo = (lens - s["window"]).clamp(min=0)
        count = min(width, s["window"] // page + 2)
    col = lo // page + torch.arange(count, device="cuda")           # [R][count]
    table = torch.gather(s["table"], 1, col.clamp(max=width - 1)).clamp(min=0).long()
    L = count * page

    def rows(cache, scale):
        return _scaled(_take(cache, table).transpose(1, 2).reshape(R, kv, L, dim), scale)

    at = (col[..., None] * page + torch.arange(page, device="cuda")).reshape(R, L)
    seen = (at < lens) & (at >= lo)
    sinks = None if s["sinks"] is None else s["sinks"].reshape(1, kv, heads // kv, 1)
    out, lse = _softmax_over(q, rows(s["k"], s["k_scale"]), rows(s["v"], s["v_scale"]),
                             seen[:, None, None, :], dim ** -0.5, sinks)
    return {"out": out.reshape(R, heads, dim).to(s["q"].dtype), "lse": lse.reshape(R, heads)}


def _sparse_plain(s):
    q, (R, heads, dim) = _grouped(s), s["q"].shape
    kv, page, keep = s["k"].shape[1], s["page"], s["keep"]
    table = s["table"].clamp(min=0)
    width = table.shape[1]
    # 7-bit codes of the group's positive and negative parts
    a = q.abs().amax((2, 3), keepdim=True)
    fixed = torch.round(q * _two_to(13 - _floor_log2(a)))
    parts = torch.stack([fixed.clamp(min=0).sum(2), (-fixed).clamp(min=0).sum(2)], 2)
    top = parts.amax((2, 3), keepdim=True).clamp(min=1.0)
    parts = torch.round(parts * _two_to(6 - _floor_log2(top))).clamp(max=127)
    parts[:, :, 1] *= -1
    score = (s["codes"][table].float() * parts[:, None]).sum((3, 4)) * s["steps"][table]
    score = score.transpose(1, 2)                                    # [R][kv][width]
    held = ((s["lens"].long() + page - 1) // page)[:, None, None]
    col = torch.arange(width, device="cuda")
    score = torch.where((col == 0) | (col == held - 1), math.inf, score)
    score = torch.where(col < held, score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    if order.shape[-1] < keep:
        order = torch.cat([order, order.new_full((R, kv, keep - order.shape[-1]), width)], -1)
    order = torch.where(order < held, order, width + 1).sort(-1).values
    pages = torch.where(order < held, order, -1)
    # attention over the chosen pages
    physical = torch.gather(table[:, None].expand(R, kv, width), 2, pages.clamp(min=0).long())
    head = torch.arange(kv, device="cuda")[None, :, None]

    def rows(cache, scale):
        return _scaled(_take(cache, physical.long(), head).reshape(R, kv, keep * page, dim), scale)

    at = pages[..., None] * page + torch.arange(page, device="cuda")
    seen = (pages[..., None] >= 0) & (at < s["lens"][:, None, None, None])
    out, _ = _softmax_over(q, rows(s["k"], s["k_scale"]), rows(s["v"], s["v_scale"]),
                           seen.reshape(R, kv, 1, keep * page), dim ** -0.5, None)
    return {"out": out.reshape(R, heads, dim).to(s["q"].dtype), "pages": pages.to(torch.int32)}


def _norm_plain(s):
    z = s["y"].float()
    if s["post"] is not None:
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS) * s["post"]
    if s["gate"] is not None:
        z = z * s["gate"].float()
    h = s["h"].float() + s["scale"] * z
    x = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["pre"]
    return {"h": h.to(s["h_out"].dtype), "x": x.to(s["x"].dtype)}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    s, kind = state, state["case"]["kind"]
    if not own:
        if kind == "plan":
            names = ("table", "lens", "starts", "slots", "positions", "requests", "taken")
            return dict(zip(names, _plan_plain(s)))
        return {"append": _append_plain, "attend": _attend_plain, "sparse": _sparse_plain,
                "norm": _norm_plain}[kind](s)
    if kind == "plan":
        p = s["plan"]
        p.update(s["prev"], s["new"], s["free"])
        return {"table": p.table, "lens": p.lens, "starts": p.starts, "slots": p.slots,
                "positions": p.positions, "requests": p.requests, "taken": p.taken}
    if kind == "append":
        s["cache"].append(s["k_new"], s["v_new"], s["slots"])
        return {"k": s["k"], "v": s["v"], "codes": s["codes"], "steps": s["steps"]}
    if kind == "attend":
        s["cache"].attend(s["q"], s["table"], s["lens"], s["out"], window=s["window"],
                          sinks=s["sinks"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "sparse":
        s["cache"].select(s["q"], s["table"], s["lens"], s["pages"])
        s["cache"].attend(s["q"], s["table"], s["lens"], s["out"], pages=s["pages"])
        return {"out": s["out"], "pages": s["pages"]}
    from calibration_free_sparse_gb300 import block

    block.residual_norm(s["h"], s["x"], y=s["y"], post_weight=s["post"], gate=s["gate"],
                        scale=s["scale"], pre_weight=s["pre"], eps=EPS, h_out=s["h_out"])
    return {"h": s["h_out"], "x": s["x"]}


def work(case):
    kind = case["kind"]
    if kind == "norm":
        T, H = case["tokens"], case["hidden"]
        n = T * H
        gate = {"none": 0, "channel": H, "token": T, "full": n}[case["gate"]] * SIZE[case["y"]]
        b = n * (2 * SIZE[case["h"]] + SIZE[case["y"]] + SIZE[case["x"]]) + gate + 8 * H
        return {"bytes": b, "flops": 8 * n}
    page, R = case["page"], case["requests"]
    if kind in ("plan", "append"):
        prev, new = _lengths(case, case["longest"], R), _new(case)
        fresh = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(prev, new))
        if kind == "plan":
            # lengths in; lengths, starts and three words a token out; fresh pages in and out
            return {"bytes": 16 * R + 12 * sum(new) + 8 * fresh, "flops": 4 * sum(new)}
        kv, D, e = case["kv_heads"], case["dim"], SIZE[case["cache"]]
        old = sum(a % page for a, b in zip(prev, new) if b)       # keys already in touched pages
        touched = sum(-(-(a + b) // page) - a // page for a, b in zip(prev, new) if b)
        b = 2 * sum(new) * kv * D * (SIZE[case["rows"]] + e) + 4 * sum(new)
        return {"bytes": b + old * kv * D * e + touched * kv * (2 * D + 4),
                "flops": 2 * (old + sum(new)) * kv * D}
    kv, D, e, heads = case["kv_heads"], case["dim"], SIZE[case["cache"]], case["heads"]
    lens = _lengths(case, case["longest"], R)
    qo = 2 * R * heads * D * SIZE[case["q"]] + 4 * R
    if kind == "attend":
        seen = sum(min(n, case["window"] or n) for n in lens)
        pages = sum(-(-min(n, case["window"] or n) // page) for n in lens)
        return {"bytes": qo + 2 * seen * kv * D * e + 4 * pages + 4 * R * heads,
                "flops": 4 * seen * heads * D}
    held = sum(-(-n // page) for n in lens)
    seen = sum(min(n, case["keep"] * page) for n in lens)
    return {"bytes": qo + held * (kv * (2 * D + 4) + 4) + 2 * seen * kv * D * e +
            4 * R * kv * case["keep"],
            "flops": 4 * held * kv * D + 4 * seen * heads * D}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _to_e4m3(x):
    """Nearest e4m3 value (ties to even), saturating, of float64 x."""
    m = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(m)
    unit = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.sign(x) * np.minimum(np.rint(m / unit) * unit, 448.0)


def _summary_of(rows):
    """hi and lo codes and the step of one page's keys [rows][dim] (float64)."""
    hi, lo = rows.max(0), rows.min(0)
    a = min(max(np.abs(hi).max(), np.abs(lo).max(), 2.0 ** -100), 2.0 ** 100)
    step = 2.0 ** (math.frexp(a)[1] - 7)
    step = 2 * step if a > 127 * step else step
    return (np.clip(np.ceil(hi / step), -127, 127), np.clip(np.floor(lo / step), -127, 127), step)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"plan": _exact_plan, "append": _exact_append, "attend": _exact_attend,
            "sparse": _exact_sparse, "norm": _exact_norm}[case["kind"]](s)


def _exact_plan(s):
    prev, new, free, table = (_np(s[n]).copy() for n in ("prev", "new", "free", "table"))
    slots, pos, req, starts, used, page = [], [], [], [0], 0, s["page"]
    for r in range(len(prev)):
        for p in range(prev[r], prev[r] + new[r]):
            if p % page == 0:
                table[r, p // page] = free[used]
                used += 1
            slots.append(table[r, p // page] * page + p % page)
            pos.append(p)
            req.append(r)
        starts.append(len(slots))
    i32 = lambda v: np.asarray(v, np.int32)  # noqa: E731
    return {"table": table, "lens": i32(prev + new), "starts": i32(starts), "slots": i32(slots),
            "positions": i32(pos), "requests": i32(req), "taken": i32([used])}


def _exact_append(s):
    page, slots = s["page"], _np(s["slots"])
    caches = []
    for name in ("k", "v"):
        cache, rows = _np(s[name]), _np(s[name + "_new"])
        if s[name + "_scale"] is not None:
            rows = _to_e4m3(rows / _np(s[name + "_scale"])[:, None])
        cache[slots // page, :, slots % page] = rows
        caches.append(cache)
    codes, steps = _np(s["codes"]).astype(np.float64), _np(s["steps"])
    for t, slot in enumerate(slots):
        if t + 1 < len(slots) and slots[t + 1] == slot + 1 and (slot + 1) % page:
            continue
        for h in range(codes.shape[1]):
            hi, lo, step = _summary_of(caches[0][slot // page, h, :slot % page + 1])
            codes[slot // page, h, 0], codes[slot // page, h, 1] = hi, lo
            steps[slot // page, h] = step
    return {"k": caches[0], "v": caches[1], "codes": codes.astype(np.int8), "steps": steps}


def _rows_of(s, name, r, positions):
    """Float64 rows [kv][n][dim] of request r's tokens at `positions`."""
    page = s["page"]
    at = s["table"][r, positions // page].long(), slice(None), positions % page
    rows = _take(s[name], *at).double().transpose(0, 1)
    scale = s[name + "_scale"]
    return rows if scale is None else rows * scale.double()[:, None, None]


def _exact_row(q, k, v, sinks):
    """Attention of q [G][dim] over k, v [n][dim] in float64: (out, lse)."""
    logits = q @ k.T / math.sqrt(q.shape[1])
    if sinks is not None:
        logits = torch.cat([logits, sinks.double()[:, None]], 1)
    lse = torch.logsumexp(logits, 1)
    return torch.softmax(logits, 1)[:, :k.shape[0]] @ v, lse


def _exact_attend(s):
    R, heads, dim = s["q"].shape
    kv = s["k"].shape[1]
    G = heads // kv
    out = np.zeros((R, heads, dim))
    lse = np.full((R, heads), -np.inf)
    if s["sinks"] is not None:
        lse[:] = _np(s["sinks"])
    for r, n in enumerate(_np(s["lens"])):
        if n == 0:
            continue
        at = torch.arange(max(0, n - s["window"]) if s["window"] else 0, int(n), device="cuda")
        k, v = _rows_of(s, "k", r, at), _rows_of(s, "v", r, at)
        for h in range(kv):
            mine = slice(h * G, h * G + G)
            sinks = None if s["sinks"] is None else s["sinks"][mine]
            o, e = _exact_row(s["q"][r, mine].double(), k[h], v[h], sinks)
            out[r, mine], lse[r, mine] = o.cpu().numpy(), e.cpu().numpy()
    return {"out": out, "lse": lse}


def _exact_sparse(s):
    R, heads, dim = s["q"].shape
    kv, page, keep = s["k"].shape[1], s["page"], s["keep"]
    G = heads // kv
    codes, steps, table = _np(s["codes"]).astype(np.int64), _np(s["steps"]), _np(s["table"])
    out, pages = np.zeros((R, heads, dim)), np.full((R, kv, keep), -1, np.int32)
    for r, n in enumerate(_np(s["lens"])):
        if n == 0:
            continue
        held = -(-int(n) // page)
        mine = table[r, :held]
        for h in range(kv):
            q = _np(s["q"][r, h * G:h * G + G])
            biggest = max(np.abs(q).max(), 2.0 ** -100)
            fixed = np.rint(q * 2.0 ** (14 - math.frexp(biggest)[1]))
            up, down = np.maximum(fixed, 0).sum(0), np.maximum(-fixed, 0).sum(0)
            unit = 2.0 ** (math.frexp(max(up.max(), down.max(), 1.0))[1] - 7)
            up = np.minimum(np.rint(up / unit), 127).astype(np.int64)
            down = np.minimum(np.rint(down / unit), 127).astype(np.int64)
            score = (codes[mine, h, 0] @ up - codes[mine, h, 1] @ down) * steps[mine, h]
            score[0] = score[held - 1] = np.inf
            best = np.sort(np.lexsort((np.arange(held), -score))[:keep])
            pages[r, h, :len(best)] = best
            at = (best[:, None] * page + np.arange(page)).reshape(-1)
            at = torch.from_numpy(at[at < n]).cuda()
            where = s["table"][r, at // page].long()
            k, v = (_take(s[m], where, h, at % page).double() for m in ("k", "v"))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            o, _ = _exact_row(s["q"][r, h * G:h * G + G].double(), k, v, None)
            out[r, h * G:h * G + G] = o.cpu().numpy()
    return {"out": out, "pages": pages}


def _exact_norm(s):
    z = _np(s["y"])
    if s["post"] is not None:
        z = z / np.sqrt(np.mean(z ** 2, axis=1, keepdims=True) + EPS) * _np(s["post"])
    if s["gate"] is not None:
        z = z * _np(s["gate"])
    h = _np(s["h"]) + s["scale"] * z
    return {"h": h, "x": h / np.sqrt(np.mean(h ** 2, axis=1, keepdims=True) + EPS) * _np(s["pre"])}
