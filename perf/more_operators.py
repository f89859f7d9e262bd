"""Cases of the operators that take a prompt through a decoder block.

Five kinds: ``chunk`` (attention of several new tokens per request over the
paged cache), ``act`` (the plan of a batch's experts, and their gated
activations by products grouped by expert), ``down`` (the experts' down
products, weighted and summed per token), ``fork`` (continuations that share a
request's pages and copy its last one) and ``compact`` (references and free
pages, and the pages in use moved to the front of the pool).

``run`` computes a case with plain torch operations in 32 bits when ``own`` is
false, and through ``calibration_free_sparse_gb300`` when it is true.
"""

import json
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}
I32 = torch.int32


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _chunk(requests, longest, new, heads, kv_heads, dim, page, cache, q, window=0, sinks=False):
    return {"kind": "chunk", "requests": requests, "longest": longest, "new": new, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "cache": cache, "q": q,
            "window": window, "sinks": sinks}


def _experts(kind, tokens, hidden, inter, experts, topk, dtype):
    return {"kind": kind, "tokens": tokens, "hidden": hidden, "inter": inter, "experts": experts,
            "topk": topk, "dtype": dtype}


def _pages(kind, requests, longest, kv_heads, dim, page, cache):
    return {"kind": kind, "requests": requests, "longest": longest, "kv_heads": kv_heads,
            "dim": dim, "page": page, "cache": cache}


def listed():
    def named(name, case):
        return dict(case, name=name)

    return [
        # five drafted tokens of 16 requests, to be verified
        named("chunk_verify_16", _chunk(16, 4096, 5, 32, 4, 128, 16, "bf16", "bf16")),
        # eight ragged prompts, heads of 64 with learned sinks and a sliding window
        named("chunk_prompts_8", _chunk(8, 2000, 2000, 64, 8, 64, 32, "f16", "f16", 128, True)),
        # the next chunk of one long document in an 8-bit cache
        named("chunk_1_long_e4m3", _chunk(1, 32768, 500, 32, 8, 128, 64, "e4m3", "bf16")),
        # a whole prompt of 8192 tokens at once
        named("chunk_prompt_8k", _chunk(1, 8192, 8192, 32, 4, 128, 64, "bf16", "bf16")),
        # a short prompt: every expert has a few tokens
        named("act_57", _experts("act", 57, 2048, 768, 128, 8, "bf16")),
        # a long prompt's chunk
        named("act_4096", _experts("act", 4096, 2048, 768, 128, 8, "bf16")),
        # a short prompt, the way back
        named("down_57", _experts("down", 57, 2048, 768, 128, 8, "bf16")),
        # a prompt's chunk through few wide experts
        named("down_2000", _experts("down", 2000, 2880, 2880, 32, 4, "bf16")),
        # a request continued in four ways
        named("fork_4", _pages("fork", 4, 301, 4, 128, 16, "bf16")),
        # a whole batch forked
        named("fork_512", _pages("fork", 512, 2048, 8, 128, 64, "bf16")),
        # the pool of a small batch, a third of its requests ended
        named("compact_16", _pages("compact", 16, 4096, 4, 128, 16, "bf16")),
        # a large pool in 8 bits
        named("compact_512", _pages("compact", 512, 2048, 8, 128, 64, "e4m3")),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(["chunk", "chunk", "act", "down", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128, 256])
    cache = rng.choice(["bf16", "f16", "e4m3"])
    if kind == "chunk":
        q = rng.choice(["bf16", "f16"]) if cache == "e4m3" else cache
        kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        heads = kv_heads * rng.choice([1, 2, 4, 7, 8, 16])
        requests = _log(rng, 1, 64)
        # products and cache no larger than the largest listed case's
        longest = _log(rng, 1, min(65536, (1 << 27) // (requests * kv_heads * dim)))
        most = 8192 * 8192 * 32 * 128 // (2 * longest * requests * heads * dim)
        new = min(longest, max(1, rng.choice([_log(rng, 1, 8), _log(rng, 1, 2048), longest])))
        return _chunk(requests, longest, max(1, min(new, most)), heads, kv_heads, dim, page, cache,
                      q, rng.choice([0, 0, 128, 777]), rng.choice([False, False, True]))
    if kind in ("act", "down"):
        experts = rng.choice([8, 16, 32, 64, 128])
        topk = rng.choice([1, 2, 4, 8])
        hidden = rng.choice([256, 2048, 2880, 4096, 8 * rng.randrange(1, 512)])
        inter = rng.choice([128, 768, 1536, 2880, 8 * rng.randrange(1, 256)])
        while experts * hidden * inter > 128 * 2048 * 768:
            experts //= 2
        topk = min(topk, experts)
        most = 4096 * 8 * 2048 * 768 // (topk * hidden * inter)
        return _experts(kind, _log(rng, 1, min(8192, most)), hidden, inter, experts, topk,
                        rng.choice(["bf16", "bf16", "f16"]))
    kv_heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    requests = _log(rng, 2, 512)
    most = 512 * 2048 * 8 * 128 // (requests * kv_heads * dim)
    return _pages(kind, requests, _log(rng, 1, min(16384, most)), kv_heads, dim, page, cache)


def _rand(case, which):
    fields = {k: v for k, v in case.items() if k != "name"}
    return random.Random(json.dumps(dict(fields, which=which), sort_keys=True))


def _lengths(case, longest, which):
    """Ragged lengths of a case, from its fields alone: the longest, then
    anything from a quarter of it; in larger batches an empty and a
    one-token request."""
    r, requests = _rand(case, which), case["requests"]
    out = [longest] + [r.randint(max(1, longest // 4), longest) for _ in range(requests - 1)]
    if requests >= 8:
        out[3], out[5] = 0, 1
    return out


def _chunk_lengths(case):
    """(lengths with the new tokens, new tokens)."""
    lens = _lengths(case, case["longest"], "held")
    if case["new"] <= 8:
        new = [case["new"]] * len(lens)
    else:
        new = _lengths(case, case["new"], "new")
    if case["new"] == case["longest"]:
        return new, new
    return lens, [min(a, b) for a, b in zip(new, lens)]


def _forks(case):
    """(lengths of the parents, parent of each child): the first quarter of
    the table's rows are parents, every child has one of them, drawn anew."""
    r = _rand(case, "forks")
    lens = _lengths(case, case["longest"], "held")
    parents = max(1, case["requests"] // 4)
    return lens[:parents], [r.randrange(parents) for _ in range(case["requests"] - parents)]


def _ended(case):
    r = _rand(case, "ended")
    return [r.random() < 0.35 for _ in range(case["requests"])]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _table(g, held, width, spare=0):
    """A page table for requests that hold `held` pages each, in random order,
    the other pages, and the number of pages of the pool."""
    total = sum(held)
    order = torch.randperm(total + spare, generator=g, device="cuda").to(I32)
    n = torch.tensor(held, device="cuda")
    col = torch.arange(width, device="cuda")
    at = (torch.cumsum(n, 0) - n)[:, None] + col[None, :]
    mine = col[None, :] < n[:, None]
    table = torch.where(mine, order[at.clamp(max=max(0, total + spare - 1))], -1).to(I32)
    return table.contiguous(), order[total:].contiguous(), total + spare


def _draw_cache(g, pages, kv_heads, page, dim, cache, scale):
    out = torch.empty((pages, kv_heads, page, dim), device="cuda", dtype=DTYPES[cache])
    step = max(1, (1 << 27) // (kv_heads * page * dim))
    for a in range(0, pages, step):
        v = _randn(g, (min(step, pages - a), kv_heads, page, dim))
        if cache == "e4m3":
            v = (v / scale[:, None, None]).clamp(-448.0, 448.0)
        out[a:a + step] = v.to(DTYPES[cache])
    return out


def _with_cache(g, case, pages):
    s = {"case": case, "page": case["page"], "k_scale": None, "v_scale": None}
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.012 + 0.004 * torch.rand(case["kv_heads"], generator=g, device="cuda")
        s["v_scale"] = 0.012 + 0.004 * torch.rand(case["kv_heads"], generator=g, device="cuda")
    for name in ("k", "v"):
        s[name] = _draw_cache(g, max(1, pages), case["kv_heads"], case["page"], case["dim"],
                              case["cache"], s[name + "_scale"])
    return s


def _cache(s, heads, requests, summaries=False):
    from calibration_free_sparse_gb300 import block

    extra = {"codes": s["codes"], "steps": s["steps"]} if summaries else {}
    return block.PagedCache(s["k"], s["v"], heads, max_requests=requests, k_scale=s["k_scale"],
                            v_scale=s["v_scale"], **extra)


def _prepare_chunk(case, g):
    lens, new = _chunk_lengths(case)
    held = [-(-n // case["page"]) for n in lens]
    table, _, pool = _table(g, held, max(1, max(held)))
    s = _with_cache(g, case, pool)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    kv, dim, heads, T = case["kv_heads"], case["dim"], case["heads"], starts[-1]
    # the queries are slices of a joint projection's output
    qkv = _randn(g, (T, heads + 2 * kv, dim))
    s.update(table=table, lens=_ints(lens), starts=_ints(starts),
             q=(1.5 * qkv).to(DTYPES[case["q"]])[:, :heads])
    s["out"] = torch.empty((T, heads, dim), dtype=s["q"].dtype, device="cuda")
    s["lse"] = torch.empty((T, heads), device="cuda")
    s["sinks"] = _randn(g, (heads,)) if case["sinks"] else None
    # what the plain form indexes with, known to the program on the host too
    s["host"] = (lens, starts)
    if own:
        s["cache"] = _cache(s, heads, case["requests"])
    return s


def _route(g, case):
    """Distinct experts per token, some asked for more often than others, and
    their weights."""
    T, E = case["tokens"], case["experts"]
    logits = _randn(g, (T, E)) + 0.5 * _randn(g, (E,))
    top = torch.topk(logits, case["topk"])
    return top.indices.to(I32).contiguous(), top.values.softmax(-1).contiguous()


def _prepare_experts(case, g):
    T, H, I, E, dt = (case["tokens"], case["hidden"], case["inter"], case["experts"],
                      DTYPES[case["dtype"]])
    ids, w = _route(g, case)
    s = {"case": case, "ids": ids, "w": w}

    def weights(rows, cols):
        out = torch.empty((E, rows, cols), dtype=dt, device="cuda")
        for e in range(E):
            out[e] = (_randn(g, (rows, cols)) / cols ** 0.5).to(dt)
        return out

    rows = T * case["topk"]
    if case["kind"] == "act":
        s["gate"], s["up"] = weights(I, H), weights(I, H)
        s["x"] = _randn(g, (T, H), dt)
        s["act"] = torch.empty((rows, I), dtype=dt, device="cuda")
    else:
        s["down"] = weights(H, I)
        a, b = _randn(g, (rows, I)), _randn(g, (rows, I))
        s["act"] = (a * torch.sigmoid(a) * b).to(dt)
        s["y"] = torch.empty((T, H), dtype=dt, device="cuda")
    if own:
        from calibration_free_sparse_gb300 import experts

        s["plan"] = experts.ExpertPlan(E, case["topk"], T, hidden=H)
        if case["kind"] == "act":
            s["experts"] = experts.Experts(gate=s["gate"], up=s["up"])
        else:
            s["experts"] = experts.Experts(down=s["down"])
            s["plan"].update(ids)
    elif case["kind"] == "down":
        s["order"], s["offsets"], s["places"] = _plan_plain(ids, E)
    return s


def _prepare_pages(case, g):
    page, R = case["page"], case["requests"]
    kv, dim = case["kv_heads"], case["dim"]
    if case["kind"] == "fork":
        lens, parents = _forks(case)
        held = [-(-n // page) for n in lens]
        width = max(1, max(held)) + 1
        table, free, pool = _table(g, held + [0] * len(parents), width, len(parents) + 4)
        s = _with_cache(g, case, pool)
        s["parents"] = _ints(parents)
        s["children"] = torch.arange(len(lens), R, dtype=I32, device="cuda")
        s["lens"], s["free"] = _ints(lens + [0] * len(parents)), free
    else:
        held = [-(-n // page) for n in _lengths(case, case["longest"], "held")]
        table, _, pool = _table(g, held, max(1, max(held)), 5)
        s = _with_cache(g, case, pool)
        lens = _lengths(case, case["longest"], "held")
        s["lens"] = _ints([0 if e else n for n, e in zip(lens, _ended(case))])
    s["table"], s["pool"] = table, pool
    s["codes"] = torch.randint(-127, 128, (pool, kv, 2, dim), generator=g, device="cuda",
                               dtype=torch.int32).to(torch.int8)
    s["steps"] = torch.rand((pool, kv), generator=g, device="cuda")
    if own:
        s["cache"] = _cache(s, kv, R, summaries=True)
        s["pages"] = s["cache"].pool(R)
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["kind"] == "chunk":
        return _prepare_chunk(case, g)
    if case["kind"] in ("act", "down"):
        return _prepare_experts(case, g)
    return _prepare_pages(case, g)


# --------------------------------------------------------------------------
# the operators, plainly
# --------------------------------------------------------------------------
def _take(cache, *at):
    """Rows of a cache by index, as float32 (8-bit floats are indexed as bytes)."""
    if cache.element_size() > 1:
        return cache[at].float()
    return cache.view(torch.uint8)[at].view(cache.dtype).float()


def _chunk_plain(s):
    T, heads, dim = s["q"].shape
    kv, page, window = s["k"].shape[1], s["page"], s["case"]["window"]
    G, scale = heads // kv, dim ** -0.5
    out = torch.zeros((T, heads, dim), dtype=s["q"].dtype, device="cuda")
    lse = torch.full((T, heads), -math.inf, device="cuda")
    lens, starts = s["host"]
    for r, n in enumerate(lens):
        a, b = starts[r], starts[r + 1]
        if a == b:
            continue
        step = max(1, (1 << 28) // (heads * n))              # tokens whose logits fit a few GB
        for t in range(a, b, step):
            e = min(t + step, b)
            first = n - (b - a) + t - a                       # position of token t
            last = first + e - t                              # keys that the block sees
            lo = max(0, first + 1 - window) // page * page if window else 0
            pages = s["table"][r, lo // page:-(-last // page)].long()

            def rows(name):
                x = _take(s[name], pages).transpose(0, 1).reshape(kv, -1, dim)[:, :last - lo]
                scales = s[name + "_scale"]
                return x if scales is None else x * scales[:, None, None]

            q = s["q"][t:e].float().reshape(e - t, kv, G, dim).permute(1, 2, 0, 3)
            q = q.reshape(kv, G * (e - t), dim)
            logits = torch.matmul(q, rows("k").transpose(1, 2)).view(kv, G, e - t, last - lo)
            logits *= scale
            at = torch.arange(lo, last, device="cuda")[None, :]
            pos = torch.arange(first, last, device="cuda")[:, None]
            seen = at <= pos
            if window:
                seen = seen & (at > pos - window)
            logits.masked_fill_(~seen, -math.inf)
            top = logits.amax(-1, keepdim=True)
            if s["sinks"] is not None:
                sinks = s["sinks"].view(kv, G, 1, 1)
                top = torch.maximum(top, sinks)
            p = logits.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            if s["sinks"] is not None:
                total = total + torch.exp(sinks - top)
            o = torch.matmul(p.view(kv, G * (e - t), last - lo), rows("v"))
            o = o.view(kv, G, e - t, dim) / total
            out[t:e] = o.permute(2, 0, 1, 3).reshape(e - t, heads, dim).to(out.dtype)
            lse[t:e] = (torch.log(total) + top).reshape(heads, e - t).T
    return {"out": out, "lse": lse}


def _plan_plain(ids, experts):
    """Pairs (token * topk + slot) in order of their experts, the experts'
    first rows, and each pair's row."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(experts + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=experts), 0)
    places = torch.empty_like(order)
    places[order] = torch.arange(order.shape[0], device="cuda")
    return order.to(I32), offsets.to(I32), places.to(I32).view(ids.shape)


def _act_plain(s):
    E, topk = s["case"]["experts"], s["case"]["topk"]
    order, offsets, places = _plan_plain(s["ids"], E)
    x, act = s["x"].float(), torch.empty_like(s["act"])
    ends = offsets.tolist()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        mine = x[order[a:b].long() // topk]
        g, v = mine @ s["gate"][e].float().T, mine @ s["up"][e].float().T
        act[a:b] = (g / (1.0 + torch.exp(-g)) * v).to(act.dtype)
    return {"order": order, "offsets": offsets, "places": places, "act": act}


def _down_plain(s):
    E, (rows, _) = s["case"]["experts"], s["act"].shape
    z = torch.empty((rows, s["y"].shape[1]), device="cuda")
    ends = s["offsets"].tolist()
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a < b:
            z[a:b] = s["act"][a:b].float() @ s["down"][e].float().T
    y = (z[s["places"].long()] * s["w"][..., None]).sum(1)
    return {"y": y.to(s["y"].dtype)}


def _move(s, src, dst):
    """Pages copied, all from what stood before."""
    for name in ("k", "v", "codes", "steps"):
        bits = s[name] if s[name].element_size() > 1 else s[name].view(torch.uint8)
        bits[dst] = bits[src]
    return {name: s[name] for name in ("k", "v", "codes", "steps")}


def _fork_plain(s):
    page, table, lens = s["page"], s["table"], s["lens"]
    parents, children = s["parents"].long(), s["children"].long()
    n = lens[parents]
    cut = n % page != 0
    rank = torch.cumsum(cut, 0) - 1
    fresh = s["free"][rank.clamp(min=0)]
    last = (n.long() // page)[:, None]
    rows = table[parents]
    src = torch.where(cut, rows.gather(1, last).squeeze(1), -1)
    dst = torch.where(cut, fresh, -1)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    rows = torch.where(cut[:, None] & (col == last), fresh[:, None], rows)
    held = col < -(-n // page)[:, None]
    table[children] = torch.where(held, rows, table[children])
    lens[children] = n
    pages = _move(s, src[cut].long(), dst[cut].long())
    return dict(pages, table=table, lens=lens, src=src, dst=dst, taken=cut.sum().reshape(1).to(I32))


def _collect_plain(table, lens, page, pool):
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    held = col < (-(-lens // page))[:, None]
    return held, torch.bincount(table[held].long(), minlength=pool)


def _compact_plain(s):
    pool, table = s["pool"], s["table"]
    held, refs = _collect_plain(table, s["lens"], s["page"], pool)
    used = refs > 0
    n = int(used.sum())
    src = torch.nonzero(used[n:]).squeeze(1) + n
    dst = torch.nonzero(~used[:n]).squeeze(1)
    to = torch.arange(pool, device="cuda")
    to[src] = dst
    table = torch.where(held, to[table.clamp(min=0).long()].to(I32), table)
    refs[dst] = refs[src]
    refs[n:] = 0
    free = torch.full((pool,), -1, dtype=I32, device="cuda")
    free[:pool - n] = torch.arange(n, pool, dtype=I32, device="cuda")
    pages = _move(s, src, dst)
    moved = torch.full((2, pool // 2), -1, dtype=I32, device="cuda")
    moved[0, :src.shape[0]], moved[1, :src.shape[0]] = src.to(I32), dst.to(I32)
    return dict(pages, table=table, refs=refs.to(I32), free=free, count=_ints([pool - n]),
                src=moved[0], dst=moved[1], moves=_ints([src.shape[0]]))


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    s, kind = state, state["case"]["kind"]
    if not own:
        return {"chunk": _chunk_plain, "act": _act_plain, "down": _down_plain,
                "fork": _fork_plain, "compact": _compact_plain}[kind](s)
    if kind == "chunk":
        s["cache"].attend_chunk(s["q"], s["table"], s["lens"], s["starts"], s["out"],
                                window=s["case"]["window"], sinks=s["sinks"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "act":
        p = s["plan"].update(s["ids"])
        s["experts"].activate(s["x"], p, s["act"])
        return {"order": p.order, "offsets": p.offsets, "places": p.places, "act": s["act"]}
    if kind == "down":
        s["experts"].combine(s["act"], s["plan"], s["w"], s["y"])
        return {"y": s["y"]}
    p = s["pages"]
    pages = {name: s[name] for name in ("k", "v", "codes", "steps")}
    if kind == "fork":
        p.fork(s["parents"], s["children"], s["table"], s["lens"], s["free"])
        s["cache"].copy_pages(p.src, p.dst)
        return dict(pages, table=s["table"], lens=s["lens"], src=p.src, dst=p.dst, taken=p.taken)
    table = s["table"].clone()               # a second pass finds the same pool
    p.compact(table, s["lens"])
    s["cache"].copy_pages(p.src, p.dst, count=p.moves)
    return dict(pages, table=table, refs=p.refs, free=p.free, count=p.count, src=p.src, dst=p.dst,
                moves=p.moves)


def work(case):
    kind = case["kind"]
    if kind == "chunk":
        lens, new = _chunk_lengths(case)
        kv, D, heads, w = case["kv_heads"], case["dim"], case["heads"], case["window"]
        seen = pairs = pages = 0
        for n, m in zip(lens, new):
            if m == 0:
                continue
            first = max(0, n - m + 1 - w) if w else 0
            seen += n - first
            pages += -(-n // case["page"]) - first // case["page"]
            # token at position p sees min(p + 1, w) keys
            if w:
                full = min(m, max(0, n - w))
                pairs += full * w
                short = m - full
            else:
                short = m
            top = n if not w else min(n, n - (m - short))
            pairs += short * top - short * (short - 1) // 2
        T = sum(new)
        b = 2 * T * heads * D * SIZE[case["q"]] + 4 * T * heads + 8 * len(lens) + 4 * pages
        return {"bytes": b + 2 * seen * kv * D * SIZE[case["cache"]], "flops": 4 * pairs * heads * D}
    if kind in ("act", "down"):
        T, H, I, E, k = (case[n] for n in ("tokens", "hidden", "inter", "experts", "topk"))
        pairs = T * k
        # experts that some pair asks for, about
        asked = E * (1.0 - (1.0 - k / E) ** T)
        if kind == "act":
            b = 2 * (T * H + pairs * I) + 4 * (3 * pairs + E)
            return {"bytes": int(b + asked * 4 * H * I), "flops": 4 * pairs * H * I}
        return {"bytes": int(2 * (T * H + pairs * I) + 12 * pairs + asked * 2 * H * I),
                "flops": 2 * pairs * H * I}
    page, kv, D, e = case["page"], case["kv_heads"], case["dim"], SIZE[case["cache"]]
    whole = kv * (2 * page * D * e + 2 * D + 4)               # a page and its summary
    if kind == "fork":
        lens, parents = _forks(case)
        held = sum(-(-lens[p] // page) for p in parents)
        cut = sum(1 for p in parents if lens[p] % page)
        return {"bytes": 8 * held + 20 * len(parents) + 2 * cut * whole, "flops": held}
    lens, ended = _lengths(case, case["longest"], "held"), _ended(case)
    held = [-(-n // page) for n in lens]
    pool, used = sum(held) + 5, sum(h for h, e in zip(held, ended) if not e)
    # a page in use lies behind the first `used` ones with this share
    moves = used * (pool - used) // pool
    return {"bytes": 12 * used + 16 * pool + 2 * moves * whole, "flops": used + pool}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_chunk(s):
    T, heads, dim = s["q"].shape
    kv, page, window = s["k"].shape[1], s["page"], s["case"]["window"]
    G = heads // kv
    out = torch.zeros((T, heads, dim), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, heads), dtype=torch.float64, device="cuda")
    lens, starts = s["host"]
    for r, n in enumerate(lens):
        m = starts[r + 1] - starts[r]
        if m == 0:
            continue
        lo = max(0, n - m + 1 - window) if window else 0
        at = torch.arange(lo, n, device="cuda")
        where = s["table"][r].long()[at // page], at % page
        for h in range(kv):
            k, v = (_take(s[name], where[0], h, where[1]).double() for name in ("k", "v"))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for g in range(h * G, h * G + G):
                for i in range(0, m, 4096):
                    t = torch.arange(i, min(i + 4096, m), device="cuda")
                    pos = (n - m + t)[:, None]
                    rows = starts[r] + t
                    x = s["q"][rows, g].double() @ k.T / math.sqrt(dim)
                    hidden = at[None, :] > pos
                    if window:
                        hidden |= at[None, :] <= pos - window
                    x[hidden] = -math.inf
                    if s["sinks"] is not None:
                        x = torch.cat([x, s["sinks"][g].double().expand(x.shape[0], 1)], 1)
                    norm = torch.logsumexp(x, 1)
                    out[rows, g] = torch.exp(x[:, :n - lo] - norm[:, None]) @ v
                    lse[rows, g] = norm
    return {"out": out, "lse": lse}


def _exact_pairs(ids):
    """For every expert the pairs that ask for it, ascending, on the host."""
    flat, lists = ids.reshape(-1).tolist(), {}
    for pair, e in enumerate(flat):
        lists.setdefault(e, []).append(pair)
    return lists


def _exact_act(s):
    E, topk = s["case"]["experts"], s["case"]["topk"]
    lists, order, offsets = _exact_pairs(s["ids"]), [], [0]
    act = torch.empty(s["act"].shape, dtype=torch.float64, device="cuda")
    for e in range(E):
        mine = lists.get(e, [])
        if mine:
            x = s["x"][torch.tensor(mine, device="cuda") // topk].double()
            g, v = (torch.einsum("th,ih->ti", x, s[name][e].double()) for name in ("gate", "up"))
            act[len(order):len(order) + len(mine)] = g * torch.special.expit(g) * v
        order += mine
        offsets.append(len(order))
    places = [0] * len(order)
    for row, pair in enumerate(order):
        places[pair] = row
    return {"order": _ints(order), "offsets": _ints(offsets),
            "places": _ints(places).view(s["ids"].shape), "act": act}


def _exact_down(s):
    topk, at = s["case"]["topk"], 0
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    w = s["w"].double().reshape(-1)
    for e, mine in sorted(_exact_pairs(s["ids"]).items()):
        pairs = torch.tensor(mine, device="cuda")
        z = s["act"][at:at + len(mine)].double() @ s["down"][e].double().T
        # a token asks for an expert once: no two rows of z meet
        y[pairs // topk] += w[pairs, None] * z
        at += len(mine)
    return {"y": y}


def _exact_moves(s, moves):
    out = {}
    for name in ("k", "v", "codes", "steps"):
        bits = s[name] if s[name].element_size() > 1 else s[name].view(torch.uint8)
        bits = bits.clone()
        for a, b in moves:
            bits[b] = (s[name] if s[name].element_size() > 1 else s[name].view(torch.uint8))[a]
        out[name] = bits.view(s[name].dtype)
    return out


def _exact_fork(s):
    page, free = s["page"], s["free"].tolist()
    table, lens = s["table"].tolist(), s["lens"].tolist()
    src, dst, used = [], [], 0
    for p, c in zip(s["parents"].tolist(), s["children"].tolist()):
        lens[c] = lens[p]
        for i in range(-(-lens[p] // page)):
            table[c][i] = table[p][i]
        src.append(-1)
        dst.append(-1)
        if lens[p] % page:
            src[-1], dst[-1] = table[p][lens[p] // page], free[used]
            table[c][lens[p] // page] = free[used]
            used += 1
    out = _exact_moves(s, [(a, b) for a, b in zip(src, dst) if a >= 0])
    return dict(out, table=_ints(table), lens=_ints(lens), src=_ints(src), dst=_ints(dst),
                taken=_ints([used]))


def _exact_compact(s):
    page, pool, table = s["page"], s["pool"], s["table"].tolist()
    refs = [0] * pool
    for row, n in zip(table, s["lens"].tolist()):
        for i in range(-(-n // page)):
            refs[row[i]] += 1
    used = sum(1 for n in refs if n)
    src = [p for p in range(used, pool) if refs[p]]
    dst = [p for p in range(used) if not refs[p]]
    to = dict(zip(src, dst))
    for row, n in zip(table, s["lens"].tolist()):
        for i in range(-(-n // page)):
            row[i] = to.get(row[i], row[i])
    for a, b in zip(src, dst):
        refs[a], refs[b] = 0, refs[a]
    out = _exact_moves(s, list(zip(src, dst)))
    fill = lambda v, n: _ints(v + [-1] * (n - len(v)))  # noqa: E731
    return dict(out, table=_ints(table), refs=_ints(refs), free=fill(list(range(used, pool)), pool),
                count=_ints([pool - used]), src=fill(src, pool // 2), dst=fill(dst, pool // 2),
                moves=_ints([len(src)]))


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"chunk": _exact_chunk, "act": _exact_act, "down": _exact_down, "fork": _exact_fork,
            "compact": _exact_compact}[case["kind"]](s)
