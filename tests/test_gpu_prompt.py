"""The operators that take a prompt through the block (attention of a chunk,
experts' grouped products, pages forked and compacted) against their
definitions in 64 bits, at the sizes and masks where they can go wrong, and
their device error bits.

Tolerances follow from the arithmetic: u = half an ulp of a type relative to
the value (bf16 2^-8, fp16 2^-11, fp32 2^-24).  Attention as in the decode
step's tests: with A = the weighted mean of |v| an output is within (u_weights
+ 2 d + 2^-20) A + u_out |o|, where d = (D + 16) 2^-24 scale sum |q k| bounds a
logit's error; fp16 weights below 2^-24 of the row's largest are lost.  A
product of n terms in fp32 is off by n 2^-23 of the sum of its terms'
magnitudes at most (each addition by an ulp: tensor instructions truncate)."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from calibration_free_sparse_gb300 import block, experts
    from calibration_free_sparse_gb300 import reader as rd

BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HALF_ULP = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}
I32 = torch.int32


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(v):
    return torch.as_tensor(np.asarray(v), dtype=I32).cuda()


# --------------------------------------------------------------------------
# attention of a chunk
# --------------------------------------------------------------------------
class Chunk:
    """A paged cache whose unwritten rows are NaN, with the new tokens' queries
    as a slice of a wider matrix whose other columns are NaN."""

    def __init__(self, lens, new, kv, group, dim, page, cache, qt, seed=0, pool_extra=3, width=None,
                 drift=0.0):
        g = torch.Generator().manual_seed(seed)
        held = [-(-n // page) for n in lens]
        pool = sum(held) + pool_extra
        order = torch.randperm(pool, generator=g).tolist()
        self.table_np = np.full((len(lens), width or max(held + [1]) + 1), -1, np.int32)
        shape = (pool, kv, page, dim)
        k, v = torch.full(shape, math.nan), torch.full(shape, math.nan)
        self.scales = [None, None]
        if cache == E4:
            self.scales = [0.01 + 0.01 * torch.rand(kv, generator=g) for _ in range(2)]
        at = 0
        for r, n in enumerate(lens):
            self.table_np[r, :held[r]] = order[at:at + held[r]]
            at += held[r]
            for c, sc in ((k, self.scales[0]), (v, self.scales[1])):
                rows = torch.randn(held[r] * page, kv, dim, generator=g)
                if c is k and drift:
                    rows += drift * torch.linspace(-1, 1, max(1, held[r] * page))[:, None, None]
                if sc is not None:
                    rows = (rows / sc[:, None]).clamp(-448, 448)
                rows[n:] = math.nan
                for p in range(held[r]):
                    c[self.table_np[r, p]] = rows[p * page:(p + 1) * page].transpose(0, 1)
        self.k, self.v = k.to(cache).cuda(), v.to(cache).cuda()
        self.lens, self.new, self.page, self.group, self.kv = list(lens), list(new), page, group, kv
        self.heads, self.dim, self.qt = kv * group, dim, qt
        self.starts_np = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.table, self.lens_t, self.starts = (ints(x) for x in (self.table_np, lens,
                                                                  self.starts_np))
        self.scales = [None if s is None else s.cuda() for s in self.scales]
        self.cache = block.PagedCache(self.k, self.v, self.heads, max_requests=len(lens),
                                      k_scale=self.scales[0], v_scale=self.scales[1])
        T = int(self.starts_np[-1])
        wide = torch.full((T, self.heads + 2 * kv, dim), math.nan)
        wide[:, kv:kv + self.heads] = 1.3 * torch.randn(T, self.heads, dim, generator=g)
        self.q = wide.to(qt).cuda()[:, kv:kv + self.heads]
        self.T = T

    def rows(self, r, h, at):
        where = torch.from_numpy(self.table_np[r, at // self.page]).long().cuda()
        off = torch.from_numpy(at % self.page).long().cuda()
        out = []
        for c, s in ((self.k, self.scales[0]), (self.v, self.scales[1])):
            bits = c if c.element_size() > 1 else c.view(torch.uint8)
            x = bits[where, h, off].view(c.dtype).float().double()
            out.append(x if s is None else x * s[h].double())
        return out

    def run(self, out=None, lse=None, **kw):
        out = torch.full((self.T, self.heads, self.dim), math.nan, dtype=self.qt,
                         device="cuda") if out is None else out
        lse = torch.full((self.T, self.heads), math.nan, device="cuda") if lse is None else lse
        self.cache.attend_chunk(self.q, self.table, self.lens_t, self.starts, out, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, window=0, sinks=None, scale=None, ignore=()):
        scale = self.dim ** -0.5 if scale is None else scale
        for r, (n, m) in enumerate(zip(self.lens, self.new)):
            if m == 0:
                continue
            a = int(self.starts_np[r])
            pos = torch.arange(n - m, n, device="cuda")[:, None]
            at = np.arange(n)
            for h in range(self.kv):
                k, v = self.rows(r, h, at)
                seen = torch.arange(n, device="cuda")[None, :] <= pos
                if window:
                    seen &= torch.arange(n, device="cuda")[None, :] > pos - window
                for g in range(self.group):
                    head = h * self.group + g
                    q = self.q[a:a + m, head].double()
                    # what is not seen takes no part, whatever it holds
                    s = torch.where(seen, scale * q @ k.nan_to_num(0, 0, 0).T, -math.inf)
                    d = torch.where(seen, q.abs() @ k.nan_to_num(0, 0, 0).abs().T, 0.0).amax(1)
                    d = (self.dim + 16) * 2.0 ** -24 * abs(scale) * d[:, None]
                    top = s.amax(1, keepdim=True)
                    sink = None
                    if sinks is not None:
                        sink = sinks[head].double()
                        top = torch.maximum(top, sink)
                    p = torch.exp(s - top)
                    den = p.sum(1, keepdim=True)
                    if sink is not None:
                        den = den + torch.exp(sink - top)
                    vv = v.nan_to_num(0, 0, 0)
                    ref, A = p @ vv / den, p @ vv.abs() / den
                    tol = (HALF_ULP[self.qt] + 2 * d + 2.0 ** -20) * A + \
                        HALF_ULP[self.qt] * ref.abs() + 2.0 ** -24
                    if self.qt == HF:
                        tol = tol + n * 2.0 ** -25 * vv.abs().max()
                    err = (out[a:a + m, head].double() - ref).abs()
                    bad = ~(err <= tol)
                    for t, c in ignore:
                        bad[t - a, c] = False
                    assert not bad.any(), (r, head, float((err / tol).nan_to_num(9e9).max()),
                                           torch.nonzero(bad)[:4].tolist())
                    want = (torch.log(den) + top)[:, 0]
                    off = (lse[a:a + m, head].double() - want).abs()
                    assert (off <= 2 * d[:, 0] + 2.0 ** -20 * (1 + want.abs())).all(), (r, head)


RAGGED = ([1, 40, 0, 300, 17, 128, 129, 513, 5], [1, 40, 0, 7, 1, 128, 2, 260, 0])


@pytest.mark.parametrize("dim,group,cache,qt", [
    (64, 1, BF, BF), (64, 8, HF, HF), (64, 7, E4, HF), (64, 64, BF, BF), (128, 1, HF, HF),
    (128, 8, BF, BF), (128, 16, E4, BF), (128, 12, E4, HF), (128, 33, HF, HF), (256, 1, BF, BF),
    (256, 5, HF, HF), (256, 8, E4, BF)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_chunk_ragged(dim, group, cache, qt, page):
    """Whole prompts, chunks and single tokens in one call, around tile and
    page ends; requests without tokens or without new ones."""
    c = Chunk(*RAGGED, 2, group, dim, page, cache, qt, seed=dim + group)
    out, lse = c.run()
    assert c.cache.status() == (0, 0)
    c.check(out, lse)
    again, _ = c.run()
    assert torch.equal(out, again)


@pytest.mark.parametrize("lens,new,kv,group", [
    ([1], [1], 1, 1), ([2000], [2000], 1, 4), ([5000], [3], 2, 8), ([9001], [130], 1, 2),
    ([3000, 40, 700], [64, 40, 1], 4, 8), ([700] * 24, [5] * 24, 2, 4), ([640] * 40, [90] * 40, 4, 8)])
@pytest.mark.parametrize("cache", [BF, E4])
def test_chunk_shares(lens, new, kv, group, cache):
    """Long rows split between CTAs, whole rows dealt, one and many."""
    c = Chunk(lens, new, kv, group, 128, 32, cache, BF, seed=3)
    out, lse = c.run()
    assert c.cache.status() == (0, 0)
    c.check(out, lse)
    again, _ = c.run()
    assert torch.equal(out, again)


@pytest.mark.parametrize("dim,qt,cache", [(64, HF, HF), (128, BF, E4), (256, BF, BF)])
@pytest.mark.parametrize("window", [1, 16, 100, 128, 129, 5000])
@pytest.mark.parametrize("with_sinks", [False, True])
def test_chunk_windows_and_sinks(dim, qt, cache, window, with_sinks):
    c = Chunk([600, 130, 1, 257], [600, 4, 1, 129], 2, 4, dim, 32, cache, qt, seed=window)
    sinks = None
    if with_sinks:
        sinks = torch.tensor([0.3, -2.0, 9.0, -math.inf, 0.0, 1.0, 30.0, -40.0], device="cuda")
    # pages before every window are gone
    for r, (n, m) in enumerate(zip(c.lens, c.new)):
        gone = max(0, n - m + 1 - window) // c.page
        c.table[r, :gone] = -7
    out, lse = c.run(window=window, sinks=sinks)
    assert c.cache.status() == (0, 0)
    c.check(out, lse, window=window, sinks=sinks)


@pytest.mark.parametrize("scale", [0.0, -0.11, 1.7])
def test_chunk_scales(scale):
    c = Chunk([300, 77], [300, 5], 1, 8, 128, 64, BF, BF)
    out, lse = c.run(scale=scale)
    c.check(out, lse, scale=scale)


@pytest.mark.parametrize("cache,qt", [(BF, BF), (HF, HF), (E4, HF)])
def test_chunk_logits_that_climb(cache, qt):
    """The maximum moves by much from tile to tile, in both directions."""
    for drift in (6.0, -6.0):
        c = Chunk([1500, 400], [700, 400], 1, 4, 64, 16, cache, qt, drift=drift)
        out, lse = c.run()
        c.check(out, lse)


@pytest.mark.parametrize("dim,cache,qt", [(64, BF, BF), (128, HF, HF), (256, BF, BF), (128, E4, BF)])
@pytest.mark.parametrize("new", [70, 513])
def test_chunk_later_tokens_do_not_leak(dim, cache, qt, new):
    """Keys and values of NaN and infinity reach the rows that see them only."""
    n = 600
    c = Chunk([n], [new], 2, 4, dim, 32, cache, qt)
    first, at = n - new, n - new + 61                  # the token that holds them
    page, off = int(c.table_np[0, at // 32]), at % 32
    c.v[page, 0, off, 5] = math.nan
    if cache != E4:
        c.v[page, 0, off, 6] = math.inf
    c.k[page, 1, off, 3] = math.nan
    out, lse = c.run()
    o, l = out.double(), lse.double()
    assert o[:at - first].isfinite().all() and l[:at - first].isfinite().all()
    late = o[at - first:]
    assert late[:, :4, 5].isnan().all()
    if cache != E4:
        assert (late[:, :4, 6] == math.inf).all()
    keep = [i for i in range(dim) if i not in (5, 6)]
    assert late[:, :4, keep].isfinite().all()
    assert late[:, 4:].isnan().all() and l[at - first:, 4:].isnan().all()
    assert l[:, :4].isfinite().all()
    # the finite ones are right
    c.k[page, 1, off, 3] = 0
    c.v[page, 0, off, 5:7] = 0
    clean, clean_lse = c.run()
    c.check(clean, clean_lse)
    o, clean = o[..., keep], clean.double()[..., keep]
    ok = o.isfinite()
    assert (o[ok] - clean[ok]).abs().max() <= 4 * HALF_ULP[qt] * clean.abs().max()


def test_chunk_rows_outside_are_left_alone():
    c = Chunk([64, 50], [20, 30], 1, 4, 64, 16, BF, BF)
    T = 60
    q = torch.full((T, 4, 64), math.nan, dtype=BF, device="cuda")
    q[4:54] = c.q
    out = torch.full((T, 4, 64), 7.0, dtype=BF, device="cuda")
    lse = torch.full((T, 4), 7.0, device="cuda")
    c.cache.attend_chunk(q, c.table, c.lens_t, c.starts + 4, out, lse=lse)
    assert (out[:4] == 7).all() and (out[54:] == 7).all()
    assert (lse[:4] == 7).all() and (lse[54:] == 7).all()
    c.check(out[4:54], lse[4:54])


def test_chunk_agrees_with_attend():
    """One new token a request: the decode step's attention."""
    lens = [1, 5, 64, 700, 1300]
    c = Chunk(lens, [1] * 5, 2, 8, 128, 32, BF, BF)
    out, lse = c.run()
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    c.cache.attend(c.q, c.table, c.lens_t, o2, lse=l2)
    c.check(out, lse)
    assert (lse - l2).abs().max() < 1e-4
    assert (out.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * o2.float().abs().max()


def test_chunk_strides_and_alignment():
    """Head-major, odd-offset and broadcast queries."""
    c = Chunk([200, 90], [50, 90], 2, 4, 64, 16, HF, HF)
    want, _ = c.run()
    T = c.T
    flat = torch.empty(T * 8 * 64 + 3, dtype=HF, device="cuda")
    odd = flat[3:].view(8, T, 64)
    odd.copy_(c.q.transpose(0, 1))
    c.q = odd.transpose(0, 1)
    got, _ = c.run()
    assert torch.equal(got, want)
    one = c.q[:1].expand(T, 8, 64)
    c.q = one
    got, lse = c.run()
    c.check(got, lse)


def test_chunk_device_errors():
    """Lengths and pages that do not fit are cut, skipped and reported."""
    L, P = block.ERR_LENGTH, block.ERR_PAGE
    c = Chunk([200, 64], [40, 8], 1, 4, 64, 16, BF, BF)
    good, _ = c.run()
    # a page that is not in the pool is skipped
    c.table[0, 3] = 10 ** 6
    out, _ = c.run()
    assert c.cache.status() == (rd.EDEVICE, P)
    assert torch.equal(out[40:], good[40:]) and out[:40].isfinite().all()
    assert not torch.equal(out[:40], good[:40])
    c.table[0, 3] = int(c.table_np[0, 3])
    # fewer tokens than new ones: rows of nothing in front
    c.lens_t[1] = 5
    out, lse = c.run()
    assert c.cache.status() == (rd.EDEVICE, L)
    assert (out[40:43] == 0).all() and (lse[40:43] == -math.inf).all()
    assert torch.equal(out[:40], good[:40]) and out[43:].isfinite().all()
    c.lens_t[1] = -3
    out, lse = c.run()
    assert c.cache.status() == (rd.EDEVICE, L)
    assert (out[40:] == 0).all()
    c.lens_t[1] = 64
    # starts beyond the rows
    c.starts[2] = 10 ** 6
    out, _ = c.run()
    assert c.cache.status()[1] == L
    c.starts[2] = 48
    # keys beyond the table do not exist
    short = c.table[:, :5].contiguous()
    out = torch.empty_like(good)
    c.cache.attend_chunk(c.q, short, c.lens_t, c.starts, out)
    assert c.cache.status() == (rd.EDEVICE, L)
    assert out.isfinite().all() and torch.equal(out[40:], good[40:])
    again, _ = c.run()
    assert torch.equal(again, good) and c.cache.status() == (0, 0)


def test_chunk_offsets_beyond_32_bits():
    """Pages whose elements lie behind 2^32."""
    page, kv, dim = 256, 8, 256
    pool = (1 << 32) // (page * kv * dim) + 2
    k = torch.zeros((pool, kv, page, dim), dtype=E4, device="cuda")
    v = torch.zeros_like(k)
    one = torch.ones(kv, device="cuda")
    cache = block.PagedCache(k, v, kv, max_requests=1, k_scale=one, v_scale=one)
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((2, kv, page, dim), generator=g, device="cuda")
    for i, p in enumerate((pool - 1, pool - 2)):
        k[p], v[p] = rows[0].to(E4), rows[1].to(E4)
    table = ints([[pool - 1, pool - 2]])
    q = torch.randn((3, kv, dim), generator=g, device="cuda").to(BF)
    out = torch.empty_like(q)
    cache.attend_chunk(q, table, ints([512]), ints([0, 3]), out)
    keys, vals = (torch.cat([c[pool - 1], c[pool - 2]], 1).float().double() for c in (k, v))
    s = torch.einsum("thd,hnd->htn", q.double(), keys) / 16
    s = s.masked_fill(torch.arange(512, device="cuda") > torch.arange(509, 512,
                                                                      device="cuda")[:, None],
                      -math.inf)
    ref = torch.einsum("htn,hnd->thd", s.softmax(-1), vals)
    assert (out.double() - ref).abs().max() <= 2.0 ** -7 * vals.abs().max()
    # and the copy of such a page
    cache.copy_pages(ints([pool - 1]), ints([3]))
    assert torch.equal(k[3].view(torch.uint8), k[pool - 1].view(torch.uint8))
    assert torch.equal(v[3].view(torch.uint8), v[pool - 1].view(torch.uint8))


def test_chunk_on_another_stream_and_captured():
    c = Chunk([3000, 65], [33, 65], 2, 8, 128, 64, BF, BF)
    want, want_lse = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    c.cache.attend_chunk(c.q, c.table, c.lens_t, c.starts, out, lse=lse, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        c.cache.attend_chunk(c.q, c.table, c.lens_t, c.starts, out, lse=lse)
        c.cache.attend_chunk(c.q, c.table, c.lens_t, c.starts, out, lse=lse)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # other lengths in the same graph
    c.lens_t[0] = 1000
    graph.replay()
    torch.cuda.synchronize()
    c.lens[0] = 1000
    c.check(out, lse)
    assert c.cache.status() == (0, 0)


# --------------------------------------------------------------------------
# experts
# --------------------------------------------------------------------------
def layer(E, H, I, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: (torch.randn(s, generator=g, device="cuda") / s[-1] ** 0.5).to(dt)  # noqa: E731
    return draw(E, I, H), draw(E, I, H), draw(E, H, I)


def check_plan(ids, E, p):
    flat = ids.reshape(-1).cpu().numpy()
    ok = (flat >= 0) & (flat < E)
    pairs = np.flatnonzero(ok)
    order = pairs[np.argsort(flat[pairs], kind="stable")]
    n = len(order)
    assert np.array_equal(p.order.cpu().numpy()[:n], order)
    assert (p.order.cpu().numpy()[n:] == -1).all()
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))])
    assert np.array_equal(p.offsets.cpu().numpy(), offsets)
    places = np.full(len(flat), -1)
    places[order] = np.arange(n)
    assert np.array_equal(p.places.cpu().numpy().reshape(-1), places)
    assert int(p.skipped) == len(flat) - n
    return order, offsets


def check_experts(ids, w, x, weights, topk, yt, rows_left=7.0):
    gate, up, down = weights
    (E, I, H), dt = gate.shape, gate.dtype
    T = ids.shape[0]
    plan = experts.ExpertPlan(E, topk, max(T, 1), hidden=H).update(ids)
    order, offsets = check_plan(ids, E, plan)
    ex = experts.Experts(gate=gate, up=up, down=down)
    act = torch.full((T * topk, I), rows_left, dtype=dt, device="cuda")
    ex.activate(x, plan, act)
    pad = torch.full((T, H + 8), rows_left, dtype=yt, device="cuda")
    y = pad[:, :H]
    ex.combine(act, plan, w, y)
    assert ex.status() == (0, 0)
    assert (act[len(order):] == rows_left).all() and (pad[:, H:] == rows_left).all()
    ref_y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    mag_y = torch.zeros_like(ref_y)
    tol_y = torch.zeros_like(ref_y)
    wf = w.double().reshape(-1)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        pairs = torch.from_numpy(order[a:b]).cuda()
        xe = x[pairs // topk].double()
        G, V, D = (m[e].double() for m in weights)
        g, v = xe @ G.T, xe @ V.T
        dg, dv = (H * 2.0 ** -23 * (xe.abs() @ m.abs().T) for m in (G, V))
        s = torch.special.expit(g)
        ref = g * s * v
        tol = (1.1 * dg + 2.0 ** -20 * (g * s).abs()) * (v.abs() + dv) + (g * s).abs() * dv + \
            HALF_ULP[dt] * ref.abs() + 2.0 ** -24
        err = (act[a:b].double() - ref).abs()
        assert (err <= tol).all(), (e, float((err / tol).max()))
        z, m = act[a:b].double() @ D.T, act[a:b].double().abs() @ D.abs().T
        for j, p in enumerate(pairs.tolist()):
            ref_y[p // topk] += wf[p] * z[j]
            mag_y[p // topk] += (wf[p] * z[j]).abs()
            tol_y[p // topk] += wf[p].abs() * I * 2.0 ** -23 * m[j]
    tol_y += topk * 2.0 ** -23 * mag_y + HALF_ULP[yt] * ref_y.abs() + 2.0 ** -24
    err = (y.double() - ref_y).abs()
    assert (err <= tol_y).all(), float((err / tol_y).max())
    # the same bits again
    act2, y2 = torch.full_like(act, rows_left), torch.empty_like(y)
    ex.activate(x, plan, act2)
    ex.combine(act2, plan, w, y2)
    assert torch.equal(act, act2) and torch.equal(y, y2)


def routing(T, E, topk, seed, skew=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((T, E), generator=g, device="cuda")
    logits += skew * torch.randn((E,), generator=g, device="cuda")
    top = torch.topk(logits, topk)
    return top.indices.to(I32).contiguous(), top.values.softmax(-1).contiguous()


@pytest.mark.parametrize("T,E,topk,H,I,dt,yt", [
    (1, 8, 2, 256, 128, BF, BF), (3, 16, 1, 64, 64, HF, HF), (57, 16, 8, 520, 136, BF, F32),
    (200, 8, 4, 256, 384, BF, BF), (130, 1, 1, 8, 8, HF, F32), (129, 2, 2, 136, 1000, BF, HF),
    (700, 4, 2, 1032, 264, HF, HF), (64, 64, 4, 2880, 72, BF, BF), (1000, 3, 3, 72, 130 * 8, BF, F32)])
@pytest.mark.parametrize("skew", [0.0, 3.0])
def test_experts(T, E, topk, H, I, dt, yt, skew):
    """Ragged numbers of rows, odd widths, each type."""
    ids, w = routing(T, E, topk, T, skew)
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn((T, H + 16), generator=g, device="cuda").to(dt)
    check_experts(ids, w, wide[:, 8:8 + H], layer(E, H, I, dt), topk, yt)


def test_experts_of_nobody():
    """Ids that are no expert, an expert twice in a token, experts without rows."""
    ids = ints([[0, 3], [-1, 5], [7, 7], [100, -5], [3, 0], [7, 8]])
    w = torch.rand((6, 2), device="cuda")
    x = torch.randn((6, 128), device="cuda").to(BF)
    weights = layer(8, 128, 64, BF)
    check_experts(ids, w, x, weights, 2, F32)
    none = torch.full((6, 2), -1, dtype=I32, device="cuda")
    check_experts(none, w, x, weights, 2, BF)


def test_experts_without_tokens():
    weights = layer(4, 64, 64, BF)
    ex = experts.Experts(*weights)
    plan = experts.ExpertPlan(4, 2, 5, hidden=64).update(torch.empty((0, 2), dtype=I32,
                                                                    device="cuda"))
    assert plan.offsets.tolist() == [0] * 5 and int(plan.skipped) == 0
    e = lambda *s, dt=BF: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
    ex.activate(e(0, 64), plan, e(0, 64))
    ex.combine(e(0, 64), plan, e(0, 2, dt=F32), e(0, 64))
    assert ex.status() == (0, 0)


def test_experts_infinities_stay_in_their_rows():
    """NaN and infinity in a token, an activation or a weight reach the rows
    and channels that they belong to and no others."""
    T, E, H, I = 40, 4, 256, 128
    weights = layer(E, H, I, BF)
    ids, w = routing(T, E, 2, 3)
    x = torch.randn((T, H), device="cuda").to(BF)
    plan = experts.ExpertPlan(E, 2, T, hidden=H).update(ids)
    ex = experts.Experts(*weights)
    act, y = torch.empty((T * 2, I), dtype=BF, device="cuda"), torch.empty((T, H), device="cuda")
    ex.activate(x, plan, act)
    ex.combine(act, plan, w, y)
    bad = x.clone()
    bad[7, 100] = math.nan
    act2, y2 = torch.empty_like(act), torch.empty_like(y)
    ex.activate(bad, plan, act2)
    ex.combine(act2, plan, w, y2)
    rows = plan.places[7].long()
    mine = torch.zeros(T * 2, dtype=torch.bool, device="cuda")
    mine[rows] = True
    assert act2[mine].isnan().all() and torch.equal(act2[~mine], act[~mine])
    keep = torch.arange(T, device="cuda") != 7
    assert y2[7].isnan().all() and torch.equal(y2[keep], y[keep])
    weights[2][1, 9, 3] = math.inf
    ex.combine(act, plan, w, y2)
    hit = (ids == 1).any(1)
    assert not y2[hit, 9].isfinite().any() and torch.equal(y2[~hit], y[~hit])
    cols = torch.arange(H, device="cuda") != 9
    assert torch.equal(y2[:, cols], y[:, cols])


def test_experts_captured_and_on_another_stream():
    T, E, H, I = 300, 8, 256, 128
    weights = layer(E, H, I, BF)
    ids, w = routing(T, E, 2, 3)
    x = torch.randn((T, H), device="cuda").to(BF)
    plan = experts.ExpertPlan(E, 2, T, hidden=H)
    ex = experts.Experts(*weights)
    act, y = torch.empty((T * 2, I), dtype=BF, device="cuda"), torch.empty((T, H), device="cuda")

    def step(stream=None):
        plan.update(ids, stream=stream)
        ex.activate(x, plan, act, stream=stream)
        ex.combine(act, plan, w, y, stream=stream)

    step()
    want_act, want = act.clone(), y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    act.zero_(), y.zero_()
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    assert torch.equal(act, want_act) and torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # another batch's routing in the same graph
    ids2, w2 = routing(T, E, 2, 9, 2.0)
    ids.copy_(ids2), w.copy_(w2)
    graph.replay()
    torch.cuda.synchronize()
    got_act, got = act.clone(), y.clone()
    step()
    assert torch.equal(act, got_act) and torch.equal(y, got)
    assert ex.status() == (0, 0)


# --------------------------------------------------------------------------
# pages
# --------------------------------------------------------------------------
def pool_cache(pages, kv=2, page=16, dim=64, dtype=BF, requests=8, summaries=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    bits = lambda: torch.randint(0, 256, (pages, kv, page, dim * dtype.itemsize), generator=g,  # noqa: E731
                                 device="cuda", dtype=torch.int32).to(torch.uint8).view(dtype)
    k, v = bits(), bits()
    codes = steps = None
    if summaries:
        codes = torch.randint(-128, 128, (pages, kv, 2, dim), generator=g, device="cuda",
                              dtype=torch.int32).to(torch.int8)
        steps = torch.rand((pages, kv), generator=g, device="cuda")
    one = torch.ones(kv, device="cuda") if dtype == E4 else None
    return block.PagedCache(k, v, kv, max_requests=requests, codes=codes, steps=steps, k_scale=one,
                            v_scale=one), codes, steps


def plain_refs(table, lens, page, pool):
    refs = np.zeros(pool, np.int64)
    for row, n in zip(table, lens):
        for p in row[:-(-max(0, n) // page)]:
            if 0 <= p < pool:
                refs[p] += 1
    return refs


def random_table(r, rows, width, pool, page, share=False):
    """Rows of distinct pages, some of which further rows share."""
    order, at = r.permutation(pool), 0
    table, lens = np.full((rows, width), -5, np.int32), np.zeros(rows, np.int32)
    for i in range(rows):
        room = min(width, (pool - at)) * page
        lens[i] = r.integers(0, room + 1) // (1 if i % 3 else 2)
        held = -(-int(lens[i]) // page)
        table[i, :held] = order[at:at + held]
        at += held
        if share and i and r.random() < 0.5:
            j = r.integers(0, i)
            n = min(-(-int(lens[j]) // page), held)
            n = int(r.integers(0, n + 1))
            table[i, :n] = table[j, :n]
    return table, lens


@pytest.mark.parametrize("pool", [1, 2, 31, 33, 512, 1000, 16384 * 2 + 77, 70001])
@pytest.mark.parametrize("share", [False, True])
def test_collect_and_compact(pool, share):
    r = np.random.default_rng(pool)
    cache, _, _ = pool_cache(pool, 1, 16, 64, E4, requests=1024, summaries=False)
    rows = min(1024, max(1, pool // 7))
    table, lens = random_table(r, rows, max(1, pool // rows) + 2, pool, 16, share)
    pages = cache.pool()
    pages.collect(ints(table), ints(lens))
    refs = plain_refs(table, lens, 16, pool)
    assert np.array_equal(pages.refs.cpu().numpy(), refs)
    free = np.flatnonzero(refs == 0)
    assert int(pages.count) == len(free)
    assert np.array_equal(pages.free.cpu().numpy()[:len(free)], free)
    assert (pages.free.cpu().numpy()[len(free):] == -1).all()

    t = ints(table)
    pages.compact(t, ints(lens))
    used = int((refs > 0).sum())
    src = [p for p in range(used, pool) if refs[p]]
    dst = [p for p in range(used) if not refs[p]]
    n = int(pages.moves)
    assert n == len(src) and pages.src.tolist()[:n] == src and pages.dst.tolist()[:n] == dst
    assert all(p == -1 for p in pages.src.tolist()[n:] + pages.dst.tolist()[n:])
    to = dict(zip(src, dst))
    want = table.copy()
    for i, m in enumerate(lens):
        for c in range(-(-int(m) // 16)):
            want[i, c] = to.get(int(table[i, c]), table[i, c])
    assert np.array_equal(t.cpu().numpy(), want)
    assert np.array_equal(pages.refs.cpu().numpy(), plain_refs(want, lens, 16, pool))
    assert int(pages.count) == pool - used
    assert pages.free.tolist() == list(range(used, pool)) + [-1] * used
    # nothing is left to move
    pages.compact(t, ints(lens))
    assert int(pages.moves) == 0 and np.array_equal(t.cpu().numpy(), want)
    assert cache.status() == (0, 0)


def test_collect_device_errors():
    cache, _, _ = pool_cache(20)
    pages = cache.pool()
    table, lens = ints([[3, 99, -1, 5], [4, 6, 7, 8]]), ints([64, -2])
    pages.collect(table, lens)
    assert cache.status() == (rd.EDEVICE, block.ERR_PAGE | block.ERR_LENGTH)
    assert pages.refs.tolist() == [1 if p in (3, 5) else 0 for p in range(20)]
    pages.compact(table, ints([1000, 16]))
    assert cache.status() == (rd.EDEVICE, block.ERR_PAGE | block.ERR_LENGTH)
    assert table.tolist() == [[0, 99, -1, 2], [1, 6, 7, 8]] and int(pages.count) == 17
    pages.collect(torch.empty((0, 4), dtype=I32, device="cuda"),
                  torch.empty(0, dtype=I32, device="cuda"))
    assert int(pages.count) == 20 and cache.status() == (0, 0)


def test_fork_and_copy():
    """Children of several parents, at page ends and inside pages, then their
    pages' contents; the rest of the pool stays."""
    page, pool = 16, 40
    for dtype in (BF, E4):
        cache, codes, steps = pool_cache(pool, 3, page, 64, dtype, requests=10)
        table = np.full((10, 6), -9, np.int32)
        lens = np.zeros(10, np.int32)
        for i, n in enumerate((33, 16, 0, 5)):
            lens[i] = n
            table[i, :-(-n // page)] = 10 * i + np.arange(-(-n // page))
        t, ln = ints(table), ints(lens)
        pages = cache.pool(6)
        parents, children = [0, 1, 0, 2, 3, 0], [4, 5, 6, 7, 8, 9]
        before = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), codes,
                                      steps)]
        free = ints([20, 21, 22, 25, 26])
        pages.fork(ints(parents), ints(children), t, ln, free)
        assert pages.src.tolist() == [2, -1, 2, -1, 30, 2]
        assert pages.dst.tolist() == [20, -1, 21, -1, 22, 25] and int(pages.taken) == 4
        want = table.copy()
        want[4, :3], want[6, :3], want[9, :3] = [0, 1, 20], [0, 1, 21], [0, 1, 25]
        want[5, 0], want[8, 0] = 10, 22
        assert np.array_equal(t.cpu().numpy(), want)
        assert ln.tolist() == [33, 16, 0, 5, 33, 16, 33, 0, 5, 33]
        cache.copy_pages(pages.src, pages.dst)
        assert cache.status() == (0, 0)
        for now, was in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), codes, steps),
                            before):
            was[[20, 21, 22, 25]] = was[[2, 2, 30, 2]]
            assert torch.equal(now, was)


def test_fork_device_errors():
    """Rows out of range, twice or parent and child at once; pages that lack."""
    cache, _, _ = pool_cache(30, requests=8)
    pages = cache.pool(8)
    table = ints([[0, 1, 2], [3, 4, 5], [6, 77, 8], [-1, -1, -1], [-1] * 3, [-1] * 3, [-1] * 3])
    lens = ints([40, 16, 20, 0, 0, 0, 0])
    free = ints([10, 11])
    pages.fork(ints([0, 0, 9, 1, 0, 1, -1]), ints([3, 3, 4, 0, 7, -2, 5]), table, lens, free)
    assert cache.status() == (rd.EDEVICE, block.ERR_ROW)
    assert pages.src.tolist() == [2] + [-1] * 6 and pages.dst.tolist() == [10] + [-1] * 6
    assert table[3].tolist() == [0, 1, 10] and table[4:].eq(-1).all() and int(pages.taken) == 1
    assert lens.tolist() == [40, 16, 20, 40, 0, 0, 0] and table[0].tolist() == [0, 1, 2]
    # too few pages, one that is not in the pool, a last page that is not
    lens[3] = 0
    pages.fork(ints([0, 2, 0, 0]), ints([3, 4, 5, 6]), table, lens, ints([10, 11, 31]))
    assert cache.status() == (rd.EDEVICE, block.ERR_POOL | block.ERR_PAGE)
    assert pages.src.tolist() == [2, -1, -1, -1] and pages.dst.tolist() == [10, -1, -1, -1]
    assert table[4].tolist() == [6, 11, -1] and table[5].tolist() == [0, 1, -1]
    assert int(pages.taken) == 3
    lens[0] = 1000
    pages.fork(ints([0]), ints([3]), table, lens, free)
    assert cache.status() == (rd.EDEVICE, block.ERR_LENGTH) and int(lens[3]) == 48
    with pytest.raises(ValueError):
        pages.fork(ints([0] * 9), ints(range(9)), table, lens, free)


@pytest.mark.parametrize("kv,page,dim,dtype,summaries", [
    (1, 16, 64, E4, False), (3, 16, 64, BF, True), (8, 256, 256, HF, True), (5, 32, 128, E4, True)])
def test_copy_pages(kv, page, dim, dtype, summaries):
    cache, codes, steps = pool_cache(12, kv, page, dim, dtype, summaries=summaries)
    arrays = [cache.k.view(torch.uint8), cache.v.view(torch.uint8)]
    arrays += [codes, steps] if summaries else []
    before = [a.clone() for a in arrays]
    cache.copy_pages(ints([3, -1, 4, 5, 2, 99, 3]), ints([7, 8, -1, 5, 9, 1, -4]))
    assert cache.status() == (rd.EDEVICE, block.ERR_PAGE)
    for now, was in zip(arrays, before):
        was[[7, 9]] = was[[3, 2]]
        assert torch.equal(now, was)
    for n, stop in ((ints([1]), 1), (ints([50]), 2), (ints([-3]), 0)):
        cache.copy_pages(ints([0, 1]), ints([10, 11]), count=n)
        for now, was in zip(arrays, before):
            was[[10, 11][:stop]] = was[[0, 1][:stop]]
            assert torch.equal(now, was)
    cache.copy_pages(ints([]).to(I32), ints([]).to(I32))
    assert cache.status() == (0, 0)


def test_pages_through_a_life():
    """Plan, append, fork, diverge, free, compact: every request keeps its keys."""
    kv, page, dim, R = 2, 16, 64, 6
    k = torch.zeros((30, kv, page, dim), dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    cache = block.PagedCache(k, v, 4, max_requests=R)
    table = torch.full((R, 5), -1, dtype=I32, device="cuda")
    lens = torch.zeros(R, dtype=I32, device="cuda")
    plan, pages = cache.plan(table, 200), cache.pool(R)
    g = torch.Generator(device="cuda").manual_seed(0)
    held = {r: torch.empty((0, kv, dim), device="cuda") for r in range(R)}

    def grow(new):
        pages.collect(table, lens)
        plan.update(lens, ints(new), pages.free)
        T = sum(new)
        rows = torch.randn((200, kv, dim), generator=g, device="cuda").to(BF)
        cache.append(rows, rows, plan.slots)
        for r in range(R):
            a, b = int(plan.starts[r]), int(plan.starts[r + 1])
            held[r] = torch.cat([held[r], rows[a:b].float()])
        assert int(plan.starts[R]) == T
        lens.copy_(plan.lens)

    def same():
        for r in range(R):
            n = int(lens[r])
            assert n == held[r].shape[0]
            at = torch.arange(n, device="cuda")
            where = table[r].long()[at // page]
            for c in (k, v):
                assert torch.equal(c[where, :, at % page].float(), held[r])

    grow([33, 16, 40, 0, 0, 0])
    pages.collect(table, lens)
    pages.fork(ints([0, 0, 1]), ints([3, 4, 5]), table, lens, pages.free)
    cache.copy_pages(pages.src, pages.dst)
    held[3], held[4], held[5] = held[0], held[0], held[1]
    same()
    grow([1, 2, 0, 20, 17, 1])                     # the continuations part
    same()
    lens[0] = lens[2] = 0
    held[0] = held[2] = held[0][:0]
    pages.compact(table, lens)
    cache.copy_pages(pages.src, pages.dst, count=pages.moves)
    same()
    used = int((pages.refs > 0).sum())
    assert int(table[[1, 3, 4, 5]].max()) < 30 and int(pages.refs[:used].min()) > 0
    grow([20, 3, 0, 1, 5, 9])
    same()
    assert cache.status() == (0, 0)


def test_pages_captured():
    """Collect, fork and compact with their copies in one graph."""
    cache, _, _ = pool_cache(64, requests=8)
    pages = cache.pool(2)
    table = ints(np.arange(32).reshape(8, 4)[:, ::-1] + 20)
    lens = ints([64, 0, 17, 0, 33, 48, 0, 5])
    t0, l0 = table.clone(), lens.clone()

    def step():
        pages.collect(table, lens)
        pages.fork(ids[0], ids[1], table, lens, pages.free)
        cache.copy_pages(pages.src, pages.dst)
        pages.compact(table, lens)
        cache.copy_pages(pages.src, pages.dst, count=pages.moves)

    ids = ints([0, 2]), ints([1, 3])
    k0 = cache.k.clone()
    step()
    want = [x.clone() for x in (table, lens, pages.refs, pages.free, cache.k)]
    table.copy_(t0), lens.copy_(l0), cache.k.copy_(k0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        table.copy_(t0), lens.copy_(l0), cache.k.copy_(k0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((table, lens, pages.refs, pages.free, cache.k), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert cache.status() == (0, 0)


# --------------------------------------------------------------------------
# refusals of the binding
# --------------------------------------------------------------------------
def test_binding_refusals():
    c = Chunk([64], [8], 1, 4, 64, 16, BF, BF)
    out = torch.empty((8, 4, 64), dtype=BF, device="cuda")
    call = c.cache.attend_chunk
    ok = (c.q, c.table, c.lens_t, c.starts, out)
    for i, bad, err in ((0, c.q.float(), TypeError), (0, c.q.cpu(), TypeError),
                        (0, c.q[:, :3], ValueError), (1, c.table.long(), TypeError),
                        (2, c.lens_t.float(), TypeError), (3, c.starts[:1], ValueError),
                        (3, c.starts.cpu(), TypeError), (4, out[:4], ValueError),
                        (4, out.half(), TypeError), (4, torch.empty((8, 64, 4), dtype=BF,
                                                                    device="cuda").mT, ValueError)):
        args = list(ok)
        args[i] = bad
        with pytest.raises(err):
            call(*args)
    with pytest.raises(rd.ReaderError):
        call(*ok, window=-1)
    big = torch.empty((16, 4, 64), dtype=BF, device="cuda")
    with pytest.raises(rd.ReaderError):
        call(big[:8], c.table, c.lens_t, c.starts, big[4:12])
    with pytest.raises(TypeError):
        call(*ok, sinks=torch.zeros(4, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        call(*ok, lse=torch.zeros((8, 5), device="cuda"))

    gate, up, down = layer(4, 64, 32, BF)
    with pytest.raises(ValueError):
        experts.Experts(gate=gate)
    with pytest.raises(TypeError):
        experts.Experts(down=down.float())
    with pytest.raises(ValueError):
        experts.Experts(gate=gate, up=up, down=gate)
    ex = experts.Experts(gate=gate, up=up)
    plan = experts.ExpertPlan(4, 2, 4)
    ids, w = routing(3, 4, 2, 0)
    plan.update(ids)
    x, act = torch.zeros((3, 64), dtype=BF, device="cuda"), torch.zeros((6, 32), dtype=BF,
                                                                       device="cuda")
    with pytest.raises(rd.ReaderError):
        experts.Experts(down=down).activate(x, plan, act)
    with pytest.raises(ValueError):
        experts.Experts(down=down).combine(act, plan, w, x)
    with pytest.raises(TypeError):
        ex.activate(x.half(), plan, act)
    with pytest.raises(ValueError):
        ex.activate(x, plan, act[:5])
    with pytest.raises(ValueError):
        plan.update(torch.zeros((5, 2), dtype=I32, device="cuda"))
    with pytest.raises(ValueError):
        ex.activate(x, experts.ExpertPlan(5, 2, 4).update(ids), act)
    with pytest.raises(rd.ReaderError):
        big = torch.zeros((6, 64), dtype=BF, device="cuda")
        ex.activate(big[:3], plan, big.view(12, 32)[:6])

    pages = c.cache.pool()
    with pytest.raises(rd.ReaderError):
        pages.collect(pages.refs[:4].view(4, 1), ints([1]))
    with pytest.raises(TypeError):
        c.cache.copy_pages(ints([1]).float(), ints([1]))
    with pytest.raises(ValueError):
        c.cache.copy_pages(ints([1]), ints([1, 2]))


def test_plan_refuses_another_device():
    """A plan made on one device is refused on another."""
    if torch.cuda.device_count() < 2:
        pytest.skip("one GPU")
    plan = experts.ExpertPlan(4, 2, 4)
    with torch.cuda.device(1), pytest.raises(ValueError):
        plan.update(ints([[0, 1]]))
