"""The decode-step operators (paged cache, attention, page selection, residual
norm) against their definitions in 64 bits, at the sizes and masks where they
can go wrong, and their refusals and device error bits.

Tolerances follow from the arithmetic: u = half an ulp of a type relative to
the value (bf16 2^-8, fp16 2^-11, fp32 2^-24).  Attention sums n weighted rows
in fp32 with weights rounded to the product's type, so with A = the weighted
mean of |v| an output is within (u_weights + 2 d + 2^-20) A + u_out |o|, where
d = (D + 16) 2^-24 scale sum |q k| bounds a logit's error; fp16 weights below
2^-24 of the row's largest are lost: n 2^-25 max |v| more."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from calibration_free_sparse_gb300 import block
    from calibration_free_sparse_gb300 import reader as rd

BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HALF_ULP = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def f64(t):
    return t.double().cpu().numpy()


def to_i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


class Cache:
    """A paged cache whose unwritten rows are NaN, its table, and the rows."""

    def __init__(self, lens, kv_heads, dim, page, dtype, seed=0, q_heads=None, summaries=True,
                 spare=3, max_requests=None):
        g = torch.Generator().manual_seed(seed)
        held = [-(-n // page) for n in lens]
        pool = sum(held) + spare
        order = torch.randperm(pool, generator=g).tolist()
        width = max(held + [1]) + 1
        table = np.full((len(lens), width), -1, np.int32)
        shape = (pool, kv_heads, page, dim)
        k, v = torch.full(shape, math.nan), torch.full(shape, math.nan)
        self.k_scale = self.v_scale = None
        if dtype == E4:
            self.k_scale = 0.01 + 0.01 * torch.rand(kv_heads, generator=g)
            self.v_scale = 0.01 + 0.01 * torch.rand(kv_heads, generator=g)
        at = 0
        for r, n in enumerate(lens):
            table[r, :held[r]] = order[at:at + held[r]]
            at += held[r]
            for c, sc in ((k, self.k_scale), (v, self.v_scale)):
                rows = torch.randn(held[r] * page, kv_heads, dim, generator=g)
                rows += 0.7 * torch.randn(held[r], 1, kv_heads, dim,
                                          generator=g).expand(-1, page, -1, -1).reshape(rows.shape)
                if sc is not None:
                    rows = (rows / sc[:, None]).clamp(-448, 448)
                rows[n:] = math.nan
                for p in range(held[r]):
                    c[table[r, p]] = rows[p * page:(p + 1) * page].transpose(0, 1)
        self.k, self.v = k.to(dtype).cuda(), v.to(dtype).cuda()
        self.lens, self.page, self.table_np = list(lens), page, table
        self.table, self.lens_t = to_i32(table), to_i32(lens)
        self.codes = self.steps = None
        if summaries:
            self.codes = torch.zeros((pool, kv_heads, 2, dim), dtype=torch.int8).cuda()
            self.steps = torch.zeros((pool, kv_heads)).cuda()
        sc = [None if s is None else s.cuda() for s in (self.k_scale, self.v_scale)]
        self.scales = sc
        self.q_heads = q_heads or kv_heads
        self.cache = block.PagedCache(self.k, self.v, self.q_heads,
                                      max_requests=max_requests or max(1, len(lens)),
                                      codes=self.codes, steps=self.steps, k_scale=sc[0],
                                      v_scale=sc[1])

    def rows(self, r, head, positions):
        """(k, v) float64 rows of request r at positions."""
        ids = torch.from_numpy(self.table_np[r, positions // self.page]).long().cuda()
        off = torch.from_numpy(positions % self.page).long().cuda()
        out = []
        for c, s in ((self.k, self.scales[0]), (self.v, self.scales[1])):
            bits = c if c.element_size() > 1 else c.view(torch.uint8)
            x = f64(bits[ids, head, off].view(c.dtype).float())
            out.append(x if s is None else x * float(s[head]))
        return out

    def summarise(self):
        """Write every page's summary by appending its own rows again."""
        for r, n in enumerate(self.lens):
            if n == 0:
                continue
            pos = np.arange(n)
            slots = self.table_np[r, pos // self.page] * self.page + pos % self.page
            k16, v16 = [], []
            for c, s, out in ((self.k, self.scales[0], k16), (self.v, self.scales[1], v16)):
                flat = c.float().transpose(1, 2).reshape(-1, c.shape[1], c.shape[3])
                x = flat[torch.from_numpy(slots).long().cuda()]
                out.append(x if s is None else x * s[:, None])
            dt = BF if self.k.dtype == E4 else self.k.dtype
            self.cache.append(k16[0].to(dt).contiguous(), v16[0].to(dt).contiguous(),
                              to_i32(slots))


def queries(R, heads, dim, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (1.3 * torch.randn(R, heads, dim, generator=g)).to(dtype).cuda()


def check_attend(c, q, out, lse=None, window=0, sinks=None, pages=None, scale=None):
    R, heads, dim = q.shape
    kv = c.k.shape[1]
    G = heads // kv
    scale = dim ** -0.5 if scale is None else scale
    weights = c.k.dtype if c.k.dtype != E4 else HF
    o_np, q_np = f64(out), f64(q)
    for r, n in enumerate(c.lens):
        for h in range(kv):
            if pages is None:
                pos = np.arange(max(0, n - window) if window else 0, n)
            else:
                pos = np.concatenate([p * c.page + np.arange(c.page)
                                      for p in pages[r, h] if p >= 0] + [np.zeros(0, int)])
                pos = pos[(pos < n) & (pos >= (max(0, n - window) if window else 0))].astype(int)
            mine = slice(h * G, h * G + G)
            sk = None if sinks is None else f64(sinks)[mine]
            if len(pos) == 0:
                assert np.all(o_np[r, mine] == 0), (r, h)
                if lse is not None:
                    want = np.full(G, -np.inf) if sk is None else sk
                    assert np.array_equal(f64(lse)[r, mine], want)
                continue
            k, v = c.rows(r, h, pos)
            s = scale * q_np[r, mine] @ k.T
            top = s.max(1) if sk is None else np.maximum(s.max(1), sk)
            p = np.exp(s - top[:, None])
            den = p.sum(1) + (0 if sk is None else np.exp(sk - top))
            ref = p @ v / den[:, None]
            A = p @ np.abs(v) / den[:, None]
            d = ((dim + 16) * 2.0 ** -24 * scale * (np.abs(q_np[r, mine]) @ np.abs(k).T)).max(1)
            tol = (HALF_ULP[weights] + 2 * d[:, None] + 2.0 ** -20) * A + \
                HALF_ULP[q.dtype] * np.abs(ref) + 2.0 ** -24
            if weights == HF:
                tol = tol + len(pos) * 2.0 ** -25 * np.abs(v).max()
            err = np.abs(o_np[r, mine] - ref)
            assert np.all(err <= tol), (r, h, float((err / tol).max()))
            if lse is not None:
                want = np.log(den) + top
                assert np.all(np.abs(f64(lse)[r, mine] - want) <=
                              2 * d + 2.0 ** -20 * (1 + np.abs(want))), (r, h)


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------
EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 100, 255, 256, 257, 517]


@pytest.mark.parametrize("dim,group,dtype,qt", [
    (64, 1, BF, BF), (64, 8, HF, HF), (64, 16, E4, BF), (64, 7, E4, HF),
    (128, 1, HF, HF), (128, 8, BF, BF), (128, 16, BF, BF), (128, 12, E4, BF), (128, 4, E4, HF),
    (128, 33, HF, HF), (256, 8, BF, BF), (256, 5, HF, HF), (256, 20, E4, BF)])
@pytest.mark.parametrize("page", [16, 64])
def test_attend_edges(dim, group, dtype, qt, page):
    """Ragged lengths around tile and page ends, an empty and a one-token row."""
    c = Cache(EDGES, 2, dim, page, dtype, seed=dim + group, q_heads=2 * group, summaries=False)
    q = queries(len(EDGES), 2 * group, dim, qt)
    out = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:2], math.nan, device="cuda")
    c.cache.attend(q, c.table, c.lens_t, out, lse=lse)
    assert c.cache.status() == (0, 0)
    check_attend(c, q, out, lse)


@pytest.mark.parametrize("lens,kv", [([1], 1), ([40], 4), ([5000], 1), ([9001], 4),
                                     ([300, 4000, 0, 7], 8), ([129] * 40, 8)])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_attend_splits(lens, kv, dtype):
    """One piece a row, rows split over many CTAs, and shares across rows."""
    c = Cache(lens, kv, 128, 32, dtype, seed=3, q_heads=4 * kv, summaries=False)
    q = queries(len(lens), 4 * kv, 128, BF)
    out, again = torch.empty_like(q), torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device="cuda")
    c.cache.attend(q, c.table, c.lens_t, out, lse=lse)
    c.cache.attend(q, c.table, c.lens_t, again)
    assert torch.equal(out, again)
    check_attend(c, q, out, lse)


@pytest.mark.parametrize("dim,dtype,qt,group", [(64, HF, HF, 16), (128, BF, BF, 8), (128, E4, BF, 5),
                                                (256, BF, BF, 3)])
@pytest.mark.parametrize("lens", [
    [2700 - 40 * i for i in range(20)],                   # rows cut by equal shares
    [1200 - 50 * i for i in range(20)],                   # whole rows per CTA
    [0, 1, 500] + [17 + 3 * i for i in range(61)],        # whole rows per warp
    [3000] + [5] * 40,                                    # one long row among short ones
    [3, 0, 1900] + [40 + i for i in range(50)] + [0, 5000, 1] + [30] * 20 + [7000]])
def test_attend_many_rows(dim, dtype, qt, group, lens):
    """More rows than CTAs, in each way that they are dealt out."""
    c = Cache(lens, 8, dim, 64, dtype, seed=len(lens), q_heads=8 * group, summaries=False)
    q = queries(len(lens), 8 * group, dim, qt)
    out, again = torch.full_like(q, math.nan), torch.empty_like(q)
    lse = torch.full(q.shape[:2], math.nan, device="cuda")
    sinks = torch.linspace(-4, 4, 8 * group).cuda()
    c.cache.attend(q, c.table, c.lens_t, out, lse=lse, sinks=sinks)
    c.cache.attend(q, c.table, c.lens_t, again, sinks=sinks)
    assert torch.equal(out, again) and c.cache.status() == (0, 0)
    check_attend(c, q, out, lse, sinks=sinks)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 300, 100000])
@pytest.mark.parametrize("sinks", [False, True])
def test_attend_window_and_sinks(window, sinks):
    c = Cache(EDGES, 2, 64, 32, HF, seed=5, q_heads=8, summaries=False)
    # rows before the window hold whatever they like
    for r, n in enumerate(c.lens):
        for p in range(max(0, n - window)):
            c.k[c.table_np[r, p // 32], :, p % 32] = math.inf
            c.v[c.table_np[r, p // 32], :, p % 32] = math.nan
    q = queries(len(EDGES), 8, 64, HF)
    sk = torch.linspace(-30, 30, 8).cuda() if sinks else None
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    c.cache.attend(q, c.table, c.lens_t, out, window=window, sinks=sk, lse=lse)
    check_attend(c, q, out, lse, window=window, sinks=sk)


def test_attend_sink_of_infinity_takes_everything():
    c = Cache([70, 0], 1, 64, 16, BF, q_heads=2, summaries=False)
    q, out = queries(2, 2, 64, BF), torch.full((2, 2, 64), 3.0, dtype=BF, device="cuda")
    lse = torch.empty((2, 2), device="cuda")
    c.cache.attend(q, c.table, c.lens_t, out, sinks=torch.tensor([math.inf, 0.0], device="cuda"),
                   lse=lse)
    assert not out[0, 0].any() and not out[1].any() and out[0, 1].any()
    assert lse[0, 0] == math.inf and lse[1].tolist() == [math.inf, 0.0]


def test_attend_refuses_an_output_over_the_queries():
    c = Cache([70, 3], 1, 64, 16, BF, q_heads=2, summaries=False)
    joint = torch.zeros((3, 2, 64), dtype=BF, device="cuda")
    with pytest.raises(rd.ReaderError) as e:
        c.cache.attend(joint[:2], c.table, c.lens_t, joint[1:])
    assert e.value.code == rd.EINVAL
    c.cache.attend(joint[:1], c.table, c.lens_t[:1], joint[1:2])


def test_select_the_widest_table():
    """As many pages as a CTA's memory holds keys for, in whole clusters."""
    held = 49152
    codes = torch.zeros((held, 1, 2, 64), dtype=torch.int8, device="cuda")
    codes[:, 0, 0, 0] = (torch.arange(held, device="cuda") % 119).to(torch.int8)
    steps = torch.ones((held, 1), device="cuda")
    k = torch.zeros((held, 1, 16, 64), dtype=BF, device="cuda")
    cache = block.PagedCache(k, k.clone(), 1, max_requests=1, codes=codes, steps=steps)
    q = torch.zeros((1, 1, 64), dtype=BF, device="cuda")
    q[0, 0, 0] = 1
    pages = torch.empty((1, 1, 500), dtype=torch.int32, device="cuda")
    table = torch.arange(held, dtype=torch.int32, device="cuda").reshape(1, -1)
    cache.select(q, table, to_i32([held * 16]), pages, first=0, last=0)
    # 413 pages score 118, then the first 87 that score 117
    top = np.arange(held) % 119
    want = np.sort(np.concatenate([np.flatnonzero(top == 118), np.flatnonzero(top == 117)[:500 - int((top == 118).sum())]]))
    assert np.array_equal(pages.cpu().numpy()[0, 0], want)
    wide = torch.zeros((1, held + 1), dtype=torch.int32, device="cuda")
    with pytest.raises(rd.ReaderError):
        cache.select(q, wide, to_i32([16]), pages)
    assert cache.status() == (0, 0)


def test_attend_sinks_of_minus_infinity_change_nothing():
    c = Cache([70, 0], 1, 64, 16, BF, q_heads=2, summaries=False)
    q = queries(2, 2, 64, BF)
    a, b = torch.empty_like(q), torch.empty_like(q)
    c.cache.attend(q, c.table, c.lens_t, a)
    c.cache.attend(q, c.table, c.lens_t, b, sinks=torch.full((2,), -math.inf, device="cuda"))
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, E4])
def test_attend_pages_given(dtype):
    """Any list of pages: holes, one page, none, the partial last page."""
    c = Cache([200, 97, 16, 0], 2, 128, 16, dtype, seed=9, q_heads=6, summaries=False)
    pages = np.full((4, 2, 5), -1, np.int32)
    pages[0, 0] = [0, 3, 7, 11, 12]
    pages[0, 1] = [12, -1, 2, -1, -1]
    pages[1, 0] = [6, -1, -1, -1, -1]
    pages[2, 1, 0] = 0
    q = queries(4, 6, 128, BF)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    c.cache.attend(q, c.table, c.lens_t, out, lse=lse, pages=to_i32(pages))
    assert c.cache.status() == (0, 0)
    check_attend(c, q, out, lse, pages=pages)
    c.cache.attend(q, c.table, c.lens_t, out, lse=lse, pages=to_i32(pages), window=50)
    check_attend(c, q, out, lse, pages=pages, window=50)


def test_attend_strided_queries_scale_and_stream():
    """q as a slice of a joint projection at an odd offset, on another stream."""
    c = Cache([50, 333, 7], 2, 64, 16, BF, q_heads=4, summaries=False)
    joint = queries(3, 13, 64, BF)
    q = torch.as_strided(joint, (3, 4, 64), (13 * 64, 128, 1), 33)
    out = torch.empty((3, 4, 64), dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.cache.attend(q, c.table, c.lens_t, out, scale=0.3)
    torch.cuda.current_stream().wait_stream(side)
    check_attend(c, q, out, scale=0.3)


def test_attend_beyond_32_bit_offsets():
    """Pages whose byte offset passes 2^32 (and element offset 2^31)."""
    pages, kv, page, dim = 16400, 4, 256, 128
    shape = (pages, kv, page, dim)
    k, v = (torch.empty(shape, dtype=BF, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    ids = [pages - 1, 3, pages - 2]
    for i in ids:
        k[i] = torch.randn(kv, page, dim, device="cuda").to(BF)
        v[i] = torch.randn(kv, page, dim, device="cuda").to(BF)
    codes = torch.zeros((pages, kv, 2, dim), dtype=torch.int8, device="cuda")
    steps = torch.zeros((pages, kv), device="cuda")
    cache = block.PagedCache(k, v, 8, max_requests=1, codes=codes, steps=steps)
    table = to_i32([ids])
    slot = (pages - 2) * page + 99
    row = torch.randn(1, kv, dim, device="cuda").to(BF)
    cache.append(row, -row, to_i32([slot]))
    assert torch.equal(k[pages - 2, :, 99], row[0]) and torch.equal(v[pages - 2, :, 99], -row[0])
    assert steps[pages - 2].min() > 0 and int((steps != 0).sum()) == kv
    q, out = queries(1, 8, dim, BF), torch.empty((1, 8, dim), dtype=BF, device="cuda")
    n = 2 * page + 100
    cache.attend(q, table, to_i32([n]), out)
    kk, vv = (torch.cat([c[i] for i in ids], 1)[:, :n].double() for c in (k, v))
    s = torch.einsum("ghd,gnd->ghn", q[0].double().reshape(4, 2, dim), kk) * dim ** -0.5
    ref = torch.einsum("ghn,gnd->ghd", s.softmax(-1), vv).reshape(8, dim)
    assert (out[0].double() - ref).abs().max() <= (2.0 ** -8) * 3 * vv.abs().max()
    assert cache.status() == (0, 0)


def test_attend_error_bits():
    c = Cache([40, 100, 30], 1, 64, 16, BF, q_heads=2, summaries=False)
    q, out = queries(3, 2, 64, BF), torch.empty((3, 2, 64), dtype=BF, device="cuda")
    room = c.table.shape[1] * 16
    c.cache.attend(q, c.table, to_i32([-4, 100, 30]), out)
    assert c.cache.status() == (rd.EDEVICE, block.ERR_LENGTH)
    assert bool((out[0] == 0).all())
    assert c.cache.status() == (0, 0)
    c.cache.attend(q, c.table, to_i32([40, room + 1, 30]), out)
    code, bits = c.cache.status()      # the entry behind the row's pages is -1
    assert code == rd.EDEVICE and bits == block.ERR_LENGTH | block.ERR_PAGE
    # an id outside the pool is skipped: the row attends to its other pages
    bad = c.table.clone()
    bad[1, 2] = c.k.shape[0]
    c.cache.attend(q, bad, c.lens_t, out)
    assert c.cache.status() == (rd.EDEVICE, block.ERR_PAGE)
    ref = torch.empty_like(out)
    pages = np.full((3, 1, 7), -1, np.int32)
    pages[0, 0, :3], pages[2, 0, :2] = np.arange(3), np.arange(2)
    pages[1, 0, :6] = [0, 1, 3, 4, 5, 6]
    c.cache.attend(q, c.table, c.lens_t, ref, pages=to_i32(pages))
    check_attend(c, q, out, pages=pages)
    check_attend(c, q, ref, pages=pages)
    # a listed page beyond the request's
    pages[0, 0, 3] = 5
    c.cache.attend(q, c.table, c.lens_t, ref, pages=to_i32(pages))
    assert c.cache.status() == (rd.EDEVICE, block.ERR_PAGE)


# --------------------------------------------------------------------------
# plan
# --------------------------------------------------------------------------
def brute_plan(prev, new, table, free, page, max_tokens):
    table, slots, pos, req, starts, used = table.copy(), [], [], [], [0], 0
    for r in range(len(prev)):
        for p in range(prev[r], prev[r] + new[r]):
            if p % page == 0:
                table[r, p // page] = free[used]
                used += 1
            slots.append(table[r, p // page] * page + p % page)
            pos.append(p)
            req.append(r)
        starts.append(len(slots))
    pad = [-1] * (max_tokens - len(slots))
    return table, slots + pad, pos + pad, req + pad, starts, used


@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("R,longest,most", [(1, 0, 1), (1, 31, 1), (5, 40, 40), (33, 300, 1),
                                            (300, 50, 64), (1024, 100, 3)])
def test_plan(R, longest, most, page):
    rng = np.random.default_rng(R + page)
    prev, new = rng.integers(0, longest + 1, R), rng.integers(0, most + 1, R)
    new[0] = most
    width = -(-(longest + most) // page) + 1
    held = -(-prev // page)
    pool = int(held.sum() + (-(-(prev + new) // page) - held).sum()) + 5
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((R, width), -7, np.int32)
    at = 0
    for r in range(R):
        table[r, :held[r]] = order[at:at + held[r]]
        at += held[r]
    kv = torch.zeros((pool, 1, page, 64), dtype=BF, device="cuda")
    cache = block.PagedCache(kv, kv.clone(), 1, max_requests=R)
    tokens = int(new.sum()) + 9
    plan = cache.plan(to_i32(table), tokens)
    plan.update(to_i32(prev), to_i32(new), to_i32(order[at:]))
    ref = brute_plan(prev, new, table, order[at:], page, tokens)
    got = [plan.table, plan.slots, plan.positions, plan.requests, plan.starts, plan.taken]
    for g, w in zip(got, ref):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w, np.int32).reshape(-1))
    assert np.array_equal(plan.lens.cpu().numpy(), prev + new)
    assert cache.status() == (0, 0)


def test_plan_error_bits():
    kv = torch.zeros((8, 1, 16, 64), dtype=BF, device="cuda")
    cache = block.PagedCache(kv, kv.clone(), 1, max_requests=4)
    fresh = lambda: to_i32(np.full((4, 3), -1))  # noqa: E731
    plan = cache.plan(fresh(), 64)
    # the pool runs out: the second request's pages are missing
    plan.update(to_i32([0, 0]), to_i32([20, 20]), to_i32([5, 6, 7]))
    assert cache.status() == (rd.EDEVICE, block.ERR_POOL)
    assert plan.table.cpu().tolist()[:2] == [[5, 6, -1], [7, -1, -1]]
    s = plan.slots.cpu().numpy()
    assert np.array_equal(s[20:36], 7 * 16 + np.arange(16)) and np.all(s[36:] == -1)
    assert int(plan.taken) == 3
    # a row that outgrows the table, a negative length
    plan = cache.plan(fresh(), 64)
    plan.update(to_i32([0, -3]), to_i32([60, 4]), to_i32(np.arange(8)))
    assert cache.status() == (rd.EDEVICE, block.ERR_LENGTH)
    assert plan.lens.cpu().tolist() == [48, 4] and plan.starts.cpu().tolist() == [0, 48, 52]
    # more tokens than the plan holds
    plan = cache.plan(fresh(), 8)
    plan.update(to_i32([0, 0]), to_i32([6, 6]), to_i32(np.arange(8)))
    assert cache.status() == (rd.EDEVICE, block.ERR_LENGTH)
    assert plan.requests.cpu().tolist() == [0] * 6 + [1] * 2
    # a page id that the pool does not have
    table = fresh()
    table[0, 0] = 99
    plan = cache.plan(table, 8)
    plan.update(to_i32([3]), to_i32([2]), to_i32(np.arange(8)))
    assert cache.status() == (rd.EDEVICE, block.ERR_PAGE)
    assert plan.slots.cpu().tolist() == [-1] * 8
    # nothing to do
    plan.update(to_i32([]), to_i32([]), to_i32([]))
    assert cache.status() == (0, 0) and plan.slots.cpu().tolist() == [-1] * 8


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------
def ref_summary(rows):
    with np.errstate(all="ignore"):
        hi, lo = np.fmax.reduce(rows, 0), np.fmin.reduce(rows, 0)
        hi, lo = np.where(np.isnan(hi), -np.inf, hi), np.where(np.isnan(lo), np.inf, lo)
        a = min(max(np.abs(hi).max(), np.abs(lo).max(), 2.0 ** -100), 2.0 ** 100)
        step = 2.0 ** (math.frexp(a)[1] - 7)
        step = 2 * step if a > 127 * step else step
        return np.clip(np.ceil(hi / step), -127, 127), np.clip(np.floor(lo / step), -127, 127), step


@pytest.mark.parametrize("dim,dtype,rows,page", [
    (64, BF, BF, 16), (128, BF, BF, 64), (256, HF, HF, 32), (64, E4, HF, 256), (128, E4, BF, 16),
    (256, E4, BF, 16)])
@pytest.mark.parametrize("case", ["decode", "prompt", "strided", "plain"])
def test_append(dim, dtype, rows, page, case):
    rng = np.random.default_rng(dim + page)
    kv = 3
    prev = np.array([0, 1, page - 1, page, 2 * page + 5, 37])
    new = np.ones(6, int) if case != "prompt" else np.array([1, 0, 2 * page + 3, 5, page, 70])
    c = Cache(list(prev + new), kv, dim, page, dtype, seed=dim, q_heads=kv,
              summaries=case != "plain")
    slots = np.concatenate([c.table_np[r, p // page] * page + p % page
                            for r in range(6) for p in [np.arange(prev[r], prev[r] + new[r])]])
    # rows to be written, then a padding token
    slots = np.concatenate([slots, [-1]])
    T = len(slots)
    joint = torch.randn((T, 2 * kv + 1, dim + (1 if case == "strided" else 0)), device="cuda")
    joint = (3 * joint).to(rows)
    k, v = joint[:, 1:kv + 1, :dim], joint[:, kv + 1:, :dim]
    old_k, old_v = c.k.float(), c.v.float()
    c.cache.append(k, v, to_i32(slots))
    assert c.cache.status() == (0, 0)
    for got, old, x, s in ((c.k, old_k, k, c.scales[0]), (c.v, old_v, v, c.scales[1])):
        want = old.clone()
        x = x.float()
        if s is not None:
            x = (x / s[:, None]).clamp(-448, 448)
        live = torch.from_numpy(slots[:-1]).cuda()
        want[live // page, :, live % page] = x[:-1].to(dtype).float()
        assert torch.equal(torch.nan_to_num(got.float(), nan=7e4),
                           torch.nan_to_num(want, nan=7e4))
    if case == "plain":
        return
    touched = set()
    keys = f64(c.k.float())
    for r in range(6):
        if new[r] == 0:
            continue
        for p in range(prev[r] // page, (prev[r] + new[r] - 1) // page + 1):
            page_id = int(c.table_np[r, p])
            touched.add(page_id)
            filled = min(page, prev[r] + new[r] - p * page)
            for h in range(kv):
                hi, lo, step = ref_summary(keys[page_id, h, :filled])
                assert float(c.steps[page_id, h]) == step
                assert np.array_equal(c.codes[page_id, h].cpu().numpy(), np.stack([hi, lo]))
    others = [i for i in range(c.k.shape[0]) if i not in touched]
    assert not c.codes[others].any() and not c.steps[others].any()


@pytest.mark.parametrize("dtype", [BF, E4])
def test_append_extreme_values(dtype):
    """Zeros, infinities and NaN in new rows."""
    c = Cache([16], 1, 64, 16, dtype, q_heads=1)
    k = torch.zeros((16, 1, 64), dtype=BF, device="cuda")
    k[3, 0, 5], k[4, 0, 6], k[5, 0, 7], k[:, 0, 8] = math.inf, -math.inf, math.nan, 1e-38
    slots = to_i32(c.table_np[0, 0] * 16 + np.arange(16))
    c.cache.append(k, k, slots)
    got = c.k[int(c.table_np[0, 0]), 0].float()
    if dtype == E4:
        assert float(got[3, 5]) == 448 and float(got[4, 6]) == -448 and math.isnan(got[5, 7])
    else:
        assert torch.equal(torch.nan_to_num(got, nan=3.), torch.nan_to_num(k[:, 0].float(), nan=3.))
    hi, lo, step = ref_summary(f64(got))
    at = int(c.table_np[0, 0])
    assert float(c.steps[at, 0]) == step
    assert np.array_equal(c.codes[at, 0].cpu().numpy(), np.stack([hi, lo]))
    c.cache.append(torch.zeros_like(k), torch.zeros_like(k), slots)
    assert not c.codes[at].any() and float(c.steps[at, 0]) == 2.0 ** -106


@pytest.mark.parametrize("rows", [BF, HF])
def test_append_quotients_are_the_divisions(rows):
    """Every bit pattern of the rows' type, over scales of every size: what is
    stored is the rounded, saturated quotient."""
    patterns = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(rows)
    x = patterns.reshape(1024, 1, 64)
    k = torch.zeros((64, 1, 16, 64), dtype=E4, device="cuda")
    v = torch.zeros_like(k)
    slots = torch.arange(1024, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(5)
    scales = [1.0, 0.0173, 3.0, 2.0 ** -100, 2.0 ** 100, 2.0 ** -101, 2.0 ** 101, 1e-38, 2e-45, 3e38]
    scales += [float(10 ** (8 * torch.rand((), generator=g) - 4)) for _ in range(20)]
    for scale in scales:
        ks = torch.tensor([scale], device="cuda")
        vs = torch.tensor([scale * 1.5 if scale < 2e38 else scale], device="cuda")
        cache = block.PagedCache(k, v, 1, max_requests=1, k_scale=ks, v_scale=vs)
        cache.append(x, x, slots)
        for got, s in ((k, ks), (v, vs)):
            want = (x.float() / s).clamp(-448, 448).to(E4).float().reshape(-1)
            have = got.float().reshape(-1)
            assert torch.equal(torch.isnan(have), torch.isnan(want)), scale
            assert torch.equal(torch.nan_to_num(have), torch.nan_to_num(want)), scale
        cache.close()


def test_append_bad_slots():
    c = Cache([16], 1, 64, 16, BF, q_heads=1)
    before = c.k.clone()
    row = torch.ones((3, 1, 64), dtype=BF, device="cuda")
    c.cache.append(row, row, to_i32([-2, c.k.shape[0] * 16, -1]))
    assert c.cache.status() == (rd.EDEVICE, block.ERR_PAGE)
    assert torch.equal(torch.nan_to_num(before), torch.nan_to_num(c.k))
    c.cache.append(row[:0], row[:0], to_i32([]))
    assert c.cache.status() == (0, 0)


# --------------------------------------------------------------------------
# selection
# --------------------------------------------------------------------------
def ref_select(c, q, keep, first, last):
    R, heads, dim = q.shape
    kv = c.k.shape[1]
    G = heads // kv
    codes, steps = c.codes.cpu().numpy().astype(np.int64), f64(c.steps)
    pages = np.full((R, kv, keep), -1, np.int32)
    for r, n in enumerate(c.lens):
        held = -(-n // c.page)
        for h in range(kv):
            x = np.nan_to_num(f64(q[r, h * G:h * G + G]), nan=0.0)
            a = min(max(np.abs(x).max(), 2.0 ** -100), 2.0 ** 100)
            f = np.clip(np.rint(x * 2.0 ** (14 - math.frexp(a)[1])), -16384, 16384)
            P, N = np.maximum(f, 0).sum(0), np.maximum(-f, 0).sum(0)
            t = math.frexp(max(P.max(), N.max(), 1.0))[1] - 1
            P, N = (np.minimum(np.rint(z * 2.0 ** (6 - t)), 127).astype(np.int64) for z in (P, N))
            ids = c.table_np[r, :held]
            ok = (ids >= 0) & (ids < c.k.shape[0])
            at = np.where(ok, ids, 0)
            s = (codes[at, h, 0] @ P - codes[at, h, 1] @ N) * steps[at, h]
            s = np.where(ok, s, -np.inf)
            s[:first] = np.inf
            s[max(0, held - last):] = np.inf
            best = np.sort(np.lexsort((np.arange(held), -s))[:keep])
            pages[r, h, :len(best)] = best
    return pages


@pytest.mark.parametrize("dim,group,dtype,qt,page", [
    (64, 8, HF, HF, 16), (128, 1, BF, BF, 16), (128, 16, E4, BF, 32), (256, 4, BF, BF, 16)])
@pytest.mark.parametrize("keep,first,last", [(2, 1, 1), (7, 1, 1), (8, 0, 0), (5, 2, 3), (1, 0, 1)])
def test_select(dim, group, dtype, qt, page, keep, first, last):
    lens = [0, 1, page, 5 * page, 8 * page + 1, 40 * page - 3, 100 * page, 2100 if page < 32 else 900]
    c = Cache(lens, 2, dim, page, dtype, seed=dim, q_heads=2 * group)
    c.summarise()
    q = queries(len(lens), 2 * group, dim, qt, seed=4)
    pages = torch.full((len(lens), 2, keep), -5, dtype=torch.int32, device="cuda")
    c.cache.select(q, c.table, c.lens_t, pages, first=first, last=last)
    assert c.cache.status() == (0, 0)
    want = ref_select(c, q, keep, first, last)
    assert np.array_equal(pages.cpu().numpy(), want)
    out = torch.empty_like(q)
    c.cache.attend(q, c.table, c.lens_t, out, pages=pages)
    check_attend(c, q, out, pages=want)


@pytest.mark.parametrize("R,kv,held,keep", [(1, 1, 20000, 300), (1, 4, 5000, 4999), (40, 2, 1500, 64)])
def test_select_long(R, kv, held, keep):
    """Whole clusters, shares that end inside a batch, summaries with ties."""
    page, dim = 16, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    kc = torch.zeros((held, kv, page, dim), dtype=BF, device="cuda")
    codes = torch.randint(-3, 4, (held, kv, 2, dim), generator=g, device="cuda").to(torch.int8)
    codes[::3] = codes[0]                                          # many equal scores
    steps = 2.0 ** torch.randint(-1, 1, (held, kv), generator=g, device="cuda").float()
    cache = block.PagedCache(kc, kc.clone(), kv * 2, max_requests=R, codes=codes, steps=steps)
    table = torch.stack([torch.randperm(held, generator=g, device="cuda") for _ in range(R)])
    table = table.to(torch.int32)
    lens = torch.full((R,), held * page - 3, dtype=torch.int32, device="cuda")
    lens[R // 2] = (held - 700) * page
    q = queries(R, kv * 2, dim, BF)
    pages = torch.empty((R, kv, keep), dtype=torch.int32, device="cuda")
    cache.select(q, table, lens, pages)

    class C:
        pass

    c = C()
    c.k, c.codes, c.steps, c.page = kc, codes, steps, page
    c.lens, c.table_np = lens.tolist(), table.cpu().numpy()
    assert np.array_equal(pages.cpu().numpy(), ref_select(c, q, keep, 1, 1))
    assert cache.status() == (0, 0)


def test_select_extreme_queries_and_bad_pages():
    """All-zero, huge, infinite and NaN queries; a page outside the pool."""
    c = Cache([800] * 5, 1, 64, 16, BF, q_heads=2)
    c.summarise()
    q = queries(5, 2, 64, BF)
    q[0] = 0
    q[1] *= 2.0 ** 110
    q[2, 0, 3], q[2, 1, 5] = math.inf, -math.inf
    q[3, 0, 4] = math.nan
    c.table_np[4, 7] = -1
    c.table[4, 7] = -1
    pages = torch.empty((5, 1, 9), dtype=torch.int32, device="cuda")
    c.cache.select(q, c.table, c.lens_t, pages)
    assert c.cache.status() == (rd.EDEVICE, block.ERR_PAGE)
    assert np.array_equal(pages.cpu().numpy(), ref_select(c, q, 9, 1, 1))
    assert pages[0, 0].cpu().tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 49]


# --------------------------------------------------------------------------
# residual norm
# --------------------------------------------------------------------------
def ref_norm(h, y, post, gate, scale, pre, eps):
    z = np.zeros_like(h) if y is None else y
    if post is not None:
        z = z / np.sqrt((z ** 2).mean(1, keepdims=True) + eps) * post
    if gate is not None:
        z = z * gate
    z = scale * z
    hh = h + z
    inv = 1 / np.sqrt((hh ** 2).mean(1, keepdims=True) + eps)
    return hh, hh * inv * (1 if pre is None else pre), np.abs(h) + np.abs(z), inv


@pytest.mark.parametrize("rows,hidden", [(1, 8), (3, 264), (16, 2048), (5, 2880), (2, 4104),
                                         (3, 8192), (2, 16384), (2, 16392), (1, 65536), (700, 256)])
@pytest.mark.parametrize("h_t,y_t,x_t,gate,post,pre", [
    (F32, BF, F32, None, False, True), (BF, BF, BF, "full", True, True),
    (HF, F32, HF, "token", True, False), (F32, F32, BF, "channel", False, True),
    (BF, None, F32, None, False, True)])
def test_residual_norm(rows, hidden, h_t, y_t, x_t, gate, post, pre):
    g = torch.Generator(device="cuda").manual_seed(rows + hidden)
    draw = lambda s, t: torch.randn(s, generator=g, device="cuda").to(t)  # noqa: E731
    h = draw((rows, hidden), h_t)
    y = None if y_t is None else draw((rows, hidden), y_t)
    w_t = F32 if h_t == F32 else BF
    pw, qw = (draw((hidden,), w_t) if on else None for on in (post, pre))
    gt = {None: None, "full": (rows, hidden), "token": (rows, 1), "channel": (hidden,)}[gate]
    gt = None if gt is None else draw(gt, BF)
    h_out, x = torch.empty_like(h), torch.empty((rows, hidden), dtype=x_t, device="cuda")
    block.residual_norm(h, x, y=y, post_weight=pw, gate=gt, scale=0.7, pre_weight=qw, eps=1e-5,
                        h_out=h_out)
    n = lambda t: None if t is None else f64(t)  # noqa: E731
    hh, xx, size, inv = ref_norm(f64(h), n(y), n(pw), n(gt), 0.7, n(qw), 1e-5)
    # a few fp32 roundings of each term, sums of up to 65536 squares by lanes
    # and warps (relative error below 2^-18), then the output's own rounding
    err_h = 2.0 ** -18 * size
    assert np.all(np.abs(f64(h_out) - hh) <= err_h + HALF_ULP[h_t] * np.abs(hh) + 2.0 ** -24)
    w = 1 if pre is False else np.abs(f64(qw))
    assert np.all(np.abs(f64(x) - xx) <= 2 * err_h * inv * w + 2.0 ** -17 * np.abs(xx) +
                  HALF_ULP[x_t] * np.abs(xx) + 2.0 ** -24)
    # in place, without x, without h_out: the same values
    h2 = h.clone()
    block.residual_norm(h2, y=y, post_weight=pw, gate=gt, scale=0.7, h_out=h2)
    h3, x3 = torch.empty_like(h), torch.empty_like(x)
    block.residual_norm(h, y=y, post_weight=pw, gate=gt, scale=0.7, h_out=h3)
    assert torch.equal(h2, h3)
    block.residual_norm(h, x3, y=y, post_weight=pw, gate=gt, scale=0.7, pre_weight=qw, eps=1e-5)
    assert torch.equal(x3, x)


def test_residual_norm_strides_and_zero_rows():
    wide = torch.randn(6, 1000, device="cuda")
    h, y = wide[:, 8:264], wide[:, 400:656]
    out = torch.zeros(6, 512, device="cuda")
    x = out[:, :256]
    h[2] = 0
    y[2] = 0
    block.residual_norm(h, x, y=y)
    hh, xx, _, _ = ref_norm(f64(h), f64(y), None, None, 1.0, None, 1e-6)
    assert np.abs(f64(x) - xx).max() < 1e-4 and bool((x[2] == 0).all())
    assert not out[:, 256:].any()
    block.residual_norm(h[:0], x[:0])


# --------------------------------------------------------------------------
# refusals and the public manner
# --------------------------------------------------------------------------
def test_refusals():
    k = torch.zeros((4, 2, 16, 64), dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    make = lambda **o: block.PagedCache(**dict(dict(k=k, v=v, q_heads=4, max_requests=3), **o))  # noqa: E731
    for over, err in [(dict(q_heads=3), rd.ReaderError), (dict(q_heads=2 * 65), rd.ReaderError),
                      (dict(max_requests=0), rd.ReaderError), (dict(max_requests=1025), rd.ReaderError),
                      (dict(v=k), rd.ReaderError), (dict(v=v.half()), TypeError),
                      (dict(k=k.float()), TypeError), (dict(v=v[:3]), ValueError),
                      (dict(k=k.cpu()), ValueError), (dict(k=k.transpose(2, 3)), ValueError),
                      (dict(k_scale=torch.ones(2, device="cuda")), rd.ReaderError),
                      (dict(steps=torch.ones((4, 2), device="cuda")), rd.ReaderError)]:
        with pytest.raises(err):
            make(**over)
    for shape in [(4, 2, 8, 64), (4, 2, 24, 64), (4, 2, 512, 64), (4, 2, 16, 96)]:
        z = torch.zeros(shape, dtype=BF, device="cuda")
        with pytest.raises(rd.ReaderError) as e:
            make(k=z, v=z.clone())
        assert e.value.code == rd.EINVAL
    c = make()
    table, lens = to_i32(np.zeros((3, 2))), to_i32([1, 2, 3])
    q, out = torch.zeros((3, 4, 64), dtype=BF, device="cuda"), torch.zeros((3, 4, 64), dtype=BF,
                                                                          device="cuda")
    for bad, err in [((q.half(), table, lens, out), TypeError), ((q, table.long(), lens, out), TypeError),
                     ((q, table[:2], lens, out), ValueError), ((q, table, lens[:2], out), ValueError),
                     ((q, table, lens, out[:2]), ValueError), ((q[:, :2], table, lens, out), ValueError),
                     ((q.cpu(), table, lens, out), TypeError), ((q, table, lens, q), rd.ReaderError),
                     (([1], table, lens, out), TypeError)]:
        with pytest.raises(err):
            c.attend(*bad)
    with pytest.raises(rd.ReaderError):
        c.attend(q, table, lens, out, window=-1)
    with pytest.raises(rd.ReaderError):
        c.attend(q, table, lens, out, pages=to_i32(np.zeros((3, 2, 0))))
    with pytest.raises(rd.ReaderError):          # no summaries
        c.select(q, table, lens, to_i32(np.zeros((3, 2, 2))))
    row = torch.zeros((2, 2, 64), dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        c.append(row, row.half(), to_i32([1, 2]))
    with pytest.raises(ValueError):
        c.append(row, row, to_i32([1, 2, 3]))
    with pytest.raises(ValueError):
        c.plan(to_i32(np.zeros((4, 2))), 8)
    p = c.plan(table, 8)
    with pytest.raises(ValueError):
        p.update(to_i32([1] * 4), to_i32([1] * 4), to_i32([1]))
    with pytest.raises(rd.ReaderError):
        p.update(p._lens[:2], to_i32([1, 1]), to_i32([1]))
    s = make(codes=torch.zeros((4, 2, 2, 64), dtype=torch.int8, device="cuda"),
             steps=torch.zeros((4, 2), device="cuda"))
    for keep, first, last in [(2, 2, 1), (0, 0, 0), (2, -1, 1)]:
        with pytest.raises(rd.ReaderError):
            s.select(q, table, lens, to_i32(np.zeros((3, 2, keep))), first=first, last=last)
    h = torch.zeros((4, 64), device="cuda")
    for kw, err in [(dict(), rd.ReaderError), (dict(x=h), rd.ReaderError),
                    (dict(x=torch.zeros(4, 32, device="cuda")), ValueError),
                    (dict(x=torch.zeros(4, 64, device="cuda", dtype=torch.float64)), TypeError),
                    (dict(x=h.clone(), gate=torch.ones(64, device="cuda")), rd.ReaderError),
                    (dict(x=h.clone(), y=h.clone(), gate=torch.ones(3, device="cuda")), ValueError),
                    (dict(x=h.clone(), post_weight=torch.ones(64, device="cuda")), rd.ReaderError),
                    (dict(h_out=h.bfloat16()), TypeError)]:
        with pytest.raises(err):
            block.residual_norm(h, **kw)
    odd = torch.zeros((4, 60), device="cuda")
    with pytest.raises(rd.ReaderError):
        block.residual_norm(odd, odd.clone())
    c.close()
    c.close()


def test_create_reports_a_failed_allocation():
    k = torch.zeros((4, 2, 16, 64), dtype=BF, device="cuda")
    rd.inject_fault(rd.INJECT_ALLOC_FAIL)
    with pytest.raises(rd.ReaderError) as e:
        block.PagedCache(k, k.clone(), 4)
    assert e.value.code == rd.ENOMEM


def test_a_step_in_a_graph():
    """Plan, append, select and attend captured once and replayed on new data."""
    c = Cache([100, 37, 0], 2, 64, 16, BF, seed=8, q_heads=4, spare=9)
    c.summarise()
    used = set(c.table_np[c.table_np >= 0].tolist())
    free = to_i32([i for i in range(c.k.shape[0]) if i not in used])
    plan = c.cache.plan(c.table, 3)
    prev, new = c.lens_t.clone(), to_i32([1, 1, 1])
    k, v = (torch.empty((3, 2, 64), dtype=BF, device="cuda") for _ in range(2))
    q, out = queries(3, 4, 64, BF), torch.empty((3, 4, 64), dtype=BF, device="cuda")
    pages = torch.empty((3, 2, 4), dtype=torch.int32, device="cuda")
    free_now = free.clone()

    def step():
        plan.update(prev, new, free_now)
        c.cache.append(k, v, plan.slots)
        c.cache.select(q, c.table, plan.lens, pages)
        c.cache.attend(q, c.table, plan.lens, out, pages=pages)

    plan.update(prev, new, free_now)     # views of this step's shape exist before capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.table.copy_(to_i32(c.table_np))
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(20):
        k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
        v.copy_(torch.randn(k.shape, generator=g, device="cuda"))
        graph.replay()
        n = int(plan.taken)
        prev.copy_(plan.lens)
        free_now.copy_(torch.roll(free_now, -n))
        c.lens = plan.lens.cpu().tolist()
        c.table_np = c.table.cpu().numpy()
        want = ref_select(c, q, 4, 1, 1)
        assert np.array_equal(pages.cpu().numpy(), want)
        check_attend(c, q, out, pages=want)
    assert c.lens == [120, 57, 20]
    assert c.cache.status() == (0, 0)


# --------------------------------------------------------------------------
# the operators together, as the example runs them
# --------------------------------------------------------------------------
def _example():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decode_block.py")
    spec = importlib.util.spec_from_file_location("decode_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_decoder_steps_match_a_plain_decoder():
    """Forty steps of the example's decoder, one request idling now and then,
    against attention, cache and norms in plain float64 (its matrix products
    and experts are shared: the bf16 projections are taken from the same x)."""
    m = _example()
    dec = m.Decoder(layers=1)
    layer, w, R = dec.layers[0], dec.w, dec.requests
    g = torch.Generator(device="cuda").manual_seed(3)
    keys = [[] for _ in range(R)]
    values = [[] for _ in range(R)]
    H, kv, dim, heads = w.H, layer.kv_heads, layer.head_dim, layer.q_heads

    def norm(h, weight):
        return h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * weight.double()

    for i in range(40):
        h = torch.randn((R, H), generator=g, device="cuda")
        new = torch.ones(R, dtype=torch.int32, device="cuda")
        if i % 5 == 2:
            new[1] = 0
        start = h.double()
        dec.step(h, new)
        x = torch.empty_like(h)
        block.residual_norm(start.float(), x, pre_weight=layer.norm1)
        assert (x.double() - norm(start, layer.norm1)).abs().max() < 1e-5
        qkv = (x.bfloat16() @ layer.qkv).view(R, -1, dim)
        out = torch.zeros((R, heads, dim), dtype=torch.float64, device="cuda")
        for r in range(R):
            if new[r]:
                keys[r].append(qkv[r, heads:heads + kv].double())
                values[r].append(qkv[r, heads + kv:].double())
            k, v = torch.stack(keys[r], 1), torch.stack(values[r], 1)      # [kv][n][dim]
            q = qkv[r, :heads].double().view(kv, heads // kv, dim)
            p = (q @ k.transpose(1, 2) * dim ** -0.5).softmax(-1)
            out[r] = (p @ v).view(heads, dim)
        # bf16 weights and output: two halves of an ulp of values below 8
        assert (dec.attended.double() - out).abs().max() < 2 * 2.0 ** -8 * out.abs().max()
        a = dec.attended.view(R, -1) @ layer.out
        mid = start + dec.scale * a.double()
        assert (dec.x.double() - norm(mid, layer.norm2)).abs().max() < 1e-4
        assert (h.double() - (mid + dec.scale * dec.y.double())).abs().max() < 1e-4
    assert dec.lens.tolist() == [40, 32, 40, 40]
    dec.status()


def test_decoder_with_every_page_kept_attends_like_dense():
    """One layer on the same inputs, over all pages and over a list of them all:
    each attention output is within 2^-8 of its weights and 2^-8 of itself."""
    m = _example()
    a, b = m.Decoder(layers=1), m.Decoder(layers=1)
    g = torch.Generator(device="cuda").manual_seed(4)
    new = torch.ones(a.requests, dtype=torch.int32, device="cuda")
    for _ in range(50):
        h = torch.randn((a.requests, a.w.H), generator=g, device="cuda")
        a.step(h.clone(), new)
        b.step(h.clone(), new, keep=a.table.shape[1])
        assert torch.equal(a.layers[0].v, b.layers[0].v)
        gap = (a.attended.float() - b.attended.float()).abs().max()
        assert gap <= 4 * 2.0 ** -8 * a.layers[0].v.abs().max()
    a.status()
    b.status()
    m.main(steps=40, keep=2)
