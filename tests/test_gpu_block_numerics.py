"""Numerical edges of the decode-step operators: what the weights of attention
keep, infinities and NaN among the rows that are read, and the range of the
page summaries.  References are in 64 bits; tolerances follow from the
arithmetic, as each test says (u: half an ulp of a type, d: the bound
(D + 16) 2^-24 scale sum |q k| of a logit's error in fp32)."""

import math
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import test_gpu_block as T  # noqa: E402

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from calibration_free_sparse_gb300 import block
    from calibration_free_sparse_gb300 import reader as rd

BF, HF, F32, E4 = T.BF, T.HF, T.F32, T.E4
U = T.HALF_ULP


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def given_cache(k, v, dtype, page=16, q_heads=None, scale=1.0):
    """A Cache of requests [R][n][kv][dim] float64 whose rows are given (all of
    one length, exact in the cache's type); 8-bit caches have one scale."""
    R, n, kv, dim = k.shape
    c = T.Cache([n] * R, kv, dim, page, dtype, q_heads=q_heads, summaries=False)
    if dtype == E4:
        c.k_scale.fill_(scale), c.v_scale.fill_(scale)
        c.scales[0].fill_(scale), c.scales[1].fill_(scale)
    pos = np.arange(n)
    for r in range(R):
        ids = torch.from_numpy(c.table_np[r, pos // page]).long().cuda()
        off = torch.from_numpy(pos % page).long().cuda()
        for cache, rows in ((c.k, k[r]), (c.v, v[r])):
            x = torch.from_numpy(rows / (scale if dtype == E4 else 1.0)).to(dtype).cuda()
            if dtype == E4:
                cache.view(torch.uint8)[ids, :, off] = x.view(torch.uint8)
            else:
                cache[ids, :, off] = x
    return c


def exact(c, q, r, h, scale):
    """(out [G][dim], lse [G], A, d, n) of a request and KV head in 64 bits; A is
    the weighted mean of |v| over the finite v, d the bound of a logit's error."""
    G, dim = q.shape[1] // c.k.shape[1], q.shape[2]
    mine = slice(h * G, h * G + G)
    k, v = c.rows(r, h, np.arange(c.lens[r]))
    x = T.f64(q[r, mine])
    with np.errstate(all="ignore"):
        s = scale * x @ k.T
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        den = p.sum(1, keepdims=True)
        out = np.where(np.isinf(v).any(0), (p[:, :, None] * v).sum(1), p @ np.where(np.isinf(v), 0, v))
        A = p @ np.abs(np.where(np.isfinite(v), v, 0)) / den
        d = ((dim + 16) * 2.0 ** -24 * scale * (np.abs(x) @ np.abs(k).T)).max(1, keepdims=True)
        return out / den, (np.log(den) + top)[:, 0], A, d, len(v)


def attended(c, q, scale=None, **kw):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    c.cache.attend(q, c.table, c.lens_t, out, lse=lse, scale=scale, **kw)
    assert c.cache.status() == (0, 0)
    return T.f64(out), T.f64(lse)


# --------------------------------------------------------------------------
# the weights of attention
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype,qt", [(BF, BF), (HF, HF), (E4, HF), (E4, BF)])
def test_attend_weights_keep_their_bits(dim, dtype, qt):
    """Two keys whose weights nearly cancel: out = tanh(delta / 2), far below
    the weights, so what their rounding loses stands out.  A weight may be off
    by the fp32 forms of its logit and exponential and by 2^-20 of itself, the
    output by its own rounding.  (Weights of 8 or 11 bits would be off by 2^-9
    or 2^-12: an output by half that.)"""
    g = torch.Generator().manual_seed(dim)
    R, G = 40, 8
    k, v = np.zeros((R, 2, 1, dim)), np.ones((R, 2, 1, dim))
    k[:, 0, :, 0], v[:, 1] = 1, -1
    c = given_cache(k, v, dtype, q_heads=G)
    q = torch.zeros((R, G, dim))
    q[:, :, 0] = 2.0 ** -(6 + 3 * torch.rand((R, G), generator=g)) * \
        torch.sign(torch.randn((R, G), generator=g))
    q = q.to(qt).cuda()
    out, _ = attended(c, q, 1.0)
    for r in range(R):
        ref, _, A, d, _ = exact(c, q, r, 0, 1.0)
        tol = (2.0 ** -19 + 2 * d) * A + U[qt] * np.abs(ref)
        assert np.all(np.abs(out[r] - ref) <= tol), r


@pytest.mark.parametrize("dim,dtype,qt", [(64, HF, HF), (128, HF, HF), (256, HF, HF), (128, E4, BF),
                                          (64, E4, HF), (128, BF, BF)])
@pytest.mark.parametrize("R,kv,n", [(64, 8, 200), (1, 1, 700), (1, 2, 9000), (25, 8, 1500)])
def test_attend_small_weights_beside_a_dominant_key(dim, dtype, qt, R, kv, n):
    """One key, the first, takes nearly all the weight and its value is zero;
    the others weigh 2^-24 to 2^-30 of it each and make the output.  Weights
    in fp16 keep 2^-35 of the largest: n 2^-35 max |v| is what they may lose."""
    g = torch.Generator().manual_seed(dim + n)
    k, v = np.zeros((R, n, kv, dim)), np.zeros((R, n, kv, dim))
    k[:, 0, :, 0] = 3
    v[:, 1:] = (2.0 ** 10 * (1 + torch.randint(0, 8, (R, n - 1, kv, dim), generator=g))).numpy()
    c = given_cache(k, v, dtype, q_heads=4 * kv, scale=64.0 if dtype == E4 else 1.0)
    q = torch.zeros((R, 4 * kv, dim))
    q[:, :, 0] = torch.tensor([5.5, 6.0, 6.5, 7.0]).repeat(kv)
    q = q.to(qt).cuda()
    out, _ = attended(c, q, 1.0)
    for r in range(R):
        for h in range(kv):
            ref, _, A, d, m = exact(c, q, r, h, 1.0)
            tol = (2.0 ** -19 + 2 * d) * A + U[qt] * np.abs(ref)
            if dtype != BF:
                tol = tol + m * 2.0 ** -35 * 2.0 ** 13
            assert np.all(np.abs(out[r, 4 * h:4 * h + 4] - ref) <= tol), (r, h)


# --------------------------------------------------------------------------
# infinities and NaN in rows that are read
# --------------------------------------------------------------------------
DEALT = [([40, 1, 33], 2), ([5000], 1), ([3, 700], 1), ([200] * 64, 8),
         ([2700 - 40 * i for i in range(20)], 8), ([3000] + [5] * 40, 8)]


def infinite_values(c, rows):
    """An infinity in some coordinates of the last and of a middle key."""
    for r in rows:
        n = c.lens[r]
        for pos, coord, value in ((n - 1, 3, math.inf), (n // 2, 5, -math.inf), (n - 1, 7, math.inf),
                                  (0, 7, -math.inf), (n // 3, 9, math.inf)):
            c.v[c.table_np[r, pos // c.page], :, pos % c.page, coord] = value


@pytest.mark.parametrize("lens,kv", DEALT)
@pytest.mark.parametrize("dim,dtype,group", [(64, HF, 4), (128, BF, 16), (128, HF, 12), (256, BF, 3)])
def test_attend_infinite_values(lens, kv, dim, dtype, group):
    """A value of infinity makes its coordinate infinite, whatever its key's
    weight; infinities of both signs make it NaN; the others stay finite."""
    c = T.Cache(lens, kv, dim, 32, dtype, seed=11, q_heads=group * kv, summaries=False)
    rows = range(0, len(lens), max(1, len(lens) // 3))
    infinite_values(c, rows)
    # in the first request one of them belongs to a key of nearly no weight
    c.k[c.table_np[0, (lens[0] // 3) // 32], :, (lens[0] // 3) % 32] *= 4
    q = T.queries(len(lens), group * kv, dim, dtype)
    out, _ = attended(c, q)
    for r in rows:
        for h in range(kv):
            ref, _, A, d, m = exact(c, q, r, h, dim ** -0.5)
            got = out[r, h * group:h * group + group]
            assert np.array_equal(np.isnan(got), np.isnan(ref)), (r, h)
            assert np.array_equal(np.where(np.isinf(got), got, 0), np.where(np.isinf(ref), ref, 0))
            fine = np.isfinite(ref)
            tol = (2.0 ** -16 + 2 * d) * A + U[dtype] * np.abs(np.where(fine, ref, 0)) + \
                m * 2.0 ** -34 * 8 + 2.0 ** -25
            assert np.all(np.abs(np.where(fine, got, 0) - np.where(fine, ref, 0)) <= tol), (r, h)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_attend_infinite_value_of_a_key_without_weight(dtype):
    """A key whose logit lies 40 below the largest still has a weight: its
    value of infinity counts.  One whose logit is -infinity has none."""
    k, v = np.zeros((2, 40, 1, 64)), np.ones((2, 40, 1, 64))
    k[:, 7, :, 0] = -4
    v[:, 7, :, 2] = math.inf
    k[1, 7, :, 0] = -math.inf
    c = given_cache(k, v, dtype, q_heads=2)
    q = torch.zeros((2, 2, 64))
    q[:, :, 0] = 10
    out, _ = attended(c, q.to(dtype).cuda(), 1.0)
    want = np.ones((2, 2, 64))
    want[0, :, 2], want[1, :, 2] = math.inf, math.nan
    assert np.array_equal(out, want, equal_nan=True)


@pytest.mark.parametrize("lens,kv", DEALT + [([513] * 30, 8), ([65] * 160, 2)])
@pytest.mark.parametrize("dim,dtype,group", [(64, HF, 4), (128, BF, 16), (128, E4, 5), (256, BF, 3)])
@pytest.mark.parametrize("sinks", [False, True])
def test_attend_nan_logits(lens, kv, dim, dtype, group, sinks):
    """A key of NaN makes its KV head's outputs and lse NaN wherever it stands
    (alone in the last tile, in the first, in the middle); a query of NaN its own head's."""
    c = T.Cache(lens, kv, dim, 32, dtype, seed=12, q_heads=group * kv, summaries=False)
    qt = BF if dtype == E4 else dtype
    q = T.queries(len(lens), group * kv, dim, qt)
    rows = list(range(0, len(lens), max(1, len(lens) // 5)))
    bad = np.zeros((len(lens), group * kv), bool)
    for i, r in enumerate(rows):
        h, pos = i % kv, (c.lens[r] - 1, 0, c.lens[r] // 2)[i % 3]
        at = c.table_np[r, pos // 32], h, pos % 32
        if dtype == E4:
            c.k.view(torch.uint8)[at] = 0x7f
        else:
            c.k[at] = math.nan
        bad[r, h * group:h * group + group] = True
        q[r, (i + 1) % kv * group, 4] = math.nan
        bad[r, (i + 1) % kv * group] = True
    sk = torch.linspace(-2, 2, group * kv).cuda() if sinks else None
    out, lse = attended(c, q, sinks=sk)
    assert np.array_equal(np.isnan(out), np.broadcast_to(bad[:, :, None], out.shape))
    assert np.array_equal(np.isnan(lse), bad) and np.all(np.isfinite(lse[~bad]))


@pytest.mark.parametrize("lens,kv", DEALT)
def test_attend_nan_values_stay_in_their_coordinate(lens, kv):
    """NaN in a value: that coordinate only, also where the key's weight is
    far below those of the other warps and CTAs."""
    c = T.Cache(lens, kv, 128, 32, BF, seed=13, q_heads=4 * kv, summaries=False)
    for r in range(len(lens)):
        pos = lens[r] - 1
        c.v[c.table_np[r, pos // 32], :, pos % 32, 6] = math.nan
        c.k[c.table_np[r, 0], :, 0] *= 8
    q = T.queries(len(lens), 4 * kv, 128, BF)
    out, lse = attended(c, q)
    want = np.zeros(out.shape, bool)
    want[:, :, 6] = True
    assert np.array_equal(np.isnan(out), want) and np.all(np.isfinite(lse))


@pytest.mark.parametrize("qt", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_small_queries_beside_a_large_one(dim, qt):
    """8-bit cache: coordinates 2^-20 to 2^-26 below the query's largest keep
    all their bits (the largest one meets keys of zero)."""
    g = torch.Generator().manual_seed(dim)
    R, G, n = 6, 8, 40
    k = torch.randint(-14, 15, (R, n, 1, dim), generator=g).double().numpy()
    v = torch.randint(-14, 15, (R, n, 1, dim), generator=g).double().numpy()
    k[:, :, :, 0] = 0
    c = given_cache(k, v, E4, q_heads=G)
    q = 2.0 ** -20 * torch.randn((R, G, dim), generator=g)
    q[:, 1::2] *= 2.0 ** (-6 if qt == BF else 4)
    q[:, :, 0] = 1.7
    q = q.to(qt).cuda()
    for scale, heads in ((2.0 ** 14, slice(0, G, 2)), (2.0 ** (20 if qt == BF else 10), slice(1, G, 2))):
        out, lse = attended(c, q, scale)
        for r in range(R):
            ref, want, A, d, _ = exact(c, q, r, 0, scale)
            tol = (2.0 ** -18 + 2 * d) * A + U[qt] * np.abs(ref)
            assert np.all(np.abs(out[r] - ref)[heads] <= tol[heads]), r
            assert np.all(np.abs(lse[r] - want)[heads] <= (2 * d[:, 0] + 2.0 ** -19 * (1 + np.abs(want)))[heads])


# --------------------------------------------------------------------------
# page selection
# --------------------------------------------------------------------------
def ranked(score, keep, first, last):
    """Pages in the order of the definition: forced, by score, NaN last, ties to
    the lower page; the first `keep` of them, ascending."""
    n = len(score)
    forced = (np.arange(n) < first) | (np.arange(n) >= n - last)
    order = np.lexsort((np.arange(n), np.where(np.isnan(score), 0, -score), np.isnan(score), ~forced))
    best = np.sort(order[:keep])
    return np.concatenate([best, np.full(keep - len(best), -1)]).astype(np.int32)


def query_codes(x):
    """P and N of a group's queries [G][dim], as the header defines them."""
    f = np.rint(x * 2.0 ** (14 - math.frexp(np.abs(x).max())[1]))
    P, N = np.maximum(f, 0).sum(0), np.maximum(-f, 0).sum(0)
    t = math.frexp(max(P.max(), N.max(), 1.0))[1] - 1
    return [np.minimum(np.rint(z * 2.0 ** (6 - t)), 127) for z in (P, N)]


@pytest.mark.parametrize("lens,page", [([640, 900], 16), ([60000], 16), ([300, 40, 20000], 32)])
@pytest.mark.parametrize("first,last", [(1, 1), (0, 0)])
def test_select_steps_that_are_not_finite(lens, page, first, last):
    """Steps of NaN rank last and infinite ones as their scores say (zero times
    infinity is NaN), in the first, a middle and the last head: the list holds
    `keep` pages and nothing is written behind it."""
    kv, G, keep = 3, 2, 6
    c = T.Cache(lens, kv, 64, page, BF, seed=21, q_heads=G * kv)
    c.summarise()
    g = torch.Generator().manual_seed(5)
    for h in range(kv):
        at = torch.randperm(c.steps.shape[0], generator=g)[:c.steps.shape[0] // 2].cuda()
        c.steps[at[0::4], h] = math.nan
        c.steps[at[1::4], h] = math.inf
        c.steps[at[2::4], h] = -math.nan
        c.steps[at[3::4], h] = math.inf
        c.codes[at[3::4], h] = 0
    q = T.queries(len(lens), G * kv, 64, BF, seed=6)
    room = torch.full((len(lens) * kv * keep + 400,), -77, dtype=torch.int32, device="cuda")
    pages = room[200:-200].view(len(lens), kv, keep)
    c.cache.select(q, c.table, c.lens_t, pages, first=first, last=last)
    assert c.cache.status() == (0, 0)
    codes, steps = T.f64(c.codes.float()), T.f64(c.steps)
    for r, n in enumerate(lens):
        for h in range(kv):
            P, N = query_codes(T.f64(q[r, G * h:G * h + G]))
            at = c.table_np[r, :-(-n // page)]
            with np.errstate(invalid="ignore"):
                score = (codes[at, h, 0] @ P - codes[at, h, 1] @ N) * steps[at, h]
            want = ranked(score, keep, min(first, len(at)), min(last, len(at)))
            assert np.array_equal(pages[r, h].cpu().numpy(), want), (r, h)
    assert bool((room[:200] == -77).all()) and bool((room[-200:] == -77).all())


def test_select_every_step_unwritten():
    """No score at all: the forced pages and the lowest others."""
    c = T.Cache([640], 2, 64, 16, BF, seed=22, q_heads=2)
    c.steps.fill_(math.nan)
    room = torch.full((2 * 5 + 100,), -77, dtype=torch.int32, device="cuda")
    pages = room[50:-50].view(1, 2, 5)
    c.cache.select(T.queries(1, 2, 64, BF), c.table, c.lens_t, pages)
    assert pages.tolist() == [[[0, 1, 2, 3, 39]] * 2]
    assert bool((room[:50] == -77).all()) and bool((room[-50:] == -77).all())


# --------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------
@pytest.mark.parametrize("keep", [1 << 22, 1 << 23, (1 << 24) + 1])
def test_attend_refuses_a_list_beyond_32_bits(keep):
    """keep * page_size from 2^30 on: the row's keys are counted in 32 bits."""
    c = T.Cache([300], 1, 64, 256, BF, q_heads=2, summaries=False)
    q = T.queries(1, 2, 64, BF)
    out = torch.full_like(q, 7.0)
    pages = torch.full((1, 1, keep), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(rd.ReaderError) as e:
        c.cache.attend(q, c.table, c.lens_t, out, pages=pages)
    assert e.value.code == rd.EINVAL and bool((out == 7).all())


def test_plan_refuses_arrays_that_overlap():
    """An input that is part of an output (not only one that begins with it),
    and outputs that share words; neighbours that only touch are taken."""
    kv = torch.zeros((8, 1, 16, 64), dtype=BF, device="cuda")
    cache = block.PagedCache(kv, kv.clone(), 1, max_requests=4)
    i32 = T.to_i32
    table = i32(np.full((4, 3), -1))
    plan = cache.plan(table, 8)
    two, free = i32([1, 1]), i32(np.arange(8))
    flat = table.view(-1)
    for prev, new, pool in [(plan._lens[1:3], two, free), (plan._starts[1:3], two, free),
                            (plan._starts[2:4], two, free), (two, plan._lens[1:3], free),
                            (two, plan.slots[3:5], free), (plan.positions[6:], two, free),
                            (two, two, plan.requests[2:5]), (two, two, flat[5:7]),
                            (flat[1:3], two, free), (two, two, plan.taken)]:
        before = [t.clone() for t in (table, plan._lens, plan._starts, plan.slots)]
        with pytest.raises(rd.ReaderError) as e:
            plan.update(prev, new, pool)
        assert e.value.code == rd.EINVAL
        for a, b in zip(before, (table, plan._lens, plan._starts, plan.slots)):
            assert torch.equal(a, b)
    shared = torch.zeros(40, dtype=torch.int32, device="cuda")
    call = block._rd._lib().moe_reader_kv_plan
    base = shared.data_ptr()
    for at in ([0, 2, 5, 13, 20, 28], [0, 1, 5, 13, 21, 29], [0, 2, 5, 13, 21, 28], [6, 0, 3, 11, 19, 27]):
        out = [base + 4 * i for i in at]       # lens 2, starts 3, slots, positions, requests 8 each, taken 1
        args = block._PLAN.pack(two.data_ptr(), two.data_ptr(), table.data_ptr(), free.data_ptr(),
                                *out, 2, 3, 8, 8)
        assert call(cache._h, args, None) == rd.EINVAL
    # lens behind the lengths that it is made of, everything else side by side
    lens = i32([3, 4, 0, 0])
    out = [lens.data_ptr() + 8] + [base + 4 * i for i in (2, 5, 13, 21, 29)]
    args = block._PLAN.pack(lens.data_ptr(), two.data_ptr(), table.data_ptr(), free.data_ptr(), *out,
                            2, 3, 8, 8)
    torch.cuda.synchronize()
    assert call(cache._h, args, torch.cuda.current_stream().cuda_stream) == rd.OK
    torch.cuda.synchronize()
    assert lens.tolist() == [3, 4, 4, 5] and shared.tolist()[2:5] == [0, 1, 2]
    cache.status()


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------
def written(c, positions, seed, rows=BF, skip=0.3, other=None):
    """Appends rows at `positions` (a list per request, ascending) with skipped
    tokens strewn between, or (skip 0) in the place of each position left out,
    and slots outside the pool, if `other` is given; checks every row and every
    touched page's summary."""
    rng = np.random.default_rng(seed)
    kv, page, dim = c.k.shape[1:]
    slots = []
    for r, pos in enumerate(positions):
        for i, p in enumerate(pos):
            slots += [-1] * (int(rng.geometric(1 - skip) - 1) if skip else p - pos[max(i - 1, 0)] - 1)
            if other is not None and rng.random() < 0.1:
                slots.append(other)
            slots.append(int(c.table_np[r, p // page]) * page + p % page)
        slots += [-1] * int(rng.integers(0, 3))
    slots = np.array(slots)
    for page_id in np.unique(slots[slots >= 0] // page):       # the contract
        at = np.flatnonzero((slots // page == page_id) & (slots >= 0))
        assert at[-1] - at[0] <= page or page_id * page >= c.k.shape[0] * page
    x = torch.from_numpy(3 * rng.standard_normal((2, len(slots), kv, dim))).to(rows).cuda()
    want = [c.k.float(), c.v.float()]
    c.cache.append(x[0], x[1], T.to_i32(slots))
    status = c.cache.status()
    live = (slots >= 0) & (slots < c.k.shape[0] * page)
    assert status == ((0, 0) if (live | (slots == -1)).all() else (rd.EDEVICE, block.ERR_PAGE))
    at = torch.from_numpy(slots[live]).cuda()
    for w, got, y, s in zip(want, (c.k, c.v), x, c.scales):
        y = y.float() if s is None else (y.float() / s[:, None]).clamp(-448, 448)
        w[at // page, :, at % page] = y[torch.from_numpy(live).cuda()].to(c.k.dtype).float()
        assert torch.equal(torch.nan_to_num(got.float(), nan=7e4), torch.nan_to_num(w, nan=7e4))
    if c.codes is None:
        return
    keys, codes, steps = T.f64(c.k.float()), c.codes.cpu().numpy(), T.f64(c.steps)
    for page_id in np.unique(slots[live] // page):
        top = (slots[live] % page)[slots[live] // page == page_id].max()
        for h in range(kv):
            hi, lo, step = T.ref_summary(keys[page_id, h, :top + 1])
            assert steps[page_id, h] == step, (page_id, h)
            assert np.array_equal(codes[page_id, h], np.stack([hi, lo])), (page_id, h)


@pytest.mark.parametrize("dim,dtype,rows,page", [(64, BF, BF, 16), (128, E4, BF, 16), (256, HF, HF, 32),
                                                 (64, E4, HF, 64), (128, BF, BF, 256)])
@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("summaries", [True, False])
def test_append_skipped_tokens_inside_a_run(dim, dtype, rows, page, other, summaries):
    """Skipped tokens between tokens of one page, rows that are left out, runs
    across page ends: the summary of a page covers all its new rows."""
    lens = [3 * page] * 5
    half = page // 2
    positions = [[0, 1, 2], [half - 1, half, half + 2, half + 5], list(range(page - 3, page + half - 2)),
                 [page + 1, page + 4, 2 * page - 1, 2 * page, 2 * page + 1], [7]]
    c = T.Cache(lens, 3, dim, page, dtype, seed=31, q_heads=3, summaries=summaries)
    outside = c.k.shape[0] * page + 5 if other else None
    for seed in range(6):
        written(c, positions, seed, rows, skip=0.25, other=outside)


@pytest.mark.parametrize("dtype,page", [(BF, 16), (E4, 64), (BF, 128)])
def test_append_skipped_tokens_in_long_lists(dtype, page):
    """The same where a CTA looks at many tokens: prompts with a few gaps."""
    n = 700
    c = T.Cache([n] * 6, 8, 64, page, dtype, seed=32, q_heads=8, max_requests=6)
    rng = np.random.default_rng(9)
    for seed in range(3):
        positions = []
        for r in range(6):
            keep = np.ones(n, bool)
            keep[rng.integers(0, n, 25)] = False
            positions.append(list(np.flatnonzero(keep)))
        written(c, positions, seed, skip=0)


def summary_of(rows):
    """Codes and step of keys [rows][dim] by the header's definition."""
    number = ~np.isnan(rows)
    seen = number.any(0)
    hi = np.where(seen, np.where(number, rows, -np.inf).max(0), 0)
    lo = np.where(seen, np.where(number, rows, np.inf).min(0), 0)
    a = min(max(np.abs(hi).max(), np.abs(lo).max(), 2.0 ** -100), 2.0 ** 100)
    step = 2.0 ** (math.frexp(a)[1] - 7)
    step = 2 * step if a > 127 * step else step
    return np.clip(np.ceil(hi / step), -127, 127), np.clip(np.floor(lo / step), -127, 127), step


@pytest.mark.parametrize("dtype", [BF, HF, E4])
@pytest.mark.parametrize("gap", [False, True])
def test_append_coordinates_that_are_nan_throughout(dtype, gap):
    """Such a coordinate is passed over: the others keep their step and codes."""
    c = T.Cache([3 * 16] * 3, 2, 64, 16, dtype, seed=33, q_heads=2)
    rows = HF if dtype == HF else BF
    g = torch.Generator().manual_seed(1)
    k = torch.randn((16, 2, 64), generator=g)
    k[:, 0, 5] = k[:, 1, 63] = math.nan
    k[3:9, 0, 7] = math.nan
    k[:, 1, 0:62] = math.nan
    k = k.to(rows).cuda()
    for r, every in enumerate((k, torch.full_like(k, math.nan))):
        slots = c.table_np[r, 1] * 16 + np.arange(16)
        if gap:                        # two runs, the second from the ninth row on
            slots = np.insert(slots, 8, -1)
            every = torch.cat([every[:8], every[:1], every[8:]])
        c.cache.append(every, every, T.to_i32(slots))
        keys = T.f64(c.k[int(c.table_np[r, 1])].float())
        for h in range(2):
            hi, lo, step = summary_of(keys[h])
            assert float(c.steps[c.table_np[r, 1], h]) == step
            assert np.array_equal(c.codes[c.table_np[r, 1], h].cpu().numpy(), np.stack([hi, lo]))
    # no stored value is above 448: no step above 4
    assert float(c.steps[c.table_np[0, 1], 0]) <= 4 and c.cache.status() == (0, 0)


# --------------------------------------------------------------------------
# status
# --------------------------------------------------------------------------
def test_status_waits_for_a_replay_on_another_stream():
    """A step that was captured on one stream and is replayed on a stream that
    does not wait for others: status sees the replay's errors, and clears them."""
    c = T.Cache([40, 30], 1, 64, 16, BF, q_heads=2, summaries=False)
    q = T.queries(2, 2, 64, BF)
    out = torch.empty_like(q)
    lens = c.lens_t.clone()
    c.cache.attend(q, c.table, lens, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.cache.attend(q, c.table, lens, out)
    side = torch.cuda.Stream()
    for bad in (True, False, True):
        lens.copy_(T.to_i32([-1 if bad else 40, 30]))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)             # some 50 ms
            graph.replay()
        assert c.cache.status() == ((rd.EDEVICE, block.ERR_LENGTH) if bad else (0, 0))
    torch.cuda.synchronize()
    assert c.cache.status() == (0, 0)


def test_status_does_not_clear_what_a_later_call_reports():
    """Calls on another stream straight after status, over and over."""
    c = T.Cache([40], 1, 64, 16, BF, q_heads=2, summaries=False)
    q = T.queries(1, 2, 64, BF)
    out, bad = torch.empty_like(q), T.to_i32([-1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(300):
            c.cache.attend(q, c.table, bad, out)
            assert c.cache.status() == (rd.EDEVICE, block.ERR_LENGTH)
    assert c.cache.status() == (0, 0)


@pytest.mark.parametrize("dim,dtype,group", [(64, HF, 4), (128, BF, 16), (128, E4, 5), (256, BF, 3)])
def test_attend_turn_that_does_not_come(dim, dtype, group):
    """Rows cut by equal shares, so that they end inside them: the waits there
    run out, a timeout within a moment and not one per row, and the next call on
    the handle is right and clean."""
    lens = [2700 - 40 * i for i in range(20)]
    c = T.Cache(lens, 8, dim, 64, dtype, seed=41, q_heads=8 * group, summaries=False)
    q = T.queries(len(lens), 8 * group, dim, BF if dtype == E4 else dtype)
    good, out = torch.empty_like(q), torch.empty_like(q)
    c.cache.attend(q, c.table, c.lens_t, good)
    assert c.cache.status() == (0, 0)
    for _ in range(2):
        rd.inject_fault(rd.INJECT_ATTEND_STALL)
        start = time.perf_counter()
        c.cache.attend(q, c.table, c.lens_t, out)
        assert c.cache.status() == (rd.ETIMEOUT, rd.ERR_TIMEOUT)
        assert time.perf_counter() - start < 1.0
        out.fill_(7.0)
        c.cache.attend(q, c.table, c.lens_t, out)
        assert c.cache.status() == (0, 0) and torch.equal(out, good)


# --------------------------------------------------------------------------
# residual norm
# --------------------------------------------------------------------------
def test_residual_norm_between_column_slices_of_one_buffer():
    """Inputs and outputs side by side in the rows of one buffer, also where the
    rows' end touches the next row's beginning; a gate beside them."""
    g = torch.Generator(device="cuda").manual_seed(2)
    rows, H = 37, 264
    wide = torch.randn((rows, 5 * H), generator=g, device="cuda")
    h, y, x, h_out, gate = (wide[:, i * H:(i + 1) * H] for i in (1, 0, 2, 4, 3))
    before = wide.clone()
    pre = torch.randn(H, generator=g, device="cuda")
    want = T.ref_norm(T.f64(h), T.f64(y), None, T.f64(gate), 0.5, T.f64(pre), 1e-6)
    block.residual_norm(h, x, y=y, gate=gate, scale=0.5, pre_weight=pre, h_out=h_out)
    hh, xx, size, inv = want                # as test_residual_norm bounds them, in fp32
    assert np.all(np.abs(T.f64(h_out) - hh) <= 2.0 ** -18 * size + 2.0 ** -24 * (1 + np.abs(hh)))
    assert np.all(np.abs(T.f64(x) - xx) <= 2.0 ** -17 * (size * inv * np.abs(T.f64(pre)) + np.abs(xx)) +
                  2.0 ** -24)
    for i in (0, 1, 3):
        assert torch.equal(wide[:, i * H:(i + 1) * H], before[:, i * H:(i + 1) * H])
    # one value for all rows is no place to write to
    with pytest.raises(rd.ReaderError):
        block.residual_norm(h, torch.empty((1, H), device="cuda").expand(rows, H))
