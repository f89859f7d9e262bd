"""The operators that take a prompt through the block at their limits: many
requests, small coordinates beside large ones, every value of an 8-bit cache,
infinite values, waits that run out, calls at once on two streams, and a decoder
that takes a prompt in chunks, forks it and decodes on."""

import math
import os
import sys
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "tests"))

import test_gpu_prompt as P  # noqa: E402

if torch.cuda.is_available():
    from calibration_free_sparse_gb300 import block, experts
    from calibration_free_sparse_gb300 import reader as rd

BF, HF, E4, I32 = torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int32


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# --------------------------------------------------------------------------
# attention of a chunk
# --------------------------------------------------------------------------
@pytest.mark.parametrize("requests,dim,group,cache,qt", [
    (1024, 64, 2, BF, BF), (700, 128, 4, E4, HF), (333, 256, 1, HF, HF), (1000, 64, 3, E4, BF)])
def test_chunk_many_requests(requests, dim, group, cache, qt):
    """As many requests as a call takes, most with a token or a few, some with
    none, one long."""
    r = np.random.default_rng(requests)
    lens = r.integers(0, 70, requests)
    new = np.minimum(lens, r.choice([0, 1, 1, 2, 5, 40], requests))
    lens[17], new[17] = 900, 300
    c = P.Chunk(lens.tolist(), new.tolist(), 1, group, dim, 16, cache, qt, seed=5)
    out, lse = c.run()
    assert c.cache.status() == (0, 0)
    c.check(out, lse)


@pytest.mark.parametrize("group,dim", [(7, 64), (5, 256), (33, 128), (3, 128)])
@pytest.mark.parametrize("cache,qt", [(BF, BF), (E4, BF)])
def test_chunk_groups_that_do_not_divide_a_tile(group, dim, cache, qt):
    """Row tiles hold whole groups of heads: the rows behind them are nobody's."""
    c = P.Chunk([500, 90], [180, 37], 2, group, dim, 32, cache, qt, seed=group)
    out, lse = c.run()
    c.check(out, lse)
    out, lse = c.run(window=50)
    c.check(out, lse, window=50)


@pytest.mark.parametrize("scale", [-0.09, 0.0, 0.4])
@pytest.mark.parametrize("cache,qt", [(E4, BF), (E4, HF), (HF, HF)])
def test_chunk_queries_read_by_threads(scale, cache, qt):
    """A negative scale, odd addresses and rows that are one row."""
    c = P.Chunk([300, 77], [200, 5], 2, 4, 64, 64, cache, qt)
    out, lse = c.run(scale=scale)
    c.check(out, lse, scale=scale)
    flat = torch.empty(c.T * 8 * 64 + 3, dtype=qt, device="cuda")
    odd = flat[3:].view(8, c.T, 64)
    odd.copy_(c.q.transpose(0, 1))
    c.q = odd.transpose(0, 1)
    again, _ = c.run(scale=scale)
    assert torch.equal(out, again)
    c.q = c.q[3:4].expand(c.T, 8, 64)
    out, lse = c.run(scale=scale)
    c.check(out, lse, scale=scale)


@pytest.mark.parametrize("big", [2.0 ** 20, 2.0 ** -60, 3e38])
def test_chunk_small_coordinates_of_an_e4m3_cache(big):
    """A coordinate that is 2^28 times the others, and meets keys of 0, does not
    take their bits; rows of tiny and of huge queries keep theirs."""
    c = P.Chunk([200], [200], 1, 4, 128, 16, E4, BF, seed=2)
    k = c.k.view(torch.uint8)
    k[..., 9] = 0
    rest = 0.5 * torch.randn((200, 4, 128), generator=torch.Generator().manual_seed(3))
    q = (rest * (big * 2.0 ** -28)).to(BF)
    q[:, :2, 9] = big
    c.q = q.cuda()
    scale = 2.0 ** 28 / big * 128 ** -0.5
    if not math.isfinite(float(np.float32(scale))):
        scale = 1e38
    out, lse = c.run(scale=scale)
    c.check(out, lse, scale=float(np.float32(scale)))


def test_chunk_every_value_of_an_e4m3_cache():
    """Each of the 254 finite values as a key and as a value, one key a row."""
    bits = torch.arange(256, dtype=torch.int32)
    bits = bits[(bits & 127) != 127].to(torch.uint8)
    n = bits.shape[0]
    k = torch.zeros((16, 1, 16, 64), dtype=torch.uint8)
    v = torch.zeros_like(k)
    for i in range(n):
        k[i // 16, 0, i % 16, 0] = bits[i]
        v[i // 16, 0, i % 16, i % 64] = bits[i]
    k, v = (x.cuda().view(E4) for x in (k, v))
    one = torch.ones(1, device="cuda")
    for qt in (BF, HF):
        cache = block.PagedCache(k, v, 1, max_requests=n, k_scale=one, v_scale=one)
        # request i holds token i alone, in the last page it sees
        table = torch.tensor([[i // 16] for i in range(n)], dtype=I32).cuda()
        for i0 in range(16):
            rows = [i for i in range(n) if i % 16 == i0]
            t = table[rows].contiguous()
            R = len(rows)
            q = torch.zeros((R, 1, 64), dtype=qt, device="cuda")
            q[:, 0, 0] = 1
            out, lse = torch.empty_like(q), torch.empty((R, 1), device="cuda")
            cache.attend_chunk(q, t, torch.full((R,), i0 + 1, dtype=I32, device="cuda"),
                               torch.arange(R + 1, dtype=I32, device="cuda"), out, scale=1.0,
                               window=1, lse=lse)
            for j, i in enumerate(rows):
                # one weight: its exponent is rounded to 2^-21 at most below 16,
                # and the power and its logarithm to 2^-22 each
                want = float(k.float()[i // 16, 0, i % 16, 0])
                assert float(lse[j, 0]) == pytest.approx(want, rel=2.0 ** -20, abs=2.0 ** -20)
                # its weight in the product is rounded to fp16, the sum is not
                val = float(v.float()[i // 16, 0, i % 16, i % 64])
                assert float(out[j, 0, i % 64]) == pytest.approx(
                    val, rel=2.0 ** -11 + P.HALF_ULP[qt] + 2.0 ** -20, abs=2.0 ** -24)
        assert cache.status() == (0, 0)


@pytest.mark.parametrize("dim,dtype", [(64, HF), (128, BF), (256, HF)])
def test_chunk_infinite_values_that_are_seen(dim, dtype):
    """A value of infinity that all new rows see makes its coordinate infinite."""
    c = P.Chunk([400], [40], 1, 4, dim, 16, dtype, dtype)
    at = 130
    page, off = int(c.table_np[0, at // 16]), at % 16
    c.v[page, 0, off, 3] = math.inf
    c.v[page, 0, off, 4] = -math.inf
    c.k[page, 0, off] *= 0.1
    out, lse = c.run()
    assert (out[..., 3] == math.inf).all() and (out[..., 4] == -math.inf).all()
    keep = [i for i in range(dim) if i not in (3, 4)]
    assert out[..., keep].isfinite().all() and lse.isfinite().all()


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("sink", [math.inf, -math.inf, 80.0])
def test_chunk_sinks_at_the_ends(split, sink):
    c = P.Chunk([3000] if split else [40] * 30, [3] if split else [40] * 30, 2, 4, 64, 16, BF, BF)
    sinks = torch.full((8,), 0.5, device="cuda")
    sinks[2] = sink
    out, lse = c.run(sinks=sinks)
    if sink == math.inf:
        assert (out[:, 2] == 0).all() and (lse[:, 2] == math.inf).all()
        sinks[2] = 0.5
        plain, plain_lse = c.run(sinks=sinks)
        heads = [h for h in range(8) if h != 2]
        assert torch.equal(out[:, heads], plain[:, heads])
        assert torch.equal(lse[:, heads], plain_lse[:, heads])
    else:
        c.check(out, lse, sinks=sinks)


def test_chunk_rows_that_see_nothing():
    """Pages that are all missing, and rows in front of the first token."""
    c = P.Chunk([40, 64], [40, 3], 1, 4, 64, 16, BF, BF)
    sinks = torch.tensor([0.25, -math.inf, 3.0, 0.0], device="cuda")
    c.table[1] = 10 ** 6
    out, lse = c.run(sinks=sinks)
    assert c.cache.status() == (rd.EDEVICE, block.ERR_PAGE)
    assert (out[40:] == 0).all()
    assert (lse[40:] - sinks).nan_to_num(0).abs().max() <= 2.0 ** -20
    assert (lse[40:, 1] == -math.inf).all()


def test_chunks_of_two_handles_at_once():
    a = P.Chunk([5000, 300], [70, 300], 2, 8, 128, 64, BF, BF, seed=1)
    b = P.Chunk([2500, 800], [33, 800], 2, 4, 64, 16, E4, HF, seed=2)
    want = a.run()[0], b.run()[0]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, o in zip((a, b), streams, outs):
            c.cache.attend_chunk(c.q, c.table, c.lens_t, c.starts, o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


# --------------------------------------------------------------------------
# waits that run out
# --------------------------------------------------------------------------
@pytest.mark.parametrize("cache,qt,dim", [(BF, BF, 128), (E4, BF, 128), (HF, HF, 256), (E4, HF, 64)])
def test_chunk_wait_that_runs_out(cache, qt, dim):
    """A timeout after a second, and the next call on the handle is right."""
    c = P.Chunk([3000, 65], [33, 65], 2, 4, dim, 64, cache, qt)
    good, _ = c.run()
    for _ in range(2):
        rd.inject_fault(rd.INJECT_PROMPT_STALL)
        start = time.perf_counter()
        c.run()
        assert c.cache.status() == (rd.ETIMEOUT, rd.ERR_TIMEOUT)
        assert time.perf_counter() - start < 3.0
        out, _ = c.run()
        assert c.cache.status() == (0, 0) and torch.equal(out, good)


def test_experts_wait_that_runs_out():
    T, E, H, I = 200, 4, 256, 128
    weights = P.layer(E, H, I, BF)
    ids, w = P.routing(T, E, 2, 3)
    x = torch.randn((T, H), device="cuda").to(BF)
    plan = experts.ExpertPlan(E, 2, T, hidden=H).update(ids)
    ex = experts.Experts(*weights)
    act, y = torch.empty((T * 2, I), dtype=BF, device="cuda"), torch.empty((T, H), device="cuda")
    ex.activate(x, plan, act)
    ex.combine(act, plan, w, y)
    good, good_y = act.clone(), y.clone()
    for call in (lambda: ex.activate(x, plan, act), lambda: ex.combine(good, plan, w, y)):
        rd.inject_fault(rd.INJECT_PROMPT_STALL)
        start = time.perf_counter()
        call()
        assert ex.status() == (rd.ETIMEOUT, rd.ERR_TIMEOUT)
        assert time.perf_counter() - start < 3.0
        call()
        assert ex.status() == (0, 0)
    assert torch.equal(act, good) and torch.equal(y, good_y)


# --------------------------------------------------------------------------
# experts
# --------------------------------------------------------------------------
@pytest.mark.parametrize("T,E,topk", [(1, 1024, 64), (300, 1000, 8), (2500, 6, 6)])
def test_experts_many_and_few(T, E, topk):
    ids, w = P.routing(T, E, topk, T)
    x = torch.randn((T, 64), device="cuda").to(BF)
    P.check_experts(ids, w, x, P.layer(E, 64, 72, BF), topk, BF)


def test_experts_inputs_that_are_one_row():
    ids, w = P.routing(150, 8, 2, 4)
    x = torch.randn((1, 128), device="cuda").to(BF).expand(150, 128)
    P.check_experts(ids, w, x, P.layer(8, 128, 64, BF), 2, BF)


def test_plan_of_many_pairs():
    """More pairs than a run of a warp, ids at an odd address."""
    for T, E, topk in ((20011, 37, 3), (70000, 128, 8), (5, 3, 3)):
        g = torch.Generator(device="cuda").manual_seed(T)
        flat = torch.randint(-1, E + 1, (T * topk + 1,), generator=g, device="cuda", dtype=I32)
        for at in (0, 1):
            ids = flat[at:at + T * topk].view(T, topk)
            P.check_plan(ids, E, experts.ExpertPlan(E, topk, T).update(ids))


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------
def test_example_takes_a_prompt():
    """The example's decoder: a prompt at once and in chunks leave the same
    residual and cache behind; a fork decodes what its parent does."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_block as ex

    def run(chunks):
        d = ex.Decoder(max_requests=4, max_pages=16, seed=3)
        g = torch.Generator(device="cuda").manual_seed(0)
        rows = [torch.randn((n, d.w.H), generator=g, device="cuda") for n in (70, 33)]
        out = [[], []]
        for a, b in chunks:
            part = [r[int(a * len(r)):int(b * len(r))] for r in rows]
            h = torch.cat(part)
            new = P.ints([len(part[0]), len(part[1]), 0, 0])
            h = d.prompt(h, new)
            out[0].append(h[:len(part[0])])
            out[1].append(h[len(part[0]):])
        d.status()
        return d, [torch.cat(o) for o in out]

    one, whole = run([(0, 1)])
    two, parts = run([(0, 0.3), (0.3, 0.31), (0.31, 1)])
    assert one.lens.tolist() == two.lens.tolist() == [70, 33, 0, 0]
    for a, b in zip(whole, parts):
        assert a.isfinite().all()
        # the same sums in another order; a token whose choice of experts is a
        # near tie may take another one, and tokens behind it attend to that
        near = ((a - b).abs().amax(1) <= 2.0 ** -4 * a.abs().max()).float().mean()
        assert near >= 0.8
    one.fork([0, 1], [2, 3])
    one.status()
    assert one.lens.tolist() == [70, 33, 70, 33]
    g = torch.Generator(device="cuda").manual_seed(9)
    near = 0
    for _ in range(20):
        h = torch.randn((2, one.w.H), generator=g, device="cuda").repeat(2, 1)
        h = one.step(h, P.ints([1, 1, 1, 1]))
        assert h.isfinite().all()
        near += bool((h[:2] - h[2:]).abs().max() <= 2.0 ** -4 * h.abs().max())
    assert near >= 15
    one.free_requests([0, 3])
    one.status()
    held = one.table[[1, 2]]
    assert one.lens.tolist() == [0, 53, 90, 0]
    assert int(held[0, :4].max()) < 10 and int(held[1, :6].max()) < 10
    h = torch.randn((4, one.w.H), generator=g, device="cuda")
    assert one.step(h, P.ints([0, 1, 1, 0])).isfinite().all()
    one.status()
