"""A small decoder on the MoE reader: every part of a decode step in its place.

Per layer and step, with h the residual stream of a batch of requests:

    x        = rmsnorm(h)                                  residual_norm
    q, k, v  = x W_qkv                                     torch.matmul
    cache   <- k, v at the step's slots                    PagedCache.append
    a        = attention over the cache, or over the       PagedCache.attend,
               pages that score best for each KV head      PagedCache.select
    h, x     = h + scale * a W_o, rmsnorm(h)               residual_norm
    routing  = top-k softmax of x W_r                      torch
    h       += y = routed experts by the channel reader    MoeReader.decode,
                                                           residual_norm

A prompt, or a chunk of one, goes the same way with many tokens a request:
``PagedCache.attend_chunk`` in place of ``attend``, and its routed experts whole
(``Experts.activate``, ``Experts.combine``).  ``Decoder.fork`` continues a request
in several ways on shared pages, ``Decoder.free_requests`` gives pages back and
moves the others together.

The page plan (``PagePlan.update``) is made once a step for all layers, from
the requests' lengths, on the GPU.  Weights are random: there is no text here,
only the step.  Run it with ``python examples/decode_block.py``.
"""

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from calibration_free_sparse_gb300 import block, experts  # noqa: E402
from calibration_free_sparse_gb300 import synthetic as S  # noqa: E402
from calibration_free_sparse_gb300.reader import MoeReader  # noqa: E402


class Layer:
    """One decoder layer: attention weights, its cache, router and reader."""

    def __init__(self, w, seed, q_heads, kv_heads, head_dim, pages, page_size, max_requests):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def draw(*shape):
            t = torch.randn(shape, generator=g, device="cuda") / shape[0] ** 0.5
            return t.to(torch.bfloat16)

        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.qkv = draw(w.H, (q_heads + 2 * kv_heads) * head_dim)
        self.out = draw(q_heads * head_dim, w.H)
        self.router = draw(w.H, w.E)
        self.norm1 = 1 + 0.1 * torch.randn(w.H, generator=g, device="cuda")
        self.norm2 = 1 + 0.1 * torch.randn(w.H, generator=g, device="cuda")
        shape = (pages, kv_heads, page_size, head_dim)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.codes = torch.zeros((pages, kv_heads, 2, head_dim), dtype=torch.int8, device="cuda")
        self.steps = torch.zeros((pages, kv_heads), device="cuda")
        self.cache = block.PagedCache(self.k, self.v, q_heads, max_requests=max_requests,
                                      codes=self.codes, steps=self.steps)
        weights = S.weights_device(seed, w.E, w.I, w.H, "cuda")
        self.reader = MoeReader(w.H, w.E, w.topk, w.I, *weights, S.signs(seed, w.Hp),
                                screen_coords=w.c, rank=w.r, max_batch=max_requests)
        self.experts = experts.Experts(*weights)


class Decoder:
    """Layers of one shape, with the step's plan and buffers."""

    def __init__(self, workload=S.TINY, layers=2, q_heads=4, kv_heads=2, head_dim=64, page_size=16,
                 max_requests=4, max_pages=16, scale=0.5, seed=0):
        self.w, self.scale, self.requests = workload, scale, max_requests
        pages = max_requests * max_pages
        self.layers = [Layer(workload, seed + i, q_heads, kv_heads, head_dim, pages, page_size,
                             max_requests) for i in range(layers)]
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((max_requests, max_pages), -1, **i32)
        self.free = torch.arange(pages, **i32)
        self.lens = torch.zeros(max_requests, **i32)
        self.plan = self.layers[0].cache.plan(self.table, max_requests)
        self.pool = self.layers[0].cache.pool(max_requests)
        f32 = dict(device="cuda")
        self.x = torch.empty((max_requests, workload.H), **f32)
        self.y = torch.empty((max_requests, workload.H), **f32)
        self.attended = torch.empty((max_requests, q_heads, head_dim), dtype=torch.bfloat16, **f32)

    def step(self, h, new, keep=0):
        """One step: h [requests][H] float32 (updated in place), new int32
        [requests] with 1 for the requests that take part (0: the row idles).
        keep > 0 attends to that many pages per KV head."""
        w, plan = self.w, self.plan
        plan.update(self.lens, new, self.free)
        # the plan lists the new tokens in request order; a row that idles has none
        row = torch.where(plan.requests >= 0, plan.requests, self.requests).long()
        slots = torch.full((self.requests + 1,), -1, dtype=torch.int32, device="cuda")
        slots = slots.scatter_(0, row, plan.slots)[:self.requests]
        pages = None
        for layer in self.layers:
            heads, kv, dim = layer.q_heads, layer.kv_heads, layer.head_dim
            block.residual_norm(h, self.x, pre_weight=layer.norm1)
            qkv = (self.x.to(torch.bfloat16) @ layer.qkv).view(-1, heads + 2 * kv, dim)
            layer.cache.append(qkv[:, heads:heads + kv], qkv[:, heads + kv:], slots)
            q = qkv[:, :heads]
            if keep:
                pages = torch.empty((h.shape[0], kv, keep), dtype=torch.int32, device="cuda")
                layer.cache.select(q, self.table, plan.lens, pages)
            layer.cache.attend(q, self.table, plan.lens, self.attended, pages=pages)
            a = self.attended.view(h.shape[0], -1) @ layer.out
            block.residual_norm(h, self.x, y=a, scale=self.scale, pre_weight=layer.norm2, h_out=h)
            top = torch.topk(self.x.to(torch.bfloat16).float() @ layer.router.float(), w.topk)
            ids, share = top.indices.to(torch.int32), top.values.softmax(-1)
            layer.reader.decode(self.x, ids.contiguous(), share.contiguous(), w.k, self.y)
            block.residual_norm(h, y=self.y, scale=self.scale, h_out=h)
        self.lens.copy_(plan.lens)
        self.free = torch.roll(self.free, -int(plan.taken))
        return h

    def prompt(self, h, new):
        """Take a chunk of prompts: h [tokens][H] float32, the new tokens of all
        requests in order (updated in place), new int32 [requests]: how many
        each has."""
        w, T = self.w, h.shape[0]
        f32, bf = dict(device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
        plan = self.layers[0].cache.plan(self.table, T).update(self.lens, new, self.free)
        routed = experts.ExpertPlan(w.E, w.topk, T, hidden=w.H)
        x, y = torch.empty((T, w.H), **f32), torch.empty((T, w.H), **f32)
        act = torch.empty((T * w.topk, w.I), **bf)
        for layer in self.layers:
            heads, kv, dim = layer.q_heads, layer.kv_heads, layer.head_dim
            block.residual_norm(h, x, pre_weight=layer.norm1)
            qkv = (x.to(torch.bfloat16) @ layer.qkv).view(T, heads + 2 * kv, dim)
            layer.cache.append(qkv[:, heads:heads + kv], qkv[:, heads + kv:], plan.slots)
            attended = torch.empty((T, heads, dim), **bf)
            layer.cache.attend_chunk(qkv[:, :heads], self.table, plan.lens, plan.starts, attended)
            block.residual_norm(h, x, y=attended.view(T, -1) @ layer.out, scale=self.scale,
                                pre_weight=layer.norm2, h_out=h)
            xb = x.to(torch.bfloat16)
            top = torch.topk(xb.float() @ layer.router.float(), w.topk)
            routed.update(top.indices.to(torch.int32).contiguous())
            layer.experts.activate(xb, routed, act)
            layer.experts.combine(act, routed, top.values.softmax(-1).contiguous(), y)
            block.residual_norm(h, y=y, scale=self.scale, h_out=h)
        self.lens.copy_(plan.lens)
        self._collect()
        return h

    def _collect(self):
        self.pool.collect(self.table, self.lens)
        self.free = self.pool.free[:int(self.pool.count)].clone()

    def fork(self, parents, children):
        """Requests `children` (rows that hold nothing) go on from `parents`."""
        rows = [torch.tensor(r, dtype=torch.int32, device="cuda") for r in (parents, children)]
        self.pool.fork(*rows, self.table, self.lens, self.free)
        for layer in self.layers:
            layer.cache.copy_pages(self.pool.src, self.pool.dst)
        self._collect()

    def free_requests(self, rows):
        """End requests, and move the pages of the others to the front."""
        self.lens[rows] = 0
        self.pool.compact(self.table, self.lens)
        for layer in self.layers:
            layer.cache.copy_pages(self.pool.src, self.pool.dst, count=self.pool.moves)
        self.free = self.pool.free[:int(self.pool.count)].clone()

    def status(self):
        """Raise if a device-side check failed."""
        for layer in self.layers:
            for code, bits in (layer.cache.status(), layer.reader.status(),
                               layer.experts.status()):
                if code:
                    raise RuntimeError(f"device error bits {bits:#x} ({code})")


def main(steps=200, keep=4):
    decoder = Decoder()
    g = torch.Generator(device="cuda").manual_seed(1)
    new = torch.ones(decoder.requests, dtype=torch.int32, device="cuda")
    for name, kept in (("all pages", 0), (f"{keep} pages of {decoder.table.shape[1]}", keep)):
        decoder.lens.zero_()
        decoder.table.fill_(-1)
        for i in range(steps):
            if i == steps // 2:
                torch.cuda.synchronize()
                start = time.perf_counter()
            h = torch.randn((decoder.requests, decoder.w.H), generator=g, device="cuda")
            decoder.step(h, new, kept)
        torch.cuda.synchronize()
        ms = (time.perf_counter() - start) / (steps - steps // 2) * 1e3
        decoder.status()
        print(f"{name}: {decoder.requests} requests of {int(decoder.lens[0])} tokens, "
              f"{len(decoder.layers)} layers, {ms:.2f} ms a step, |h| {float(h.norm()):.3f}")
    decoder.free_requests(list(range(decoder.requests)))
    new = torch.tensor([100, 60, 0, 0], dtype=torch.int32, device="cuda")
    h = decoder.prompt(torch.randn((160, decoder.w.H), generator=g, device="cuda"), new)
    decoder.fork([0, 0], [2, 3])
    one = torch.ones(decoder.requests, dtype=torch.int32, device="cuda")
    decoder.step(torch.randn((decoder.requests, decoder.w.H), generator=g, device="cuda"), one)
    decoder.status()
    print(f"two prompts, |h| {float(h.norm()):.3f}; the first one continued in three ways: "
          f"{decoder.lens.tolist()} tokens, {decoder.free.shape[0]} pages free")


if __name__ == "__main__":
    main()
