"""The rest of a decode step around the MoE reader, and a prompt's attention: a
paged key/value cache and the norm that joins it to the reader.

``PagedCache`` wraps one layer's cache arrays: ``plan`` (page tables and slot
maps from request lengths), ``append`` (new rows into their slots),
``attend`` (one new token per request), ``attend_chunk`` (several: a prompt, a
chunk of one, drafted tokens) and ``select`` (pages by a cheap score, for
``attend(pages=...)``).  ``PagePool`` keeps track of a table's pages: free ones,
rows forked from others, the pool compacted (``copy_pages`` copies what moves).  ``residual_norm`` is post-norm, gate, scaled
residual and pre-norm in one pass.  Definitions, types and errors stand in
``include/moe_reader.h``; this module checks the tensors and marshals the
arguments.  Every call is asynchronous on the current stream (or ``stream``),
allocates nothing and can be captured in a CUDA graph.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import reader as _rd

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: 3}
ERR_LENGTH, ERR_PAGE, ERR_POOL, ERR_ROW = 0x20, 0x40, 0x80, 0x100

_I32 = torch.int32
_FLOATS = (torch.float32, torch.bfloat16, torch.float16)

# argument structs of include/moe_reader.h, packed (every pointer and 64-bit
# field stands before the 32-bit ones, so native order needs no padding)
_PLAN = struct.Struct("10Q4i")
_APPEND = struct.Struct("3Q4q2i")
_ATTEND = struct.Struct("7Q2q5if")
_SELECT = struct.Struct("4Q2q6i")
_CHUNK = struct.Struct("7Q2q5if")
_PAGES = struct.Struct("8Q2i")
_FORK = struct.Struct("8Q4i")
_COPY = struct.Struct("3Qi4x")
_NORM = struct.Struct("7Q6q7i2f4x")


class Config(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_requests", ctypes.c_int32),
                ("cache_type", ctypes.c_int32), ("flags", ctypes.c_int32)]


def _no_cuda(*_):
    raise RuntimeError("this build of torch has no CUDA")


# the current stream's handle on a device, and the current device; a torch built
# without CUDA lacks both, and the first call that needs one says so
_current = getattr(torch._C, "_cuda_getCurrentRawStream", _no_cuda)
_device = getattr(torch._C, "_cuda_getDevice", _no_cuda)


def _handle(stream):
    """The handle of a stream object, or of an integer that is one."""
    return stream if isinstance(stream, int) else stream.cuda_stream


def _check(code, what):
    if code != _rd.OK:
        raise _rd.ReaderError(code, what)


def _length(t, what):
    """Length of a tensor's first dimension."""
    if not isinstance(t, torch.Tensor) or t.dim() == 0:
        raise TypeError(f"{what} must be a CUDA tensor")
    return t.shape[0]


def _refuse(t, dtypes, shape, what, device):
    """Raise what is wrong with a tensor that failed its check."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{what} is on cuda:{t.get_device()}, not cuda:{device}")
    raise ValueError(f"{what} must be contiguous")


def _whole(t, dtype, shape, what, device):
    """Address of a contiguous CUDA tensor of one dtype and shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and \
                t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, (dtype,), shape, what, device)


def _table(t, rows, device):
    """(address, width) of a page table of at least `rows` rows."""
    try:
        n, width = t.shape
        if t.dtype is _I32 and n >= rows and t.get_device() == device and t.is_contiguous():
            return t.data_ptr(), width
    except (AttributeError, ValueError):
        pass
    width = t.shape[1] if isinstance(t, torch.Tensor) and t.dim() == 2 else 0
    _refuse(t, (_I32,), (max(rows, t.shape[0] if width else 0), width), "table", device)


class PagePlan:
    """Page table and slot map of one decode or prompt step (see
    ``PagedCache.plan``).  ``update`` fills, for the first R requests,
    ``lens`` [R], ``starts`` [R + 1], and for the new tokens ``slots``,
    ``positions`` and ``requests`` [max_tokens] (-1 behind the last), and
    ``taken`` [1], the free pages used."""

    def __init__(self, cache, table, max_tokens):
        _, self.width = _table(table, 0, cache.device)
        rows = table.shape[0]
        if rows > cache.max_requests:
            raise ValueError(f"table has {rows} rows for {cache.max_requests} requests")
        new = lambda n: torch.empty(n, dtype=_I32, device=table.device)  # noqa: E731
        self.cache, self.table, self.max_tokens = cache, table, int(max_tokens)
        self._lens, self._starts = new(max(rows, 1)), new(rows + 1)
        self.lens, self.starts = self._lens[:0], self._starts[:1]
        self.slots, self.positions = new(self.max_tokens), new(self.max_tokens)
        self.requests, self.taken = new(self.max_tokens), new(1)
        self._call = _rd._lib().moe_reader_kv_plan
        self._out = (self._lens.data_ptr(), self._starts.data_ptr(), self.slots.data_ptr(),
                     self.positions.data_ptr(), self.requests.data_ptr(), self.taken.data_ptr())

    def update(self, prev_lens, new_lens, free_pages, stream=None):
        """Plan a step: request r holds prev_lens[r] tokens and gets
        new_lens[r] more (int32 [R]); missing pages come from the front of
        free_pages (int32 [F]).  Updates ``table`` in place."""
        dev = self.cache.device
        R = _length(prev_lens, "prev_lens")
        prev = _whole(prev_lens, _I32, (R,), "prev_lens", dev)
        new = _whole(new_lens, _I32, (R,), "new_lens", dev)
        F = _length(free_pages, "free_pages")
        free = _whole(free_pages, _I32, (F,), "free_pages", dev)
        if R > self.table.shape[0]:
            raise ValueError(f"{R} requests for a table of {self.table.shape[0]} rows")
        args = _PLAN.pack(prev, new, self.table.data_ptr(), free, *self._out, R, self.width, F,
                          self.max_tokens)
        code = self._call(self.cache._h, args, _current(dev) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_kv_plan")
        if self.lens.shape[0] != R:
            self.lens, self.starts = self._lens[:R], self._starts[:R + 1]
        return self


class PagePool:
    """The pages of a pool that one page table refers to (see
    ``PagedCache.pool``): which are free, rows forked from others, and the ones
    in use moved to the front.  A table serves all layers, so these calls are
    made once, and the copies that they ask for (``src``, ``dst``) once a layer
    by ``PagedCache.copy_pages``.

    ``refs`` [pages], ``free`` [pages] (-1 behind the last) and ``count`` [1]
    are written by ``collect`` and ``compact``; ``src`` and ``dst`` by
    ``compact`` (with ``moves`` [1]) and ``fork`` (with ``taken`` [1])."""

    def __init__(self, cache, max_forks):
        n = cache.num_pages
        new = lambda n: torch.empty(n, dtype=_I32, device=cache.k.device)  # noqa: E731
        self.cache, self.max_forks = cache, int(max_forks)
        self.refs, self.free, self.count = new(n), new(n), new(1)
        self.moves, self.taken = new(1), new(1)
        self._moves = (new(n // 2), new(n // 2))
        self._forks = (new(max(self.max_forks, 1)), new(max(self.max_forks, 1)))
        self.src, self.dst = self._moves[0][:0], self._moves[1][:0]
        lib = _rd._lib()
        self._collect, self._compact = lib.moe_reader_kv_collect, lib.moe_reader_kv_compact
        self._fork = lib.moe_reader_kv_fork

    def _pages(self, call, name, table, lens, moves, stream):
        dev = self.cache.device
        R = _length(lens, "lens")
        tab, width = _table(table, R, dev)
        ln = _whole(lens, _I32, (R,), "lens", dev)
        args = _PAGES.pack(tab, ln, self.refs.data_ptr(), self.free.data_ptr(),
                           self.count.data_ptr(), *moves, R, width)
        code = call(self.cache._h, args, _current(dev) if stream is None else _handle(stream))
        if code:
            _check(code, name)
        return self

    def collect(self, table, lens, stream=None):
        """References and free pages of table (int32 [>= R][width]) with lens
        (int32 [R]; 0 frees a request's pages)."""
        return self._pages(self._collect, "moe_reader_kv_collect", table, lens, (0, 0, 0), stream)

    def compact(self, table, lens, stream=None):
        """``collect``, then the pages in use renumbered to the front of the
        pool: table is updated in place, src and dst list the moves (-1 behind
        the last of the pages // 2 that there can be)."""
        src, dst = self._moves
        self._pages(self._compact, "moe_reader_kv_compact", table, lens,
                    (src.data_ptr(), dst.data_ptr(), self.moves.data_ptr()), stream)
        self.src, self.dst = src, dst
        return self

    def fork(self, parents, children, table, lens, free_pages, stream=None):
        """Rows children (int32 [F]) of table continue rows parents (int32
        [F]): they share full pages, and a last page that is not full becomes a
        fresh one from the front of free_pages.  Updates table and lens (int32
        [rows]) in place; src and dst [F] list the copies, -1 for none."""
        dev = self.cache.device
        F = _length(parents, "parents")
        par = _whole(parents, _I32, (F,), "parents", dev)
        chi = _whole(children, _I32, (F,), "children", dev)
        if F > self.max_forks:
            raise ValueError(f"{F} forks for a pool of at most {self.max_forks}")
        R = _length(lens, "lens")
        tab, width = _table(table, R, dev)
        ln = _whole(lens, _I32, (R,), "lens", dev)
        N = _length(free_pages, "free_pages")
        free = _whole(free_pages, _I32, (N,), "free_pages", dev)
        src, dst = self._forks
        args = _FORK.pack(par, chi, tab, ln, free, src.data_ptr(), dst.data_ptr(),
                          self.taken.data_ptr(), F, R, width, N)
        code = self._fork(self.cache._h, args, _current(dev) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_kv_fork")
        self.src, self.dst = src[:F], dst[:F]
        return self


class PagedCache:
    """One layer's paged key/value cache.

    k, v: [pages][kv_heads][page_size][head_dim], bfloat16, float16 or
    float8_e4m3fn (then k_scale and v_scale, float32 [kv_heads], give what a
    stored value is multiplied by).  codes (int8 [pages][kv_heads][2][head_dim])
    and steps (float32 [pages][kv_heads]): the page summaries that ``append``
    keeps and ``select`` reads; leave both out for a cache that never selects.
    All tensors stay the caller's and are kept alive by this object."""

    def __init__(self, k, v, q_heads, max_requests=128, codes=None, steps=None, k_scale=None,
                 v_scale=None, stream=None):
        lib = _rd._lib()
        if not isinstance(k, torch.Tensor) or k.dtype not in TYPES or k.dtype == torch.float32:
            raise TypeError("k must be a bfloat16, float16 or float8_e4m3fn CUDA tensor")
        self.device = k.get_device()
        if not k.is_cuda or self.device != _device():
            raise ValueError("k must be on the current CUDA device")
        if k.dim() != 4:
            raise ValueError("k must be [pages][kv_heads][page_size][head_dim]")
        shape = tuple(int(n) for n in k.shape)
        _whole(k, k.dtype, shape, "k", self.device)
        _whole(v, k.dtype, shape, "v", self.device)
        pages, self.kv_heads, self.page_size, self.head_dim = shape
        self.k, self.v, self.num_pages = k, v, pages
        self.dtype, self.q_heads, self.max_requests = k.dtype, int(q_heads), int(max_requests)
        # rows and queries have the cache's type; an 8-bit cache takes either 16-bit one
        self._row_types = _FLOATS[1:] if k.dtype is torch.float8_e4m3fn else (k.dtype,)
        self._scale = self.head_dim ** -0.5
        ptr = [None] * 4
        for i, (t, dt, sh, name) in enumerate((
                (codes, torch.int8, (pages, self.kv_heads, 2, self.head_dim), "codes"),
                (steps, torch.float32, (pages, self.kv_heads), "steps"),
                (k_scale, torch.float32, (self.kv_heads,), "k_scale"),
                (v_scale, torch.float32, (self.kv_heads,), "v_scale"))):
            if t is not None:
                ptr[i] = _whole(t, dt, sh, name, self.device)
        self._keep = (k, v, codes, steps, k_scale, v_scale)
        cfg = Config(self.q_heads, self.kv_heads, self.head_dim, self.page_size, pages,
                     self.max_requests, TYPES[k.dtype], 0)
        self._append, self._attend = lib.moe_reader_kv_append, lib.moe_reader_kv_attend
        self._chunk = lib.moe_reader_kv_chunk
        self._select, self._copy = lib.moe_reader_kv_select, lib.moe_reader_kv_copy
        h = ctypes.c_void_p()
        at = _current(self.device) if stream is None else _handle(stream)
        _check(lib.moe_reader_kv_create(ctypes.byref(cfg), k.data_ptr(), v.data_ptr(), *ptr, at,
                                        ctypes.byref(h)), "moe_reader_kv_create")
        self._h = h

    # -- lifetime ---------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            _rd._lib().moe_reader_kv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self):
        """(code, error bits) since the last status; synchronizes the device."""
        bits = ctypes.c_uint32(0)
        code = _rd._lib().moe_reader_kv_status(self._h, ctypes.byref(bits))
        return code, bits.value

    # -- calls ------------------------------------------------------------
    def plan(self, table, max_tokens):
        """A PagePlan over table (int32 [requests][width], updated in place)
        for steps of at most max_tokens new tokens."""
        return PagePlan(self, table, max_tokens)

    def pool(self, max_forks=0):
        """A PagePool over this cache's pages, for calls of at most max_forks
        forks."""
        return PagePool(self, max_forks)

    def copy_pages(self, src, dst, count=None, stream=None):
        """Copy whole pages, keys, values and summaries: page src[i] to page
        dst[i] (int32 [n], -1 skips; a page stands once in dst at most and not
        in src too).  count (int32 [1]): only the first count[0] of them."""
        n = _length(src, "src")
        s = _whole(src, _I32, (n,), "src", self.device)
        d = _whole(dst, _I32, (n,), "dst", self.device)
        c = 0 if count is None else _whole(count, _I32, (1,), "count", self.device)
        code = self._copy(self._h, _COPY.pack(s, d, c, n),
                          _current(self.device) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_kv_copy")

    def append(self, k, v, slots, stream=None):
        """Write rows k, v ([tokens][kv_heads][head_dim], rows contiguous,
        any token and head stride) into slots (int32 [tokens], -1 skips)."""
        T = _length(slots, "slots")
        at = _whole(slots, _I32, (T,), "slots", self.device)
        shape = (T, self.kv_heads, self.head_dim)
        kp, ks, kt = self._rows(k, "k", shape)
        vp, vs, vt = self._rows(v, "v", shape)
        if vt != kt:
            raise TypeError("k and v must have one dtype")
        args = _APPEND.pack(kp, vp, at, ks[0], ks[1], vs[0], vs[1], kt, T)
        code = self._append(self._h, args,
                            _current(self.device) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_kv_append")

    def attend(self, q, table, lens, out, scale=None, window=0, sinks=None, lse=None, pages=None,
               stream=None):
        """Attention of one new token per request: q, out [R][q_heads][head_dim],
        table int32 [>= R][width], lens int32 [R].  scale defaults to
        head_dim ** -0.5; window > 0 keeps the last `window` tokens; sinks
        float32 [q_heads]; lse float32 [R][q_heads] receives the log of the
        denominator; pages int32 [R][kv_heads][keep] restricts the keys to
        these pages of each request (from ``select``)."""
        R, dev = _length(q, "q"), self.device
        shape = (R, self.q_heads, self.head_dim)
        qp, s, qt = self._rows(q, "q", shape)
        o = _whole(out, q.dtype, shape, "out", dev)
        tab, width = _table(table, R, dev)
        ln = _whole(lens, _I32, (R,), "lens", dev)
        pg = keep = sk = ls = 0
        if pages is not None:
            pg, keep = self._pages(pages, R)
        if sinks is not None:
            sk = _whole(sinks, torch.float32, (self.q_heads,), "sinks", dev)
        if lse is not None:
            ls = _whole(lse, torch.float32, (R, self.q_heads), "lse", dev)
        args = _ATTEND.pack(qp, tab, ln, pg, sk, o, ls, s[0], s[1], qt, R, width, keep, window,
                            self._scale if scale is None else scale)
        code = self._attend(self._h, args, _current(dev) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_kv_attend")

    def attend_chunk(self, q, table, lens, starts, out, scale=None, window=0, sinks=None, lse=None,
                     stream=None):
        """Attention of several new tokens per request, already appended: q,
        out [T][q_heads][head_dim], table int32 [>= R][width], lens int32 [R],
        starts int32 [R + 1] (a request's first row of q, as ``PagePlan.update``
        writes them; the rows are the last of its lens[r] tokens, and each sees
        itself and those before).  Rows outside of starts are left alone.  scale,
        window, sinks as for ``attend``; lse float32 [T][q_heads]."""
        T, R, dev = _length(q, "q"), _length(lens, "lens"), self.device
        shape = (T, self.q_heads, self.head_dim)
        qp, s, qt = self._rows(q, "q", shape)
        o = _whole(out, q.dtype, shape, "out", dev)
        tab, width = _table(table, R, dev)
        ln = _whole(lens, _I32, (R,), "lens", dev)
        st = _whole(starts, _I32, (R + 1,), "starts", dev)
        sk = ls = 0
        if sinks is not None:
            sk = _whole(sinks, torch.float32, (self.q_heads,), "sinks", dev)
        if lse is not None:
            ls = _whole(lse, torch.float32, (T, self.q_heads), "lse", dev)
        args = _CHUNK.pack(qp, tab, ln, st, sk, o, ls, s[0], s[1], qt, R, T, width, window,
                           self._scale if scale is None else scale)
        code = self._chunk(self._h, args, _current(dev) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_kv_chunk")

    def select(self, q, table, lens, pages, first=1, last=1, stream=None):
        """Choose pages.shape[2] pages per request and KV head by the page
        summaries' score against q, the first `first` and last `last` always
        among them; pages int32 [R][kv_heads][keep] receives them ascending."""
        R = _length(q, "q")
        qp, s, qt = self._rows(q, "q", (R, self.q_heads, self.head_dim))
        tab, width = _table(table, R, self.device)
        ln = _whole(lens, _I32, (R,), "lens", self.device)
        pg, keep = self._pages(pages, R)
        args = _SELECT.pack(qp, tab, ln, pg, s[0], s[1], qt, R, width, keep, first, last)
        code = self._select(self._h, args,
                            _current(self.device) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_kv_select")

    # -- checks -----------------------------------------------------------
    def _pages(self, pages, R):
        """(address, keep) of a list of pages per request and KV head."""
        keep = pages.shape[-1] if _length(pages, "pages") >= 0 else 0
        if keep < 1:      # an empty tensor's address would read as "no list"
            raise _rd.ReaderError(_rd.EINVAL, "pages holds no entry")
        return _whole(pages, _I32, (R, self.kv_heads, keep), "pages", self.device), keep

    def _rows(self, t, what, shape):
        """(address, strides, type code) of a tensor of rows for this cache."""
        try:
            if t.dtype in self._row_types and t.shape == shape and t.get_device() == self.device:
                s = t.stride()
                if s[2] == 1:
                    return t.data_ptr(), s, TYPES[t.dtype]
        except AttributeError:
            pass
        _refuse(t, self._row_types, shape, what + "'s rows", self.device)


def _matrix(t, what, shape, device):
    """(address, row stride, type code) of a float matrix with contiguous rows."""
    try:
        code = TYPES[t.dtype]
        if code < 3 and t.shape == shape and t.get_device() == device:
            if t.is_contiguous():
                return t.data_ptr(), shape[1], code
            s = t.stride()
            if s[1] == 1:
                return t.data_ptr(), s[0] if shape[0] > 1 else 0, code
    except (AttributeError, KeyError):
        pass
    _refuse(t, _FLOATS, shape, what + "'s rows", device)


def _weight(w, what, shape, device):
    """(address, type code) of a weight vector."""
    try:
        code = TYPES[w.dtype]
        if code < 3 and w.shape == shape and w.get_device() == device and w.is_contiguous():
            return w.data_ptr(), code
    except (AttributeError, KeyError):
        pass
    _refuse(w, _FLOATS, shape, what, device)


def _gate(g, rows, hidden, device):
    """(address, row stride, column stride, type code) of a gate."""
    try:
        code, shape = TYPES[g.dtype], g.shape
        if code < 3 and g.get_device() == device:
            s = g.stride()
            if shape == (rows, hidden):
                return g.data_ptr(), s[0] if rows > 1 else 0, s[1], code
            if shape == (hidden,):
                return g.data_ptr(), 0, s[0], code
            if shape == (rows, 1):
                return g.data_ptr(), s[0], 0, code
            raise ValueError(f"gate must be [hidden], [rows][1] or [rows][hidden], got "
                             f"{tuple(shape)}")
    except (AttributeError, KeyError):
        pass
    _refuse(g, _FLOATS, getattr(g, "shape", ()), "gate", device)


def residual_norm(h, x=None, y=None, post_weight=None, gate=None, scale=1.0, pre_weight=None,
                  eps=1e-6, h_out=None, stream=None):
    """z = rmsnorm(y) * post_weight (y itself without post_weight),
    h' = h + scale * gate * z (h itself without y), x = rmsnorm(h') * pre_weight.

    h, y, x, h_out: [rows][hidden], float32, bfloat16 or float16 each (h_out as
    h; it may be h).  gate: [hidden], [rows][1] or [rows][hidden].  Weights:
    [hidden] of one dtype.  x or h_out may be left out, not both."""
    try:
        dev, shape = h.get_device(), h.shape
        rows, hidden = shape
    except (AttributeError, ValueError):
        raise TypeError("h must be a CUDA tensor [rows][hidden]") from None
    if dev < 0:
        raise TypeError("h must be a CUDA tensor [rows][hidden]")
    if dev != _device():
        raise ValueError(f"h is on cuda:{dev}, not the current device")
    hp, hs, ht = _matrix(h, "h", shape, dev)
    yp = ys = yt = xp = xs = xt = op = os_ = gp = grow = gcol = gt = pp = qp = wt = 0
    if y is not None:
        yp, ys, yt = _matrix(y, "y", shape, dev)
    if x is not None:
        xp, xs, xt = _matrix(x, "x", shape, dev)
    if h_out is not None:
        op, os_, ot = _matrix(h_out, "h_out", shape, dev)
        if ot != ht:
            raise TypeError("h_out must have h's dtype")
    if gate is not None:
        gp, grow, gcol, gt = _gate(gate, rows, hidden, dev)
    if post_weight is not None:
        pp, wt = _weight(post_weight, "post_weight", (hidden,), dev)
    if pre_weight is not None:
        qp, qt = _weight(pre_weight, "pre_weight", (hidden,), dev)
        if pp and qt != wt:
            raise TypeError("post_weight and pre_weight must have one dtype")
        wt = qt
    args = _NORM.pack(hp, yp, gp, pp, qp, op, xp, hs, ys, os_, xs, grow, gcol, rows, hidden, ht, yt,
                      xt, gt, wt, scale, eps)
    code = _rd._lib().moe_reader_residual_norm(
        args, _current(dev) if stream is None else _handle(stream))
    if code:
        _check(code, "moe_reader_residual_norm")
