"""A prompt's experts: dense products grouped by expert.

The reader decodes a few tokens by reading a few channels of their experts; a
prompt's tokens want nearly all of them.  ``ExpertPlan`` sorts a batch's pairs
(token, slot) by expert, ``Experts.activate`` computes the gated activations
silu(G_e x) * (V_e x) of every pair, ``Experts.combine`` their down products,
weighted and summed per token.  Definitions, types and errors stand in
``include/moe_reader.h``; this module checks the tensors and marshals the
arguments.  Every call is asynchronous on the current stream (or ``stream``),
allocates nothing and can be captured in a CUDA graph.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import reader as _rd
from .block import _I32, _check, _current, _device, _handle, _length, _matrix, _refuse, _whole

_TYPES = {torch.bfloat16: 1, torch.float16: 2}

# argument structs of include/moe_reader.h
_PLAN = struct.Struct("5Q3i4x")
_ACTIVATE = struct.Struct("4Qq2i")
_COMBINE = struct.Struct("6Qq3i4x")


class Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("type", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class ExpertPlan:
    """Pairs (token * topk + slot) of a batch sorted by expert.  ``update``
    fills, for T tokens, ``order`` [T * topk] (the pair of each row, -1 behind
    the last), ``offsets`` [experts + 1] (each expert's first row), ``places``
    [T][topk] (each pair's row; -1 for an id that is no expert) and ``skipped``
    [1] (how many of those).  One plan serves all layers of a step in turn.
    hidden: the width of ``combine``'s scratch, float32 [max_tokens *
    topk][hidden]; leave it out where ``combine`` is not called."""

    def __init__(self, experts, topk, max_tokens, hidden=0):
        self.device = _device()
        new = lambda n, dt=_I32: torch.empty(n, dtype=dt, device=f"cuda:{self.device}")  # noqa: E731
        self.experts, self.topk, self.max_tokens = int(experts), int(topk), int(max_tokens)
        pairs = self.max_tokens * self.topk
        self._order, self._places = new(pairs), new(pairs)
        self.offsets, self.skipped = new(self.experts + 1), new(1)
        self.slots = new((pairs, int(hidden)), torch.float32) if hidden else None
        self._call = _rd._lib().moe_reader_experts_plan
        self._resize(0)

    def _resize(self, tokens):
        self.tokens = tokens
        self.order = self._order[:tokens * self.topk]
        self.places = self._places[:tokens * self.topk].view(tokens, self.topk)

    def update(self, ids, stream=None):
        """Plan a batch: ids int32 [T][topk], the experts of each token."""
        T = _length(ids, "ids")
        at = _whole(ids, _I32, (T, self.topk), "ids", self.device)
        if T > self.max_tokens:
            raise ValueError(f"{T} tokens for a plan of at most {self.max_tokens}")
        if self.device != _device():
            raise ValueError(f"the plan is on cuda:{self.device}, not the current device")
        args = _PLAN.pack(at, self._order.data_ptr(), self.offsets.data_ptr(),
                          self._places.data_ptr(), self.skipped.data_ptr(), T, self.topk,
                          self.experts)
        code = self._call(args, _current(self.device) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_experts_plan")
        if T != self.tokens:
            self._resize(T)
        return self


class Experts:
    """One layer's expert weights: gate, up [experts][inter][hidden] and down
    [experts][hidden][inter], bfloat16 or float16, contiguous.  Leave out gate
    and up, or down, where only one of the calls is made.  The tensors stay the
    caller's and are kept alive by this object."""

    def __init__(self, gate=None, up=None, down=None, stream=None):
        lib = _rd._lib()
        first = gate if gate is not None else down
        if not isinstance(first, torch.Tensor) or first.dtype not in _TYPES or first.dim() != 3:
            raise TypeError("gate or down must be a bfloat16 or float16 CUDA tensor [experts][.][.]")
        if (gate is None) != (up is None):
            raise ValueError("gate and up go together")
        self.device = first.get_device()
        if not first.is_cuda or self.device != _device():
            raise ValueError("the weights must be on the current CUDA device")
        self.experts, a, b = (int(n) for n in first.shape)
        self.inter, self.hidden = (a, b) if gate is not None else (b, a)
        self.dtype = first.dtype
        wide, tall = (self.experts, self.inter, self.hidden), (self.experts, self.hidden, self.inter)
        ptr = [None if t is None else _whole(t, self.dtype, shape, name, self.device)
               for t, shape, name in ((gate, wide, "gate"), (up, wide, "up"), (down, tall, "down"))]
        self._keep = (gate, up, down)
        self._activate = lib.moe_reader_experts_activate
        self._combine = lib.moe_reader_experts_combine
        cfg = Config(self.hidden, self.inter, self.experts, _TYPES[self.dtype], 0)
        h = ctypes.c_void_p()
        at = _current(self.device) if stream is None else _handle(stream)
        _check(lib.moe_reader_experts_create(ctypes.byref(cfg), *ptr, at, ctypes.byref(h)),
               "moe_reader_experts_create")
        self._h = h

    # -- lifetime ---------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            _rd._lib().moe_reader_experts_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self):
        """(code, error bits) since the last status; synchronizes the device."""
        bits = ctypes.c_uint32(0)
        code = _rd._lib().moe_reader_experts_status(self._h, ctypes.byref(bits))
        return code, bits.value

    # -- calls ------------------------------------------------------------
    def activate(self, x, plan, act, stream=None):
        """act [T * topk][inter]: row j gets silu(G_e x_t) * (V_e x_t) of the
        plan's pair order[j]; x [T][hidden] (rows contiguous), both of the
        weights' dtype.  Rows behind the plan's last are left alone."""
        T = self._plan(plan)
        xp, xs = self._rows(x, "x", (T, self.hidden))
        rows = T * plan.topk
        ap = _whole(act, self.dtype, (rows, self.inter), "act", self.device)
        args = _ACTIVATE.pack(xp, plan._order.data_ptr(), plan.offsets.data_ptr(), ap, xs, T,
                              plan.topk)
        code = self._activate(self._h, args,
                              _current(self.device) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_experts_activate")

    def combine(self, act, plan, weights, y, stream=None):
        """y [T][hidden] (float32, bfloat16 or float16, rows contiguous): the
        sum over a token's slots of weights[t][slot] (float32) times D_e act of
        the pair's row.  Uses the plan's scratch (``hidden`` at its creation)."""
        T = self._plan(plan)
        rows = T * plan.topk
        ap = _whole(act, self.dtype, (rows, self.inter), "act", self.device)
        wp = _whole(weights, torch.float32, (T, plan.topk), "weights", self.device)
        yp, ys, yt = _matrix(y, "y", (T, self.hidden), self.device)
        if plan.slots is None or plan.slots.shape[1] < self.hidden:
            raise ValueError(f"the plan has no scratch for {self.hidden} columns")
        args = _COMBINE.pack(ap, plan.offsets.data_ptr(), plan._places.data_ptr(), wp,
                             plan.slots.data_ptr(), yp, ys, T, plan.topk, yt)
        code = self._combine(self._h, args,
                             _current(self.device) if stream is None else _handle(stream))
        if code:
            _check(code, "moe_reader_experts_combine")

    # -- checks -----------------------------------------------------------
    def _plan(self, plan):
        """Tokens of a plan that fits these weights."""
        if not isinstance(plan, ExpertPlan):
            raise TypeError("plan must be an ExpertPlan")
        if plan.experts != self.experts:
            raise ValueError(f"a plan over {plan.experts} experts for {self.experts}")
        if plan.device != self.device:
            raise ValueError(f"the plan is on cuda:{plan.device}, not cuda:{self.device}")
        return plan.tokens

    def _rows(self, t, what, shape):
        """(address, row stride) of a matrix of the weights' type."""
        at, stride, code = _matrix(t, what, shape, self.device)
        if code != _TYPES[self.dtype]:
            _refuse(t, (self.dtype,), shape, what, self.device)
        return at, stride
