"""Shared-prefix cache: binding of the hkv_shared_* calls (include/hkv.h).

A batch whose sequences continue shared prompts (the images of one prompt,
the unconditional streams of all of them) holds each prompt's keys and values
once; every sequence adds its own tokens, whose attention weights accumulate
and decide what an eviction drops.  This module marshals arguments only.
"""
from __future__ import annotations

import ctypes as C
from bisect import bisect_right
from contextlib import contextmanager
from dataclasses import dataclass, replace

import torch

from ._lib import DTYPE_BF16, DTYPE_F32, _check, lib


class _Cache(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "dtype", "head_dim", "num_seqs", "num_heads", "num_kv_heads", "capacity", "num_prefixes",
        "prefix_capacity")] + [
        ("k", C.c_void_p), ("v", C.c_void_p), ("k_stride", C.c_int64 * 3), ("v_stride", C.c_int64 * 3),
        ("pos", C.c_void_p), ("weight", C.c_void_p), ("len", C.c_void_p), ("next_pos", C.c_void_p),
        ("prefix_k", C.c_void_p), ("prefix_v", C.c_void_p), ("prefix_k_stride", C.c_int64 * 3),
        ("prefix_v_stride", C.c_int64 * 3), ("prefix_len", C.c_void_p), ("prefix_of", C.c_void_p),
        ("status", C.c_void_p)]


#: Attributes that the C descriptor points into.
_BUFFERS = frozenset(("k", "v", "pos", "weight", "lens", "next_pos", "prefix_k", "prefix_v", "prefix_lens", "prefix_of",
                      "status"))
_Strides = C.c_int64 * 3
_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _reaches(dims, lo, hi):
    """Whether some sum of n_i s_i lies in (lo, hi): dims are (s_i, least n_i, most
    n_i), largest s_i first."""
    if not dims:
        return lo < 0 < hi
    (s, a, b), rest = dims[0], dims[1:]
    least, most = sum(t * x for t, x, _ in rest), sum(t * y for t, _, y in rest)
    # n s + [least, most] meets (lo, hi): n from (lo - most) / s to (hi - least) / s
    return any(_reaches(rest, lo - n * s, hi - n * s)
               for n in range(max(a, -((most - lo) // s)), min(b, (hi - least) // s) + 1))


def _extent(x):
    """The bytes from the first to the last of a tensor's elements."""
    at, last = x.data_ptr(), 1
    if x.is_contiguous():
        return at, at + x.nbytes
    for n, s in zip(x.shape, x.stride()):
        if n == 0:
            return at, at
        last += (n - 1) * s
    return at, at + last * x.element_size()


def _overlap(x, y):
    """Whether two tensors hold a common byte.  Their last dimensions are
    contiguous rows of one dtype's elements; views that lie between each other's
    rows do not overlap."""
    (xa, xb), (ya, yb) = _extent(x), _extent(y)
    if xb <= ya or yb <= xa:
        return False
    span = {}  # stride in bytes -> the range of index differences
    for t, sign in ((x, 1), (y, -1)):
        for n, s in zip(t.shape[:-1], t.stride()):
            if n > 1 and s:
                a, b = span.get(s * t.element_size(), (0, 0))
                span[s * t.element_size()] = (a, b + n - 1) if sign > 0 else (a - n + 1, b)
    # a row of x starts less than a row of x before, or of y behind, the start of one of y
    rx, ry = x.shape[-1] * x.element_size(), y.shape[-1] * y.element_size()
    return _reaches([(s, *r) for s, r in sorted(span.items(), reverse=True)], ya - xa - rx, ya - xa + ry)


@dataclass
class SharedConfig:
    num_seqs: int
    num_heads: int          # query heads, a multiple of num_kv_heads
    num_kv_heads: int
    head_dim: int           # 64 or 128
    capacity: int           # own slots of each (sequence, KV head)
    num_prefixes: int = 0   # prompts shared by the sequences
    prefix_capacity: int = 0
    dtype: int = DTYPE_BF16

    @property
    def torch_dtype(self):
        return torch.float32 if self.dtype == DTYPE_F32 else torch.bfloat16


class SharedPrefixCache:
    """Keys and values of a batch: prompts held once, and each sequence's own
    tokens with the attention weight they have received.

    The buffers are ordinary tensors, allocated here or given by the caller
    (any strides with unit stride in d and 16-byte rows for the four row
    buffers), and may be read and written in place between calls; the cache
    stays bound to them, so that none can be replaced by another:
      k, v                [S, Hkv, capacity, d]       own rows
      pos, weight         [S, Hkv, capacity]          int32, float32
      lens, next_pos      [S, Hkv]                    int32
      prefix_k, prefix_v  [G, Hkv, prefix_capacity, d]
      prefix_lens         [G]                         int32
      prefix_of           [S]                         int32; outside 0..G-1: no prompt
    Calls only enqueue on the stream (the current one of the cache's device
    unless given) and must be ordered when they write the same buffers.  Tensors
    given to a call on another stream than their own are to be kept until it has
    run there; what it returns belongs to its stream.
    Scratch is allocated per call from the stream's memory pool, so calls on
    several streams and captured graphs never share it.
    No call has a gradient: a tensor that asks for one is refused where
    gradients are recorded (detach it, or call under torch.no_grad()).
    """

    def __init__(self, cfg: SharedConfig, device=None, *, k=None, v=None, pos=None, weight=None, lens=None,
                 next_pos=None, prefix_k=None, prefix_v=None, prefix_lens=None, prefix_of=None):
        self.cfg = cfg = replace(cfg)  # (the caller's may change, and serve another cache)
        dev = torch.device(device if device is not None else "cuda")
        if dev.type != "cuda":
            raise ValueError(f"device: expected a CUDA device, got {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self._index = dev, dev.index
        S, Hk, d, cap, G = cfg.num_seqs, cfg.num_kv_heads, cfg.head_dim, cfg.capacity, cfg.num_prefixes
        if cfg.dtype not in (DTYPE_F32, DTYPE_BF16) or d not in (64, 128) or S < 1 or Hk < 1 or \
                cfg.num_heads < 1 or cfg.num_heads % Hk or cap < 1 or G < 0 or (G > 0 and cfg.prefix_capacity < 1):
            raise ValueError(f"unusable config {cfg}")
        # the sizes that the descriptor is made of, and that calls are checked against
        self._S, self._H, self._Hk, self._d, self._cap = S, cfg.num_heads, Hk, d, cap
        dt = cfg.torch_dtype

        def own(x, name, shape, dtype, rows=False):
            if x is None:
                return torch.zeros(shape, dtype=dtype, device=dev)
            if not isinstance(x, torch.Tensor) or x.device != dev or x.dtype != dtype or tuple(x.shape) != shape:
                raise ValueError(f"{name}: expected a {dtype} tensor {list(shape)} on {dev}")
            if x.requires_grad:
                self._no_grad(name)
            if rows:
                self._rows(x, name)
            elif not x.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous tensor")
            return x

        self._dtype = dt
        self._off16 = 16 // dt.itemsize - 1  # bits that strides on 16-byte boundaries leave clear
        i32, f32 = torch.int32, torch.float32
        self.k = own(k, "k", (S, Hk, cap, d), dt, True)
        self.v = own(v, "v", (S, Hk, cap, d), dt, True)
        self.pos = own(pos, "pos", (S, Hk, cap), i32)
        self.weight = own(weight, "weight", (S, Hk, cap), f32)
        self.lens = own(lens, "lens", (S, Hk), i32)
        self.next_pos = own(next_pos, "next_pos", (S, Hk), i32)
        if not G:
            self.prefix_k = self.prefix_v = self.prefix_lens = self.prefix_of = None
        else:
            P = cfg.prefix_capacity
            self.prefix_k = own(prefix_k, "prefix_k", (G, Hk, P, d), dt, True)
            self.prefix_v = own(prefix_v, "prefix_v", (G, Hk, P, d), dt, True)
            self.prefix_lens = own(prefix_lens, "prefix_lens", (G,), i32)
            self.prefix_of = own(prefix_of, "prefix_of", (S,), i32)
        self.status = torch.zeros(2, dtype=i32, device=dev)
        self._buffers = [x for x in (getattr(self, n) for n in sorted(_BUFFERS)) if x is not None]
        # their extents in ascending order, those that meet as one (see _apart)
        self._starts, self._ends = [], []
        for a, b in sorted(_extent(x) for x in self._buffers):
            if self._ends and a < self._ends[-1]:
                self._ends[-1] = max(self._ends[-1], b)
            else:
                self._starts.append(a)
                self._ends.append(b)

        c = _Cache(cfg.dtype, d, S, cfg.num_heads, Hk, cap, G, cfg.prefix_capacity if G else 0)
        c.k, c.v = self.k.data_ptr(), self.v.data_ptr()
        c.k_stride, c.v_stride = _Strides(*self.k.stride()[:3]), _Strides(*self.v.stride()[:3])
        c.pos, c.weight = self.pos.data_ptr(), self.weight.data_ptr()
        c.len, c.next_pos = self.lens.data_ptr(), self.next_pos.data_ptr()
        if G:
            c.prefix_k, c.prefix_v = self.prefix_k.data_ptr(), self.prefix_v.data_ptr()
            c.prefix_k_stride = _Strides(*self.prefix_k.stride()[:3])
            c.prefix_v_stride = _Strides(*self.prefix_v.stride()[:3])
            c.prefix_len, c.prefix_of = self.prefix_lens.data_ptr(), self.prefix_of.data_ptr()
        c.status = self.status.data_ptr()
        self._c = c
        self._ref = C.byref(c)
        n = C.c_size_t()
        _check(lib().hkv_shared_evict_bytes(self._ref, C.byref(n)), "hkv_shared_evict_bytes")
        self._evict_bytes = n.value
        self._evict_like = self.lens.new_empty(1).expand(self._evict_bytes // 4)
        self._plans = {}  # (T, accumulate) -> see _plan
        L = lib()
        self._append_fn, self._attend_fn, self._evict_fn = L.hkv_shared_append, L.hkv_shared_attend, L.hkv_shared_evict

    def __setattr__(self, name, value):
        if name in _BUFFERS and getattr(self, name, value) is not value:
            raise AttributeError(f"{name}: the cache stays bound to this buffer; write into it, or make another cache")
        super().__setattr__(name, value)

    # -- argument checks (each a few hundred nanoseconds: a decode step's calls
    #    take the GPU ten to twenty microseconds) ------------------------------
    def _rows(self, x, name):
        st = x.stride()
        if st[3] != 1 or (st[0] | st[1] | st[2]) & self._off16 or x.data_ptr() & 15:
            raise ValueError(f"{name}: rows of d contiguous elements on 16-byte boundaries, got strides {st}")
        return _Strides(st[0], st[1], st[2])

    def _tensor(self, x, name, heads):
        """Checks a [S, heads, T, d] tensor; its strides for the C call."""
        if isinstance(x, torch.Tensor) and x.dtype == self._dtype and x.dim() == 4:
            n0, n1, _, n3 = x.shape
            if n0 == self._S and n1 == heads and n3 == self._d and x.device == self.device:
                if x.requires_grad:
                    self._no_grad(name)
                return self._rows(x, name)
        raise ValueError(f"{name}: expected a {self._dtype} tensor [{self._S}, {heads}, T, {self._d}] on {self.device}")

    def _apart(self, q, out, lse):
        """Refuses an out or lse that shares memory with q, each other or the
        cache.  Their extents nearly always lie apart, which takes 2 us."""
        seen = [(*_extent(q), q)]
        for name, x in (("out", out), ("lse", lse)):
            if x is None:
                continue
            a, b = _extent(x)
            i = bisect_right(self._ends, a)  # the first extent that ends behind x's start
            if i < len(self._starts) and self._starts[i] < b and any(_overlap(x, y) for y in self._buffers):
                raise ValueError(f"{name}: overlaps a buffer of the cache")
            for lo, hi, y in seen:
                if a < hi and lo < b and _overlap(x, y):
                    raise ValueError(f"{name}: overlaps q or out")
            seen.append((a, b, x))

    def _no_grad(self, name):
        if torch.is_grad_enabled():
            raise ValueError(f"{name}: asks for a gradient, which the cache's calls do not have")

    @contextmanager
    def _on(self, stream):
        """The cache's device and `stream` (its current one by default) as
        torch's current ones, for allocations and launches; gives the handle."""
        if stream is None:
            with torch.cuda.device(self._index):
                yield _current_stream(self._index)
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device) if int(stream) else \
                torch.cuda.default_stream(self.device)
        if stream.device != self.device:
            raise ValueError(f"stream: of {stream.device}, the cache is on {self.device}")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream

    # -- calls ---------------------------------------------------------------
    def append(self, k_t, v_t, weight_t=None, stream=None):
        """Adds T tokens to every head: k_t, v_t [S, Hkv, T, d]; weight_t
        [S, Hkv, T] fp32, their accumulated weights (default 0); none of them
        views of the cache.  A head without T free slots is left as it was
        (see check)."""
        ks = self._tensor(k_t, "k_t", self._Hk)
        vs = self._tensor(v_t, "v_t", self._Hk)
        T = k_t.shape[2]
        if v_t.shape[2] != T or T > self._cap:
            raise ValueError("k_t, v_t: as many tokens each, at most the capacity")
        if weight_t is not None and (weight_t.dtype != torch.float32 or weight_t.device != self.device or
                                     weight_t.shape != (self._S, self._Hk, T) or
                                     not weight_t.is_contiguous()):
            raise ValueError("weight_t: expected a contiguous float32 [S, Hkv, T] tensor on the device")
        if weight_t is not None and weight_t.requires_grad:
            self._no_grad("weight_t")
        if T == 0:
            return
        w = None if weight_t is None else weight_t.data_ptr()
        if stream is None and _current_device() == self._index:
            code = self._append_fn(self._ref, k_t.data_ptr(), ks, v_t.data_ptr(), vs, w, T, _current_stream(self._index))
        else:
            with self._on(stream) as handle:
                code = self._append_fn(self._ref, k_t.data_ptr(), ks, v_t.data_ptr(), vs, w, T, handle)
        if code:
            _check(code, "hkv_shared_append")

    def attend(self, q, out=None, lse=None, accumulate=True, scale=None, stream=None):
        """Attention of each sequence's newest T tokens (appended before, with
        no eviction in between: it moves tokens to other slots):
        q [S, H, T, d] over the sequence's prompt and own tokens, query t
        seeing the own slots before len - T + t + 1.  Returns (out
        [S, H, T, d], lse float32 [S, H, T]); a query that sees nothing gets
        zeros and -inf.  out and lse, where given, share no memory with q, each
        other or the cache.  accumulate adds to `weight` the softmax weights each
        own token received.  scale of the logits: 1 / sqrt(d) by default."""
        qs = self._tensor(q, "q", self._H)
        accumulate = bool(accumulate)
        plan = self._plans.get((q.shape[2], accumulate))
        if plan is None:
            plan = self._plan(q.shape[2], accumulate)
        if not (qs[0] and qs[1] and qs[2]) and any(n > 1 and st == 0 for n, st in zip(q.shape, q.stride())):
            raise ValueError("q: no repeated rows")
        if scale is None:
            scale = 0.0
        elif not (scale != 0 and abs(scale) < float("inf")):
            raise ValueError("scale: a finite number other than 0")
        if out is not None:
            self._tensor(out, "out", self._H)
            if out.shape != q.shape or 0 in out.stride() or out.data_ptr() == q.data_ptr():
                raise ValueError("out: expected q's shape, no repeated rows, and not q itself")
        if lse is not None and (lse.dtype != torch.float32 or lse.device != self.device or
                                lse.shape != q.shape[:3] or not lse.is_contiguous()):
            raise ValueError("lse: expected a contiguous float32 [S, H, T] tensor on the device")
        if out is not None or lse is not None:
            self._apart(q, out, lse)

        if stream is None and _current_device() == self._index:
            return self._attend(q, qs, out, lse, plan, scale, _current_stream(self._index))
        with self._on(stream) as handle:
            return self._attend(q, qs, out, lse, plan, scale, handle)

    def _attend(self, q, qs, out, lse, plan, scale, handle):
        T, accumulate, need, lse_like, scratch_like = plan
        so = qs
        if out is None and q.is_contiguous():
            out = torch.empty_like(q)
        else:
            if out is None:
                out = q.new_empty(q.shape)
            so = _Strides(*out.stride()[:3])
        if lse is None:
            lse = torch.empty_like(lse_like)
        scratch = torch.empty_like(scratch_like)  # (held until the launches are enqueued)
        code = self._attend_fn(self._ref, q.data_ptr(), qs, out.data_ptr(), so, lse.data_ptr(), T, scale, accumulate,
                               scratch.data_ptr(), need, handle)
        if code:
            _check(code, "hkv_shared_attend")
        return out, lse

    def _plan(self, T, accumulate):
        """What a call of these sizes needs: kept, as it depends on nothing
        else.  (empty_like of an expanded element is the cheapest allocation.)"""
        if T < 1 or T > self._cap:
            raise ValueError("q: between 1 token and the capacity")
        acc, n = int(accumulate), C.c_size_t()
        _check(lib().hkv_shared_attend_bytes(self._ref, T, acc, C.byref(n)), "hkv_shared_attend_bytes")
        plan = (T, acc, n.value, self.weight.new_empty(1).expand(self._S, self._H, T),
                self.lens.new_empty(1).expand(n.value // 4))
        self._plans[(T, accumulate)] = plan
        return plan

    def evict(self, budgets, recent: int = 0, slack: int = 1, stream=None):
        """Brings every head holding at least budget + slack tokens back to
        its budget (int32 [S, Hkv] on the device): the tokens lowest in
        (recent, weight, position, slot) go, `recent` being those less than
        that many positions behind the newest; survivors behind the budget
        move into the holes before it."""
        if not isinstance(budgets, torch.Tensor) or budgets.dtype != torch.int32 or budgets.device != self.device or \
                budgets.shape != (self._S, self._Hk) or not budgets.is_contiguous():
            raise ValueError("budgets: expected a contiguous int32 [S, Hkv] tensor on the device")
        if not (0 <= recent < 1 << 31 and 1 <= slack < 1 << 31):
            raise ValueError("recent at least 0, slack at least 1, both below 2**31")

        if stream is None and _current_device() == self._index:
            self._evict(budgets, recent, slack, _current_stream(self._index))
        else:
            with self._on(stream) as handle:
                self._evict(budgets, recent, slack, handle)

    def _evict(self, budgets, recent, slack, handle):
        scratch = torch.empty_like(self._evict_like)
        code = self._evict_fn(self._ref, budgets.data_ptr(), recent, slack, scratch.data_ptr(), self._evict_bytes, handle)
        if code:
            _check(code, "hkv_shared_evict")

    def check(self, stream=None):
        """(code, detail) of the first error latched on the device by the calls
        enqueued on the stream (waits for them)."""
        with self._on(stream):
            code, detail = self.status.tolist()
        return code, detail

    def clear_error(self, stream=None):
        with self._on(stream):
            self.status.zero_()
