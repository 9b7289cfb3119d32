"""A paged key/value cache in 16 bits over torch tensors: the dfl_paged_* calls of include/dfl.h with their
arguments checked and marshalled. Nothing here computes: every call is one of the library's.

A step of a server over it, lengths staying on the device (`length`, `n`: int32 [n_seq], the tokens that each
sequence has committed and the rows that it brings; a sequence that has ended has 0 of both):

    cu, slots = cache.plan(length, n, rows)         # rows of the step's buffers, spare ones among them
    cache.append(k, v, slots)                       # a layer's new keys and values, rows packed
    out = cache.prompt(q, k, v, cu)                 # whole prompts, or
    out = cache.attn(q, cu, length, 8)              # a token's or a verify's rows, at most 8 a sequence
    length += kept                                  # rows that are not kept are written again by the next step
"""
from __future__ import annotations

import ctypes

from . import _abi
from ._abi import DFL_BF16, DFL_E_INVALID_ARG, DFL_F16, DFL_OK, DflError, dfl_paged


def _refuse(msg: str):
    raise DflError(DFL_E_INVALID_ARG, msg)


MOST = 2 ** 31 - 1       # of a size: the library's are 32-bit numbers, and what is larger would arrive as another one


class PagedCache:
    """A dfl_paged over the caller's tensors (layouts in include/dfl.h), or `empty(...)` to allocate them.

    Calls enqueue on the device's current stream and return without synchronising; `status()` synchronises and
    raises what a call met on the device. The attention's scratch belongs to the object: calls of one cache must
    not overlap on the GPU. It grows with the largest call so far, and no piece of it is ever freed before the
    object, so captured graphs stay valid. The layers of a model each have a PagedCache with k and v of their own
    over the same table, held, free and queue; one of them plans.
    """

    def __init__(self, k, v, table, held, free, queue):
        import torch
        self.torch = torch
        types = {torch.bfloat16: DFL_BF16, torch.float16: DFL_F16}
        if k.dim() != 4 or k.dtype not in types or table.dim() != 2:
            _refuse("k must be bf16 or fp16 [n_pages][n_kv][page][head_dim], table int32 [n_seq][max_pages]")
        N, H, P, hd = k.shape
        S, most = table.shape
        i32 = torch.int32
        want = {"k": (k, k.dtype, (N, H, P, hd)), "v": (v, k.dtype, (N, H, P, hd)), "table": (table, i32, (S, most)), "held": (held, i32, (S,)),
                "free": (free, i32, (N,)), "queue": (queue, i32, (4,))}
        for name, (t, dtype, shape) in want.items():
            if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != k.device:
                _refuse(f"{name} must be contiguous {dtype} {list(shape)} on {k.device}")
        if max(N, H, P, hd, S, most) > MOST:
            _refuse("sizes of the cache must be below 2^31")
        self.n_seq, self.n_kv, self.head_dim, self.page, self.n_pages, self.max_pages = S, H, hd, P, N, most
        self.device, self.dtype = k.device, k.dtype
        if self.device.type != "cuda":
            _refuse("the cache's tensors must be on a CUDA device")
        self.k, self.v, self.table, self.held, self.free, self.queue = k, v, table, held, free, queue
        self.err = torch.zeros(64, dtype=i32, device=self.device)
        self.L = _abi.lib()
        self._idx, self._i32 = self.device.index, i32
        self._current_device, self._stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self._streams = set()         # that calls have used since the tensors were last recorded with them
        self.c = dfl_paged(S, H, hd, P, N, most, types[k.dtype], *(t.data_ptr() for t in (k, v, table, held, free, queue, self.err)))
        self._c = ctypes.byref(self.c)
        self._scale = hd ** -0.5
        self._kept, self._scratch, self._scratch_ptr, self._scratch_bytes, self._need = [], None, 0, 0, {}

    @classmethod
    def empty(cls, n_seq: int, n_kv: int, head_dim: int, n_pages: int, max_pages: int, page: int = 64, dtype=None, device="cuda:0") -> "PagedCache":
        """An empty cache of n_pages pages of `page` tokens, at most max_pages of them a sequence; dtype: torch.bfloat16 or torch.float16."""
        import torch
        if head_dim not in (64, 128, 256) or page not in (16, 32, 64, 128) or min(n_seq, n_kv, n_pages, max_pages) < 1:
            _refuse("head_dim must be 64, 128 or 256, page 16, 32, 64 or 128 and the sizes positive")
        dtype = torch.bfloat16 if dtype is None else dtype
        mk = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        shape, i32 = (n_pages, n_kv, page, head_dim), torch.int32
        self = cls(mk(dtype, *shape), mk(dtype, *shape), mk(i32, n_seq, max_pages), mk(i32, n_seq), mk(i32, n_pages), mk(i32, 4))
        self._call(self.L.dfl_paged_init, "dfl_paged_init")
        return self

    # ---- marshalling (a short call's time is mostly the host's: attributes that are cheap to read come first) ----
    def _use(self, stream):
        """The cache's memory is in use on another stream than before: none of it is given to anyone else before that stream is done."""
        self._streams.add(stream)
        now = self.torch.cuda.current_stream(self._idx)
        for t in (self.k, self.v, self.table, self.held, self.free, self.queue, self.err, self._scratch, *self._kept):
            if t is not None:
                t.record_stream(now)

    def _call(self, f, what, *args):
        idx = self._idx
        stream = self._stream(idx)
        if stream not in self._streams:
            self._use(stream)
        if self._current_device() != idx:
            with self.torch.cuda.device(idx):
                rc = f(self._c, *args, stream)
        else:
            rc = f(self._c, *args, stream)
        if rc != DFL_OK:
            raise DflError(rc, what)

    def _ints(self, t, name, count):
        if t is None or t.dtype is not self._i32 or t.get_device() != self._idx or t.dim() != 1 or (count and t.numel() != count) or not t.is_contiguous():
            _refuse(f"{name} must be int32 [{count or 'rows'}] on {self.device}")
        return t.data_ptr()

    def _rows(self, t, name, heads):
        """A tensor of packed rows [rows][heads][head_dim]: (pointer, rows, distance of rows in elements)."""
        if t.dtype is self.dtype and t.get_device() == self._idx and t.dim() == 3:
            n, H, hd = t.shape
            if hd == self.head_dim and (H == heads or not heads):
                if t.is_contiguous():
                    return t.data_ptr(), n, H * hd
                s0, s1, s2 = t.stride()
                if s2 == 1 and (H == 1 or s1 == hd):
                    return t.data_ptr(), n, s0 if n > 1 else H * hd
        _refuse(f"{name} must be {self.dtype} [rows][{heads or 'heads'}][{self.head_dim}] on {self.device}, heads and channels contiguous")

    # ---- the calls ----
    def plan(self, length, n, rows=None, out=None):
        """dfl_paged_plan: the pages that sequences of length + n tokens need (int32 [n_seq] each). Returns (cu, slots), int32 [n_seq + 1] and
        [rows]; `out`: the two tensors to write."""
        if out is None:
            if rows is None or rows < 1:
                _refuse("plan needs the rows of the step's buffers, or out")
            out = self.torch.empty(self.n_seq + 1, dtype=self._i32, device=self.device), self.torch.empty(rows, dtype=self._i32, device=self.device)
        cu, slots = out
        if rows is not None and slots.numel() != rows or slots.numel() > MOST:
            _refuse(f"slots must be int32 [{'rows' if rows is None else rows}] on {self.device}, rows below 2^31")
        self._call(self.L.dfl_paged_plan, "dfl_paged_plan", self._ints(length, "length", self.n_seq), self._ints(n, "n", self.n_seq),
                   self._ints(cu, "cu", self.n_seq + 1), self._ints(slots, "slots", 0), slots.numel())
        return out

    def append(self, k, v, slots):
        """dfl_paged_append: rows k, v [rows][n_kv][head_dim] into the places of slots (int32 [rows]; rows of negative ones are left out)."""
        pk, n, ldk = self._rows(k, "k", self.n_kv)
        pv, nv, ldv = self._rows(v, "v", self.n_kv)
        if nv != n:
            _refuse("k and v must have the same rows")
        self._call(self.L.dfl_paged_append, "dfl_paged_append", self._ints(slots, "slots", n), n, pk, ldk, pv, ldv)

    def prompt(self, q, k, v, cu, window: int = 0, scale=None, out=None):
        """dfl_paged_prompt: causal attention of packed prompts among their own rows, q [rows][n_q][head_dim], k and v [rows][n_kv][head_dim];
        scale defaults to head_dim ** -0.5. Returns `out` (allocated when None, rows behind the last sequence's then zero)."""
        pq, n, ldq = self._rows(q, "q", 0)
        pk, nk, ldk = self._rows(k, "k", self.n_kv)
        pv, nv, ldv = self._rows(v, "v", self.n_kv)
        n_q = q.shape[1]
        if out is None:
            out = self.torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        po, no, ldo = self._rows(out, "out", n_q)
        if nk != n or nv != n or no != n or not 0 <= window <= MOST:
            _refuse("q, k, v and out must have the same rows, and window be 0 to 2^31 - 1")
        self._call(self.L.dfl_paged_prompt, "dfl_paged_prompt", pq, ldq, n_q, pk, ldk, pv, ldv, self._ints(cu, "cu", self.n_seq + 1), n, window,
                   self._scale if scale is None else scale, po, ldo)
        return out

    def attn(self, q, cu, length, rows: int, window: int = 0, causal: bool = True, scale=None, out=None):
        """dfl_paged_attn: attention over the pages of at most `rows` rows a sequence, q [total][n_q][head_dim] packed by cu, the first of them
        at position length. Returns `out` (allocated when None, rows behind the last sequence's then zero)."""
        pq, n, ldq = self._rows(q, "q", 0)
        n_q = q.shape[1]
        need = self._need.get((n_q, rows))
        if need is None:
            need = int(self.L.dfl_paged_attn_scratch_bytes(self._c, n_q, rows)) if 0 < rows <= MOST else -1
            if need < 0:
                _refuse(f"{n_q} query heads and {rows} rows: n_q must be a multiple of n_kv = {self.n_kv}, up to 16 a head, with 1..16 rows")
            if self._scratch_bytes < need:
                scratch = self.torch.empty(need, dtype=self.torch.uint8, device=self.device)
                self._kept.append(self._scratch)       # a captured graph may hold its address
                self._scratch, self._scratch_ptr, self._scratch_bytes = scratch, scratch.data_ptr(), need
                self._streams.clear()
            self._need[(n_q, rows)] = need
        if out is None:
            out = self.torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        po, no, ldo = self._rows(out, "out", n_q)
        if no != n or not 0 <= window <= MOST:
            _refuse("out must have q's rows, and window be 0 to 2^31 - 1")
        self._call(self.L.dfl_paged_attn, "dfl_paged_attn", pq, ldq, n_q, n, self._ints(cu, "cu", self.n_seq + 1), self._ints(length, "length", self.n_seq),
                   rows, window, causal, self._scale if scale is None else scale, po, ldo, self._scratch_ptr, self._scratch_bytes)
        return out

    def status(self):
        """Synchronise the current stream and raise what the calls so far met on the device."""
        self._call(self.L.dfl_paged_status, "dfl_paged_status")
