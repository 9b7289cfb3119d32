"""A key/value cache in 8 bits over torch tensors: the dfl_kv8_* calls of include/dfl.h with their
arguments checked and marshalled. Nothing here computes: every call is one of the library's.

A step of speculative decode over it, lengths staying on the device (`length`: int32 [n_seq], the
committed tokens, shared by a model's layers):

    cache.append(k, v, length); length += rows      # a prompt's rows (committed)
    cache.stage(k, v, length)                       # a verify's rows (may be rolled back)
    out = cache.attn(q, length, score=True)
    length += kept                                  # commit the accepted rows; the others are overwritten
    length = cache.evict(length, keep=256)          # now and then: thin the cache
"""
from __future__ import annotations

import ctypes

from . import _abi
from ._abi import DFL_E_INVALID_ARG, DFL_OK, DflError, dfl_kv8

BLOCK, TAIL = 32, 48          # DFL_KV8_BLOCK, DFL_KV8_TAIL


def _refuse(msg: str):
    raise DflError(DFL_E_INVALID_ARG, msg)


class Kv8Cache:
    """A dfl_kv8 over the caller's tensors (layouts in include/dfl.h), or `empty(...)` to allocate them.

    Calls enqueue on the device's current stream and return without synchronising; `status()` synchronises
    and raises what a call met on the device (a capacity passed, a state or table out of order). The
    attention's scratch belongs to the object: calls of one cache must not overlap on the GPU. It grows with
    the largest call so far, and no piece of it is ever freed before the object, so captured graphs stay
    valid.
    """

    def __init__(self, k, v, k_scale, v_scale, k_tail, v_tail, table, sealed, score=None):
        import torch
        self.torch = torch
        if k.dim() != 6 or k.shape[4:] != (BLOCK, 64):
            _refuse("k must be uint8 [n_seq][n_kv][n_blocks][head_dim/64][32][64]")
        S, H, B = k.shape[:3]
        hd = k.shape[3] * 64
        u8, f32, i32 = torch.uint8, torch.float32, torch.int32
        want = {"k": (k, u8, (S, H, B, hd // 64, BLOCK, 64)), "v": (v, u8, (S, H, B, hd, BLOCK)),
                "k_scale": (k_scale, f32, (S, H, B)), "v_scale": (v_scale, f32, (S, H, B)),
                "k_tail": (k_tail, f32, (S, H, TAIL, hd)), "v_tail": (v_tail, f32, (S, H, hd, TAIL)),
                "table": (table, i32, (S, H, B)), "sealed": (sealed, i32, (S, H)), "score": (score, f32, (S, H, B))}
        for name, (t, dtype, shape) in want.items():
            if t is None and name == "score":
                continue
            if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != k.device:
                _refuse(f"{name} must be contiguous {dtype} {list(shape)} on {k.device}")
        self.n_seq, self.n_kv, self.n_blocks, self.head_dim = S, H, B, hd
        self.device = k.device
        if self.device.type != "cuda":
            _refuse("the cache's tensors must be on a CUDA device")
        self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail = k, v, k_scale, v_scale, k_tail, v_tail
        self.err = torch.zeros(64, dtype=i32, device=self.device)
        self.L = _abi.lib()
        self._idx, self._f32, self._i32 = self.device.index, f32, i32
        self._current_device, self._stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self._streams = set()         # that calls have used since the tensors were last recorded with them
        self._evicted = self._scratch = None
        self._take(table, sealed, score)
        self._scale = self.head_dim ** -0.5
        self._kept, self._scratch_ptr, self._scratch_bytes = [], 0, 0
        self._need = {}

    def _take(self, table, sealed, score):
        self.table, self.sealed, self.score = table, sealed, score
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self.c = dfl_kv8(self.n_seq, self.n_kv, self.head_dim, self.n_blocks, p(self.k), p(self.v), p(self.k_scale), p(self.v_scale),
                         p(self.k_tail), p(self.v_tail), p(table), p(sealed), p(score), p(self.err))
        self._c = ctypes.byref(self.c)
        self._streams.clear()

    def _use(self, stream):
        """The cache's memory is in use on another stream than before: none of it is given to anyone else before that stream is done."""
        self._streams.add(stream)
        now = self.torch.cuda.current_stream(self._idx)
        for t in (self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail, self.table, self.sealed, self.score, self.err, self._scratch, *self._kept,
                  *(self._evicted or {}).values()):
            if t is not None:
                t.record_stream(now)

    @classmethod
    def empty(cls, n_seq: int, n_kv: int, head_dim: int, n_blocks: int, device="cuda:0", score: bool = True) -> "Kv8Cache":
        """An empty cache of 32 * n_blocks tokens a sequence."""
        import torch
        if head_dim not in (64, 128, 256) or min(n_seq, n_kv, n_blocks) < 1:
            _refuse("head_dim must be 64, 128 or 256 and the sizes positive")
        mk = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        u8, f32, i32 = torch.uint8, torch.float32, torch.int32
        lead = (n_seq, n_kv, n_blocks)
        self = cls(mk(u8, *lead, head_dim // 64, BLOCK, 64), mk(u8, *lead, head_dim, BLOCK), mk(f32, *lead), mk(f32, *lead),
                   mk(f32, n_seq, n_kv, TAIL, head_dim), mk(f32, n_seq, n_kv, head_dim, TAIL), mk(i32, *lead), mk(i32, n_seq, n_kv),
                   mk(f32, *lead) if score else None)
        self._call(self.L.dfl_kv8_init, "dfl_kv8_init")
        return self

    # ---- marshalling (a short call's time is mostly the host's: attributes that are cheap to read come first) ----
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

    def _ints(self, t, name, optional=False):
        if t is None and optional:
            return None
        if t is None or t.dtype is not self._i32 or t.get_device() != self._idx or t.dim() != 1 or t.numel() != self.n_seq or not t.is_contiguous():
            _refuse(f"{name} must be int32 [{self.n_seq}] on {self.device}")
        return t.data_ptr()

    def _rows(self, t, name, heads):
        """A row tensor fp32 [n_seq][rows][heads][head_dim] whose rows lie a fixed distance apart: (pointer, rows, distance in floats)."""
        if t.dtype is self._f32 and t.get_device() == self._idx and t.dim() == 4:
            S, M, H, hd = t.shape
            if S == self.n_seq and hd == self.head_dim and (H == heads or not heads):
                if t.is_contiguous():
                    return t.data_ptr(), M, H * hd
                s0, s1, s2, s3 = t.stride()
                ld = s1 if M > 1 else s0 if S > 1 else H * hd
                if s3 == 1 and (H == 1 or s2 == hd) and (S == 1 or s0 == M * ld):
                    return t.data_ptr(), M, ld
        _refuse(f"{name} must be fp32 [{self.n_seq}][rows][{heads or 'heads'}][{self.head_dim}] on {self.device}, heads and channels contiguous "
                "and the rows of all sequences one fixed distance apart")

    def _write(self, f, what, k, v, length, n):
        pk, M, ld = self._rows(k, "k", self.n_kv)
        pv, Mv, ldv = self._rows(v, "v", self.n_kv)
        if Mv != M or ldv != ld:
            _refuse("k and v must have the same rows and strides")
        self._call(f, what, self._ints(length, "length"), self._ints(n, "n", True), M, pk, pv, ld)

    # ---- the calls ----
    def append(self, k, v, length, n=None):
        """dfl_kv8_append: rows k, v (fp32 [n_seq][rows][n_kv][head_dim]; n: int32 [n_seq], the rows that count) become committed
        tokens length .. length + n - 1. The caller adds n to length."""
        self._write(self.L.dfl_kv8_append, "dfl_kv8_append", k, v, length, n)

    def stage(self, k, v, length, n=None):
        """dfl_kv8_stage: at most 16 rows that may still be rolled back, behind the committed tokens."""
        self._write(self.L.dfl_kv8_stage, "dfl_kv8_stage", k, v, length, n)

    def attn(self, q, length, n=None, window: int = 0, causal: bool = True, scale=None, score: bool = False, out=None):
        """dfl_kv8_attn: attention of the staged rows, q fp32 [n_seq][rows][n_q][head_dim]; scale defaults to head_dim ** -0.5. Returns
        `out` (allocated when None, rows behind n then zero), which overlaps none of the inputs."""
        pq, M, ldq = self._rows(q, "q", 0)
        n_q = q.shape[2]
        pl, pn = self._ints(length, "length"), self._ints(n, "n", True)
        key = (n_q, M, window, score)
        need = self._need.get(key)
        if need is None:
            need = int(self.L.dfl_kv8_attn_scratch_bytes(self._c, n_q, M, window, score))
            if need < 0:
                _refuse(f"{n_q} query heads and {M} rows: n_q must be a multiple of n_kv = {self.n_kv}, up to 16 a head, with 1..16 rows and a window >= 0")
            if self._scratch_bytes < need:
                scratch = self.torch.empty(need, dtype=self.torch.uint8, device=self.device)
                self._kept.append(self._scratch)       # a captured graph may hold its address
                self._scratch, self._scratch_ptr, self._scratch_bytes = scratch, scratch.data_ptr(), need
                self._streams.clear()
            self._need[key] = need
        if out is None:
            out = (self.torch.empty if n is None else self.torch.zeros)(q.shape, dtype=q.dtype, device=q.device)
        po, Mo, ldo = self._rows(out, "out", n_q)
        if Mo != M:
            _refuse("out must have q's rows")
        self._call(self.L.dfl_kv8_attn, "dfl_kv8_attn", pq, ldq, n_q, M, pl, pn, window, causal, self._scale if scale is None else scale,
                   score, po, ldo, self._scratch_ptr, self._scratch_bytes)
        return out

    def evict(self, length, keep: int, sink: int = 0, recent: int = 0, out=None):
        """dfl_kv8_evict: keep at most `keep` sealed blocks a head. Without `out` the result replaces the cache's table, scores and sealed
        counts where they lie (a captured graph that uses them stays valid) and the new length is returned; with `out` (a dict of tensors
        "table", "score", "sealed" and "len") it is written there, the cache keeps its own, and `take(out)` changes over."""
        pl = self._ints(length, "length")
        if self.score is None:
            _refuse("the cache keeps no scores")
        new = out
        if new is None:
            if self._evicted is None:
                self._evicted = {name: self.torch.empty_like(getattr(self, name)) for name in ("table", "score", "sealed")}
                self._streams.clear()
            new = dict(self._evicted, len=self.torch.empty_like(length))
        else:
            self._check_out(new)
        self._call(self.L.dfl_kv8_evict, "dfl_kv8_evict", pl, keep, sink, recent, new["table"].data_ptr(), new["score"].data_ptr(),
                   new["sealed"].data_ptr(), self._ints(new["len"], "len"))
        if out is None:
            for name in ("table", "score", "sealed"):
                getattr(self, name).copy_(new[name])
            return new["len"]
        return out

    def _check_out(self, new):
        for name, like in (("table", self.table), ("score", self.score), ("sealed", self.sealed)):
            t = new[name]
            if t.dtype is not like.dtype or t.shape != like.shape or not t.is_contiguous() or t.get_device() != self._idx:
                _refuse(f"{name} must be contiguous {like.dtype} {list(like.shape)} on {self.device}")

    def take(self, new):
        """Go on with an eviction's result (`evict(..., out=new)`) in the tensors given; returns its length. Graphs captured before go on
        with the tensors that the cache had then."""
        self._check_out(new)
        self._take(new["table"], new["sealed"], new["score"])
        return new["len"]

    def read(self, length, rows: int, first=None, out=None):
        """dfl_kv8_read: tokens first .. first + rows - 1 below length, as fp32 (keys, values) [n_seq][rows][n_kv][head_dim]."""
        shape = (self.n_seq, rows, self.n_kv, self.head_dim)
        if out is None:
            out = [self.torch.zeros(shape, dtype=self.torch.float32, device=self.device) for _ in range(2)]
        for t in out:
            if t.dtype is not self._f32 or t.shape != shape or not t.is_contiguous() or t.get_device() != self._idx:
                _refuse(f"out must be two contiguous fp32 tensors {list(shape)} on {self.device}")
        self._call(self.L.dfl_kv8_read, "dfl_kv8_read", self._ints(length, "length"), self._ints(first, "first", True), rows,
                   out[0].data_ptr(), out[1].data_ptr())
        return out

    def status(self):
        """Synchronise the current stream and raise what the calls so far met on the device."""
        self._call(self.L.dfl_kv8_status, "dfl_kv8_status")
