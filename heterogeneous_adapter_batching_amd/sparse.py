"""Sparse attention over a paged cache: every new token sees the pages that a
cheap score chooses for it.

``KvBounds`` describes the bounds of a cache's pages (lora_kv_bounds_t);
``SparseBatch`` is an ``AttnBatch`` whose plan also serves the sparse layers of a
model: after ``write``, ``bounds`` summarises the pages that the batch has
completed, ``select`` chooses the pages of each new token and kv head, and
``sparse`` attends over them.  ``write``, ``read`` and ``attn`` work as in
AttnBatch, for the layers whose attention is not sparse.
"""
import ctypes

import torch

from . import (LORA_OK, _lib, as_int32, check_status, lora_kv_bounds_t, lora_sparse_launch_t, lora_sparse_shape_t)
from .attention import AttnBatch
from .pages import check_device


class KvBounds:
    """Bounds of the keys of a cache's pages: codes int8 [n_pages, n_kv_heads, 2,
    head_dim] (each element's largest key, then its smallest) and exps uint8
    [n_pages, n_kv_heads] (exponents biased by 127), contiguous, on the cache's
    device."""

    def __init__(self, cache, codes, exps):
        want = (cache.n_pages, cache.n_kv_heads, 2, cache.head_dim)
        if codes.dtype != torch.int8 or tuple(codes.shape) != want or not codes.is_contiguous():
            raise ValueError(f"codes: contiguous int8 {list(want)}")
        if exps.dtype != torch.uint8 or tuple(exps.shape) != want[:2] or not exps.is_contiguous():
            raise ValueError(f"exps: contiguous uint8 {list(want[:2])}")
        if codes.device != cache.k.device or exps.device != cache.k.device:
            raise ValueError("the bounds are not on the cache's device")
        self.codes, self.exps = codes, exps
        self._c = lora_kv_bounds_t(codes.data_ptr(), exps.data_ptr(), *want[:2], want[3], 0)

    @classmethod
    def empty(cls, cache):
        """Bounds of their own memory; no page has any yet."""
        shape = (cache.n_pages, cache.n_kv_heads, 2, cache.head_dim)
        return cls(cache, torch.zeros(shape, dtype=torch.int8, device=cache.k.device),
                   torch.full(shape[:2], 127, dtype=torch.uint8, device=cache.k.device))

    def shape(self):
        """(n_pages, n_kv_heads, head_dim)."""
        return self._c.n_pages, self._c.n_kv_heads, self._c.head_dim

    def c(self):
        return self._c


class SparseBatch(AttnBatch):
    """An AttnBatch whose new tokens may also see ``select`` pages only: the
    ``first`` pages of their sequence, the ``last`` ones up to their own, and of
    those between the ones of the highest scores.  Pages hold 16 tokens at least.
    One plan serves every layer, sparse or not.  The calls share the batch's one
    workspace: on one batch they must be ordered (one stream, or events)."""

    def __init__(self, cache, n_heads, select, first=1, last=1):
        super().__init__(cache, n_heads)
        n = [int(as_int32(x, name)[0]) for x, name in ((select, "select"), (first, "first"), (last, "last"))]
        self.sparse_shape = lora_sparse_shape_t(*n, 0)
        if n[1] < 0 or n[2] < 1 or n[0] < n[1] + n[2]:
            raise ValueError("select >= first + last, first >= 0, last >= 1")
        self._sparse = lora_sparse_launch_t()
        self._launch = self._sparse.attn
        self._ref, self._sparse_ref = ctypes.byref(self._launch), ctypes.byref(self._sparse)
        self._bounded = None

    def refresh(self, q_len, kv_len, block_table, stream=None, bounded=None):
        """As AttnBatch.refresh.  bounded: int [n_seq], tokens of each sequence
        whose complete pages have bounds (0 for one that has come back into the
        cache); None: those before the new tokens."""
        self._bounded = None if bounded is None else as_int32(bounded, "bounded")
        if self._bounded is not None and self._bounded.shape != as_int32(q_len, "q_len").shape:
            raise ValueError("bounded [n_seq]")
        return super().refresh(q_len, kv_len, block_table, stream)

    def _use(self, stream):
        s = super()._use(stream)
        check_device(self.device, s.cuda_stream)
        return s

    def _prepare(self, ql, kl, tab, staging, capacity, dev, h):
        return _lib.lora_sparse_prepare(ctypes.byref(self.shape), ctypes.byref(self.sparse_shape), ql.shape[0],
                                        ql.ctypes.data, kl.ctypes.data,
                                        None if self._bounded is None else self._bounded.ctypes.data,
                                        None if tab is None else tab.ctypes.data, 0 if tab is None else tab.shape[1],
                                        staging, capacity, dev, h, self._sparse_ref)

    @property
    def sparse_info(self):
        return self._sparse.info

    def _check_bounds(self, bounds):
        s = self.shape
        if bounds.shape() != (s.n_pages, s.n_kv_heads, s.head_dim):
            raise ValueError("the bounds are of a cache of another shape than the plan's")
        if bounds.codes.device != self.device:
            raise ValueError(f"the bounds are not on {self.device}")
        return ctypes.byref(bounds.c())

    def _selected(self, t):
        want = (self.shape.n_kv_heads, self.sparse_shape.select)
        if t.dim() != 3 or tuple(t.shape[1:]) != want or t.dtype != torch.int32 or not t.is_contiguous() or \
                t.device != self.device:
            raise ValueError(f"selected: contiguous int32 [rows, {want[0]}, {want[1]}] on {self.device}")
        return int(t.shape[0])

    def empty_selected(self, rows=None):
        """A tensor for the pages selected of ``rows`` rows (the plan's)."""
        rows = self.info.n_rows if rows is None else int(rows)
        return torch.empty(rows, self.shape.n_kv_heads, self.sparse_shape.select, dtype=torch.int32, device=self.device)

    def prepare_bounds(self, bounds, cache=None, stream=None):
        """Returns fn() that summarises the complete pages which hold tokens of
        the batch from `bounded` on: after the write, before select."""
        cache = self._check_cache(cache)
        b_ref, kv_ref, h = self._check_bounds(bounds), ctypes.byref(cache.c()), self._use(stream).cuda_stream
        ref, call = self._sparse_ref, _lib.lora_kv_bounds

        def run():
            self._need(0, 0, "")
            st = call(ref, kv_ref, b_ref, h)
            if st != LORA_OK:
                check_status(st, "lora_kv_bounds")
        run.keep = (cache, bounds)
        return run

    def prepare_select(self, q, bounds, selected, stream=None):
        """q: bf16 [rows, n_heads * head_dim]; selected: int32 [rows, n_kv_heads,
        select], takes page ids in the sequence's order, -1 behind them.  Returns
        fn() that chooses the pages of the batch's rows."""
        b_ref = self._check_bounds(bounds)
        rows = min(self._rows(q, self.n_heads, torch.bfloat16, "q"), self._selected(selected))
        h, L, ref = self._use(stream).cuda_stream, self._launch, self._sparse_ref
        qp, ldq, sp, call = q.data_ptr(), q.stride(0), selected.data_ptr(), _lib.lora_sparse_select

        def run():
            self._need(rows, L.info.n_rows, "q or selected")
            ws = self._workspace
            st = call(ref, b_ref, qp, ldq, sp, ws.data_ptr(), ws.shape[0], h)
            if st != LORA_OK:
                check_status(st, "lora_sparse_select")
        run.keep = (q, bounds, selected)
        return run

    def prepare_sparse(self, q, out, scale, selected, cache=None, stream=None):
        """q, out: bf16 [rows, n_heads * head_dim]; selected: from select on this
        plan, for this layer or another one.  Returns fn() that runs the batch's
        attention over the pages selected."""
        cache = self._check_cache(cache)
        rows = min(self._rows(q, self.n_heads, torch.bfloat16, "q"),
                   self._rows(out, self.n_heads, torch.bfloat16, "out"), self._selected(selected))
        h, L, ref, kv_ref = self._use(stream).cuda_stream, self._launch, self._sparse_ref, ctypes.byref(cache.c())
        qp, ldq, sp, op, ldo = q.data_ptr(), q.stride(0), selected.data_ptr(), out.data_ptr(), out.stride(0)
        scale, call = float(scale), _lib.lora_sparse_attn

        def run():
            self._need(rows, L.info.n_rows, "q, out or selected")
            ws = self._workspace
            st = call(ref, kv_ref, qp, ldq, sp, op, ldo, scale, ws.data_ptr(), ws.shape[0], h)
            if st != LORA_OK:
                check_status(st, "lora_sparse_attn")
        run.keep = (q, out, selected, cache)
        return run

    def bounds(self, bounds, cache=None, stream=None):
        self.prepare_bounds(bounds, cache, stream)()

    def select(self, q, bounds, selected, stream=None):
        self.prepare_select(q, bounds, selected, stream)()

    def sparse(self, q, out, scale, selected, cache=None, stream=None):
        self.prepare_sparse(q, out, scale, selected, cache, stream)()
