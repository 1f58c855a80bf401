"""The pages of a paged cache: who holds which, and their copies.

``KvPages`` is the library's host-side manager (lora_kv_pages_*): it hands out
pages to sequences, shares them between forks, takes them back and compacts
them, and says what has to be copied for it.  ``KvCopy`` copies pages of one or
more caches (lora_kv_copy), the layers of a model in one call.  The lists that
the manager gives go to the copy as they are:

    copies = pages.append(seqs, tokens)      # room for new tokens
    copy.copy(*copies)                       # before the new tokens are written
    batch.refresh(tokens, *pages.table(seqs)[::-1])
"""
import ctypes

import numpy as np
import torch

from . import (LORA_ECAPACITY, LORA_OK, _i32, _lib, _vp, as_int32, check_status, lora_kv_bounds_t, lora_kv_t)


def _list(x, name):
    a = as_int32(x, name)
    if a.ndim != 1:
        raise ValueError(f"{name}: one number for each")
    return a


def _one(x, name):
    a = as_int32(x, name)
    if a.size != 1:
        raise ValueError(f"{name}: one number")
    return int(a.reshape(-1)[0])


def check_device(device, handle):
    """A launch on the default stream goes to the current device."""
    if handle == 0 and torch.cuda.is_initialized() and torch.cuda.current_device() != device.index:
        raise ValueError(f"{device} is not the current device, whose default stream this is: make it current, or give "
                         "a stream of it")


class KvPages:
    """Pages 0 .. n_pages-1 of ``page_tokens`` tokens, and the sequences 0 ..
    n_seqs-1 that hold them.  One manager serves all layers' caches.  Serves one
    thread at a time; raises LoraError (LORA_ECAPACITY where pages are short) and
    then has changed nothing."""

    def __init__(self, n_pages, page_tokens, n_seqs):
        n = [_one(n_pages, "n_pages"), _one(page_tokens, "page_tokens"), _one(n_seqs, "n_seqs")]
        self._h = None
        self.n_pages, self.page_tokens, self.n_seqs = n
        h = _vp()
        check_status(_lib.lora_kv_pages_create(*n, ctypes.byref(h)), "lora_kv_pages_create")
        self._h = h

    def __del__(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.lora_kv_pages_destroy(self._h)
            self._h = None

    def append(self, seqs, tokens):
        """Room for tokens[i] more tokens of each sequence.  Returns the copies
        (src, dst, tokens) that have to come before these are written."""
        s, t = _list(seqs, "seqs"), _list(tokens, "tokens")
        if s.shape != t.shape:
            raise ValueError("seqs and tokens have different lengths")
        out, n = np.empty((3, max(1, s.shape[0])), np.int32), _i32(0)
        check_status(_lib.lora_kv_pages_append(self._h, s.shape[0], s.ctypes.data, t.ctypes.data,
                                               *(x.ctypes.data for x in out), ctypes.byref(n)), "lora_kv_pages_append")
        return tuple(out[:, :n.value])

    def fork(self, parent, children):
        """The children, sequences that hold no tokens, get the parent's."""
        c = _list(children, "children")
        check_status(_lib.lora_kv_pages_fork(self._h, _one(parent, "parent"), c.shape[0], c.ctypes.data),
                     "lora_kv_pages_fork")

    def truncate(self, seq, tokens):
        """The sequence keeps its first ``tokens`` tokens."""
        check_status(_lib.lora_kv_pages_truncate(self._h, _one(seq, "seq"), _one(tokens, "tokens")),
                     "lora_kv_pages_truncate")

    def free(self, seqs):
        """The sequences hold no tokens any more."""
        s = _list(seqs, "seqs")
        check_status(_lib.lora_kv_pages_free(self._h, s.shape[0], s.ctypes.data), "lora_kv_pages_free")

    def compact(self):
        """The pages in use become the first ones.  Returns the moves (src, dst,
        tokens) to copy; tables taken before no longer hold."""
        n = _i32(0)
        st = _lib.lora_kv_pages_compact(self._h, 0, None, None, None, ctypes.byref(n))
        out = np.empty((3, max(1, n.value)), np.int32)
        if st == LORA_ECAPACITY:
            st = _lib.lora_kv_pages_compact(self._h, n.value, *(x.ctypes.data for x in out), ctypes.byref(n))
        check_status(st, "lora_kv_pages_compact")
        return tuple(out[:, :n.value])

    def table(self, seqs):
        """(table int32 [n, pages], kv_len int32 [n]) of the sequences, as
        AttnBatch.refresh takes them."""
        s = _list(seqs, "seqs")
        cols = _i32(0)
        kv_len = np.empty(s.shape[0], np.int32)
        st = _lib.lora_kv_pages_table(self._h, s.shape[0], s.ctypes.data, 0, None, kv_len.ctypes.data, ctypes.byref(cols))
        table = np.zeros((s.shape[0], cols.value), np.int32)
        if st == LORA_ECAPACITY:
            st = _lib.lora_kv_pages_table(self._h, s.shape[0], s.ctypes.data, cols.value, table.ctypes.data,
                                          kv_len.ctypes.data, ctypes.byref(cols))
        check_status(st, "lora_kv_pages_table")
        return table, kv_len

    def stats(self):
        """(free pages, pages that several sequences hold, one more than the last page in use)."""
        n = [_i32(0) for _ in range(3)]
        check_status(_lib.lora_kv_pages_stats(self._h, *(ctypes.byref(x) for x in n)), "lora_kv_pages_stats")
        return tuple(x.value for x in n)


class KvCopy:
    """Copies of pages within each of ``caches``, or from them to ``to``.
    ``bounds`` (and ``to_bounds``): KvBounds of each cache, which go with whole
    pages."""

    def __init__(self, caches, bounds=None, to=None, to_bounds=None):
        caches = list(caches)
        if not caches:
            raise ValueError("no caches")
        if to is None and to_bounds is not None:
            raise ValueError("to_bounds without to")
        if to is not None and (bounds is None) != (to_bounds is None):
            raise ValueError("bounds and to_bounds go together")
        self.device = caches[0].k.device
        if self.device.type != "cuda":
            raise ValueError("the caches are not on the GPU")
        lists = [None if x is None else list(x) for x in (bounds, to, to_bounds)]
        for x in lists:
            if x is not None and len(x) != len(caches):
                raise ValueError("one of each to a cache")
        if any(c.k.device != self.device for c in caches + (lists[1] or [])) or \
                any(b.codes.device != self.device for b in (lists[0] or []) + (lists[2] or [])):
            raise ValueError(f"a cache or bounds are not on {self.device}")
        for of, b in ((caches, lists[0]), (lists[1], lists[2])):
            if b is not None and any(x.shape() != (c.n_pages, c.n_kv_heads, c.head_dim) for x, c in zip(b, of)):
                raise ValueError("bounds of a cache of another shape")
        self._keep = (caches, *lists)

        def array(kind, xs):
            return None if xs is None else (kind * len(xs))(*(x.c() for x in xs))
        self._n = len(caches)
        self._args = (array(lora_kv_t, caches), array(lora_kv_t, lists[1]), array(lora_kv_bounds_t, lists[0]),
                      array(lora_kv_bounds_t, lists[2]))

    def prepare_copy(self, src, dst, tokens=None, stream=None):
        """src, dst: page ids (host); tokens: how many of each page, or None for
        whole pages.  Returns fn() that issues the copies."""
        s, d = _list(src, "src"), _list(dst, "dst")
        t = None if tokens is None else _list(tokens, "tokens")
        if s.shape != d.shape or (t is not None and t.shape != s.shape):
            raise ValueError("src, dst and tokens have different lengths")
        s, d, t = s.copy(), d.copy(), None if t is None else t.copy()
        h = (torch.cuda.current_stream(self.device) if stream is None else stream).cuda_stream
        check_device(self.device, h)
        args = (self._n, *self._args, s.shape[0], s.ctypes.data, d.ctypes.data, None if t is None else t.ctypes.data, h)
        call = _lib.lora_kv_copy

        def run():
            st = call(*args)
            if st != LORA_OK:
                check_status(st, "lora_kv_copy")
        run.keep = (self, s, d, t)
        return run

    def copy(self, src, dst, tokens=None, stream=None):
        self.prepare_copy(src, dst, tokens, stream)()
