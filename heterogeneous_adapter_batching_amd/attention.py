"""A layer's paged cache and the attention of a batch over it.

``KvCache`` describes the cache's tensors; ``AttnBatch`` plans a batch on the
host (lora_attn_plan), uploads the plan in one pinned host->device copy on the
caller's stream, and runs the three calls on it: the new tokens' write, the
attention of their queries, and the read of whole sequences.  As in session.py,
``prepare_*`` check their tensors, build the C argument structs once and return
a callable that only issues the library call; PyTorch only provides memory and
streams.
"""
import collections
import ctypes
import sys

import numpy as np
import torch

from . import (LORA_BF16, LORA_ECAPACITY, LORA_F32, LORA_KV_BF16, LORA_KV_E4M3, LORA_OK, _lib, as_int32, check_status,
               lora_attn_launch_t, lora_attn_shape_t, lora_kv_t, lora_kv_write_args_t)
from .session import HipEvent

# staging buffers of batches let go, with the event of the copy that may be reading each
_held = collections.deque()


def _release():
    """Lets the staging buffers go whose copies have ended."""
    for _ in range(len(_held)):
        try:
            held = _held.popleft()
        except IndexError:  # another thread's
            return
        if not held[1].query():
            _held.append(held)


class KvCache:
    """The paged cache of one layer: k and v [n_pages, n_kv_heads, page_tokens,
    head_dim] on the device, bf16 or float8_e4m3fn, of the same strides (any
    order of pages, heads and tokens; a head's elements contiguous).  An e4m3
    cache has k_scale and v_scale, uint8 [n_pages, n_kv_heads, page_tokens]:
    exponents biased by 127."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v: [n_pages, n_kv_heads, page_tokens, head_dim] of one type and one layout")
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise ValueError("the cache is bfloat16 or float8_e4m3fn")
        if k.stride(3) != 1:
            raise ValueError("a head's elements must be contiguous")
        quantised = k.dtype == torch.float8_e4m3fn
        for s in (k_scale, v_scale):
            if quantised != (s is not None):
                raise ValueError("k_scale and v_scale belong to an e4m3 cache, and to no other")
            if s is not None and (s.dtype != torch.uint8 or s.shape != k.shape[:3] or not s.is_contiguous()):
                raise ValueError("scales: contiguous uint8 [n_pages, n_kv_heads, page_tokens]")
        if any(t is not None and t.device != k.device for t in (v, k_scale, v_scale)):
            raise ValueError("the cache's tensors are on different devices")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_tokens, self.head_dim = (int(x) for x in k.shape)
        self.dtype = LORA_KV_E4M3 if quantised else LORA_KV_BF16
        self._c = lora_kv_t(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if quantised else None,
                            v_scale.data_ptr() if quantised else None, self.dtype, self.n_pages, self.page_tokens,
                            self.n_kv_heads, self.head_dim, 0, *k.stride()[:3])

    @classmethod
    def empty(cls, n_pages, n_kv_heads, page_tokens, head_dim, dtype=torch.bfloat16, device="cuda"):
        """A cache of its own memory; its contents are unspecified."""
        shape = (n_pages, n_kv_heads, page_tokens, head_dim)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v)
        return cls(k, v, *(torch.full(shape[:3], 127, dtype=torch.uint8, device=device) for _ in range(2)))

    def c(self):
        return self._c


def rope_table(n_positions, rope_dim, base=10000.0, device="cuda"):
    """fp32 [n_positions, rope_dim]: cosines, then sines, of position *
    base^(-2 i / rope_dim); the angles are computed in 64 bits."""
    half = rope_dim // 2
    turn = np.arange(n_positions, dtype=np.float64)[:, None] * base ** (-np.arange(half, dtype=np.float64) / half)
    return torch.from_numpy(np.concatenate([np.cos(turn), np.sin(turn)], 1).astype(np.float32)).to(device)


class AttnBatch:
    """The plan of one batch over caches of one shape, resident on the device.

    ``refresh(q_len, kv_len, block_table)`` plans a new batch with one library
    call (lora_attn_prepare), reusing the host and device buffers, which grow
    when a batch needs more; callables from ``prepare_*`` stay valid, with
    tensors that have rows enough for the new batch (a captured graph holds the
    buffers of its own time, and has to be captured again once they have grown).
    The buffers belong to the stream of the refresh that made them: work on the
    batch from other streams has to be ordered after it by events.  One plan serves every
    layer whose cache has the same shape, mask and type: the calls take another
    ``cache`` than the one the batch was made with."""

    def __init__(self, cache, n_heads, window=0, sinks=0):
        n_heads, window, sinks = (int(as_int32(x, name)[0]) for x, name in
                                  ((n_heads, "n_heads"), (window, "window"), (sinks, "sinks")))
        self.cache, self.n_heads = cache, n_heads
        self.device = cache.k.device
        if self.device.type != "cuda":
            raise ValueError("the cache is not on the GPU")
        self.shape = lora_attn_shape_t(self.n_heads, cache.n_kv_heads, cache.head_dim, cache.page_tokens,
                                       cache.n_pages, cache.dtype, window, sinks)
        self._launch = lora_attn_launch_t()
        self._ref = ctypes.byref(self._launch)
        self._copied = HipEvent()    # the last staging copy
        self._pending = False
        self._workspace = torch.empty(0, dtype=torch.float32, device=self.device)
        self._dev = torch.empty(0, dtype=torch.int32, device=self.device)
        self._planned = False
        self._streams = {}           # streams that work on the batch's buffers was put on
        # pinned; the library's copies out of it are unknown to its allocator
        self._host = torch.empty(0, dtype=torch.int32)

    def _use(self, stream):
        """The stream that is meant; remembers it."""
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        self._streams[s.cuda_stream] = s
        return s

    def _empty(self, n, dtype, stream):
        """Device memory that was free on the stream when it was asked for: the
        allocator hands out blocks that its current stream may still be using."""
        with torch.cuda.stream(stream):
            return torch.empty(n, dtype=dtype, device=self.device)

    def _drop(self, t):
        """A device buffer is let go: its memory is not handed out again before
        the streams that may be using it have got past this point."""
        for s in self._streams.values():
            t.record_stream(s)

    def __del__(self):
        if sys.is_finalizing() or not hasattr(self, "_host"):
            return
        if self._pending:
            _held.append((self._host, self._copied))
        self._drop(self._dev)
        self._drop(self._workspace)

    def _alloc(self, cap, stream):
        _release()
        self._drop(self._dev)
        self._host = torch.empty(cap, dtype=torch.int32, pin_memory=True)
        self._dev = self._empty(cap, torch.int32, stream)

    def refresh(self, q_len, kv_len, block_table, stream=None):
        """q_len, kv_len: int [n_seq], new tokens and cached tokens with them;
        block_table: int32 [n_seq, pages] page ids (host), or None when nothing
        is cached."""
        ql, kl = as_int32(q_len, "q_len"), as_int32(kv_len, "kv_len")
        tab = None if block_table is None else as_int32(block_table, "block_table")
        if ql.ndim != 1 or ql.shape != kl.shape or (tab is not None and (tab.ndim != 2 or tab.shape[0] != ql.shape[0])):
            raise ValueError("q_len [n_seq], kv_len [n_seq], block_table [n_seq, pages]")
        if self._pending:
            self._copied.synchronize()   # the staging buffer may still be in flight
            self._pending = False
        self._planned = False
        s = self._use(stream)
        h = s.cuda_stream
        if not self._host.shape[0]:
            self._alloc(1 << 12, s)
        while True:
            st = _lib.lora_attn_prepare(ctypes.byref(self.shape), ql.shape[0], ql.ctypes.data, kl.ctypes.data,
                                        None if tab is None else tab.ctypes.data, 0 if tab is None else tab.shape[1],
                                        self._host.data_ptr(), self._host.shape[0], self._dev.data_ptr(), h,
                                        self._ref)
            if st != LORA_ECAPACITY or self._launch.info.n_staged <= self._host.shape[0]:
                break
            self._alloc(int(self._launch.info.n_staged) * 2, s)
        check_status(st, "lora_attn_prepare")
        if self.info.n_staged:
            self._copied.record(h)
            self._pending = True
        if self.info.workspace_floats > self._workspace.shape[0]:
            self._drop(self._workspace)
            self._workspace = self._empty(int(self.info.workspace_floats), torch.float32, s)
        self._planned = True
        return self

    @property
    def info(self):
        return self._launch.info

    def _check_cache(self, cache):
        cache = self.cache if cache is None else cache
        s = self.shape
        if (cache.n_pages, cache.n_kv_heads, cache.page_tokens, cache.head_dim, cache.dtype) != (
                s.n_pages, s.n_kv_heads, s.page_tokens, s.head_dim, s.kv_dtype):
            raise ValueError("the cache has another shape or type than the plan's")
        if cache.k.device != self.device:
            raise ValueError(f"the cache is not on {self.device}")
        return cache

    def _rows(self, t, heads, dtype, name):
        """[rows, heads * head_dim] with contiguous rows, on the batch's device."""
        width = heads * self.shape.head_dim
        if t.dim() != 2 or t.shape[1] != width or t.stride(1) != 1 or t.dtype != dtype or t.device != self.device:
            raise ValueError(f"{name}: {dtype} [rows, {width}] on {self.device}, rows contiguous")
        return int(t.shape[0])

    def _need(self, have, rows, name):
        if not self._planned:
            raise RuntimeError("the batch has no plan: call refresh() first")
        if have < rows:
            raise ValueError(f"{name} has {have} rows: the batch needs {rows}")

    def prepare_write(self, k, v, q=None, q_out=None, rope=None, cache=None, stream=None):
        """k, v (and q): the projections' outputs, fp32 or bf16 [rows, heads *
        head_dim]; q_out: bf16, takes the turned q; rope: fp32 [positions,
        rope_dim] (rope_table) or None.  Returns fn() that writes the batch's
        new tokens into the cache."""
        cache = self._check_cache(cache)
        if k.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("k, v and q are float32 or bfloat16")
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out go together")
        hk = self.shape.n_kv_heads
        have = [self._rows(k, hk, k.dtype, "k"), self._rows(v, hk, k.dtype, "v")]
        args = lora_kv_write_args_t(k=k.data_ptr(), v=v.data_ptr(), ldk=k.stride(0), ldv=v.stride(0),
                                    dtype=LORA_F32 if k.dtype == torch.float32 else LORA_BF16)
        if q is not None:
            have += [self._rows(q, self.n_heads, k.dtype, "q"), self._rows(q_out, self.n_heads, torch.bfloat16, "q_out")]
            args.q, args.ldq, args.q_out, args.ld_out = q.data_ptr(), q.stride(0), q_out.data_ptr(), q_out.stride(0)
        if rope is not None:
            if rope.dim() != 2 or rope.dtype != torch.float32 or not rope.is_contiguous() or rope.device != self.device:
                raise ValueError("rope: contiguous float32 [positions, rope_dim]")
            args.rope, args.rope_len, args.rope_dim = rope.data_ptr(), rope.shape[0], rope.shape[1]
        h, L, rows = self._use(stream).cuda_stream, self._launch, min(have)
        kv_ref, arg_ref, ref, call = ctypes.byref(cache.c()), ctypes.byref(args), self._ref, _lib.lora_kv_write

        def run():
            self._need(rows, L.info.n_rows, "an input or q_out")
            st = call(ref, kv_ref, arg_ref, h)
            if st != LORA_OK:
                check_status(st, "lora_kv_write")
        run.keep = (k, v, q, q_out, rope, cache, args)
        return run

    def prepare_read(self, k_out, v_out, cache=None, stream=None):
        """k_out, v_out: bf16 [tokens, n_kv_heads * head_dim].  Returns fn()
        that reads all kv_len tokens of every sequence back, sequence after
        sequence."""
        cache = self._check_cache(cache)
        hk = self.shape.n_kv_heads
        rows = min(self._rows(k_out, hk, torch.bfloat16, "k_out"), self._rows(v_out, hk, torch.bfloat16, "v_out"))
        if k_out.stride(0) != v_out.stride(0):
            raise ValueError("k_out and v_out have rows of one stride")
        h, L, ref, kv_ref = self._use(stream).cuda_stream, self._launch, self._ref, ctypes.byref(cache.c())
        kp, vp, ld, call = k_out.data_ptr(), v_out.data_ptr(), k_out.stride(0), _lib.lora_kv_read

        def run():
            self._need(rows, L.info.n_tokens, "an output")
            st = call(ref, kv_ref, kp, vp, ld, h)
            if st != LORA_OK:
                check_status(st, "lora_kv_read")
        run.keep = (k_out, v_out, cache)
        return run

    def prepare_attn(self, q, out, scale, cache=None, stream=None):
        """q, out: bf16 [rows, n_heads * head_dim]; scale: of the scores.
        Returns fn() that runs the batch's attention.  The partial results of
        split rows use the batch's one workspace: calls on one batch must be
        ordered (one stream, or events)."""
        cache = self._check_cache(cache)
        rows = min(self._rows(q, self.n_heads, torch.bfloat16, "q"), self._rows(out, self.n_heads, torch.bfloat16, "out"))
        h, L, ref, kv_ref = self._use(stream).cuda_stream, self._launch, self._ref, ctypes.byref(cache.c())
        qp, ldq, op, ldo, scale, call = q.data_ptr(), q.stride(0), out.data_ptr(), out.stride(0), float(scale), _lib.lora_attn

        def run():
            self._need(rows, L.info.n_rows, "q or out")
            ws = self._workspace
            st = call(ref, kv_ref, qp, ldq, op, ldo, scale, ws.data_ptr(), ws.shape[0], h)
            if st != LORA_OK:
                check_status(st, "lora_attn")
        run.keep = (q, out, cache)
        return run

    def write(self, k, v, q=None, q_out=None, rope=None, cache=None, stream=None):
        self.prepare_write(k, v, q, q_out, rope, cache, stream)()

    def read(self, k_out, v_out, cache=None, stream=None):
        self.prepare_read(k_out, v_out, cache, stream)()

    def attn(self, q, out, scale, cache=None, stream=None):
        self.prepare_attn(q, out, scale, cache, stream)()
