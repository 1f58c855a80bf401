"""AttnBatch without a GPU: which stream its buffers belong to and what becomes of
them, over stand-ins for the device's memory, streams and events.  The plan is
the library's own; nothing is launched."""
import contextlib
import ctypes
import gc
import types

import numpy as np
import pytest
import torch

import heterogeneous_adapter_batching_amd as hl
from heterogeneous_adapter_batching_amd import attention
from test_attn_plan import check_plan

DEVICE = torch.device("cuda", 0)
LONG = ([1] * 8, [9000] * 8, np.arange(8 * 600, dtype=np.int32).reshape(8, 600))  # splits, and a large table


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Buffer:
    """Device memory: the stream that it was allocated on and those that were recorded on it."""

    def __init__(self, n, stream):
        self.shape, self.device, self.stream, self.recorded = (n,), DEVICE, stream, []
        self.memory = np.zeros(max(1, n), np.int32)

    def data_ptr(self):
        return self.memory.ctypes.data

    def record_stream(self, stream):
        self.recorded.append(stream)


class Event:
    """Of a copy that ends when the test says so, or when somebody waits for it."""
    done = True

    def record(self, stream=None):
        self.done = False

    def query(self):
        return self.done

    def synchronize(self):
        self.done = True


class World:
    def __init__(self, monkeypatch):
        self.main = Stream(0)
        self.current, self.buffers = self.main, []

        def empty(n, dtype=None, device=None, pin_memory=False):
            if device is None:
                return torch.empty(n, dtype=dtype)
            self.buffers.append(Buffer(n, self.current))
            return self.buffers[-1]

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            yield
            self.current = before

        class Torch:
            cuda = types.SimpleNamespace(current_stream=lambda device=None: self.current, stream=stream)

            def __getattr__(self, name):
                return getattr(torch, name)
        fake = Torch()
        fake.empty = empty
        lib = types.SimpleNamespace(lora_attn_prepare=self.prepare, lora_kv_write=None, lora_kv_read=None, lora_attn=None)
        monkeypatch.setattr(attention, "torch", fake)
        monkeypatch.setattr(attention, "HipEvent", Event)
        monkeypatch.setattr(attention, "_lib", lib)

    def prepare(self, shape, n, q_len, kv_len, table, ld_table, staging, capacity, dev, stream, out):
        st = hl._lib.lora_attn_plan(shape, n, q_len, kv_len, table, ld_table, staging, capacity,
                                    ctypes.byref(out._obj.info))
        if st == hl.LORA_OK:
            out._obj.meta = dev
            ctypes.memmove(dev, staging, 4 * out._obj.info.n_staged)
        return st

    def used(self):
        """The buffers that hold something."""
        return [b for b in self.buffers if b.shape[0]]


def cache(pages=5000, device=DEVICE, dtype=hl.LORA_KV_BF16):
    return types.SimpleNamespace(k=types.SimpleNamespace(device=device), n_pages=pages, n_kv_heads=2, page_tokens=16,
                                 head_dim=64, dtype=dtype, c=lambda: hl.lora_kv_t())


@pytest.fixture
def world(monkeypatch):
    yield World(monkeypatch)
    gc.collect()
    attention._held.clear()


def test_buffers_belong_to_the_stream_that_uses_them(world):
    """The allocator orders a block's reuse by the stream that it was asked for on."""
    side = Stream(7)
    batch = attention.AttnBatch(cache(), 4)
    batch.refresh([1], [20], np.array([[1, 2]], np.int32), stream=side)
    small = len(world.used())
    batch.refresh(*LONG, stream=side)  # both buffers grow
    assert small >= 1 and len(world.used()) >= small + 2
    assert all(b.stream is side for b in world.used())
    assert world.current is world.main
    other = Stream(9)
    batch = attention.AttnBatch(cache(), 4)
    world.current = other
    before = len(world.used())
    batch.refresh(*LONG)
    assert len(world.used()) > before and all(b.stream is other for b in world.used()[before:])


def test_a_buffer_that_grows_is_held_for_the_streams_that_use_it(world):
    one, two = Stream(1), Stream(2)
    batch = attention.AttnBatch(cache(), 4)
    batch.refresh([1], [20], np.array([[1, 2]], np.int32), stream=one)
    batch._use(two)
    old = world.used()
    batch.refresh(*LONG, stream=one)
    assert all({s.cuda_stream for s in b.recorded} >= {1, 2} for b in old)


def test_a_batch_let_go_leaves_its_buffers_to_the_work_under_way(world):
    """The staging buffer is read by a copy that the allocator knows nothing of, the
    others by work on any of the batch's streams."""
    side = Stream(7)
    batch = attention.AttnBatch(cache(), 4)
    batch.refresh(*LONG, stream=side)
    assert batch._pending and not batch._copied.done
    copied, staging, buffers = batch._copied, batch._host.data_ptr(), world.used()
    del batch
    gc.collect()
    assert not copied.done  # nobody waited
    assert [h.data_ptr() for h, _ in attention._held] == [staging]
    assert all(side in b.recorded for b in buffers[-2:])
    copied.done = True
    attention.AttnBatch(cache(), 4).refresh(*LONG, stream=side)  # asks for a staging buffer
    gc.collect()
    assert all(h.data_ptr() != staging or not e.done for h, e in attention._held)
    assert len(attention._held) == 1  # that of the batch just made


def test_refuses_a_cache_that_is_not_on_the_device(world):
    cpu, other = torch.device("cpu"), torch.device("cuda", 1)
    with pytest.raises(ValueError):
        attention.AttnBatch(cache(device=cpu), 4)
    batch = attention.AttnBatch(cache(), 4).refresh([1], [20], np.array([[1, 2]], np.int32))
    q = types.SimpleNamespace(dim=lambda: 2, shape=(1, 256), stride=lambda i: (256, 1)[i], dtype=torch.bfloat16,
                              device=DEVICE, data_ptr=lambda: 0x1000)
    kv = types.SimpleNamespace(dim=lambda: 2, shape=(20, 128), stride=lambda i: (128, 1)[i], dtype=torch.bfloat16,
                               device=DEVICE, data_ptr=lambda: 0x1000)
    batch.prepare_attn(q, q, 0.1, cache=cache())
    for device in (cpu, other):
        with pytest.raises(ValueError):
            batch.prepare_attn(q, q, 0.1, cache=cache(device=device))
        with pytest.raises(ValueError):
            batch.prepare_write(kv, kv, cache=cache(device=device))
        with pytest.raises(ValueError):
            batch.prepare_read(kv, kv, cache=cache(device=device))


WRAPS = 2 ** 32  # to 0 in 32 bits


@pytest.mark.parametrize("q_len,kv_len,table", [
    ([WRAPS + 1], [20], [[1, 2]]), ([1], [WRAPS + 20], [[1, 2]]), ([1], [20], [[1, WRAPS + 2]]),
    ([1], [20], [[1, -WRAPS + 2]]), ([1], [20.5], [[1, 2]]), ([float("nan")], [20], [[1, 2]])])
def test_refuses_numbers_that_32_bits_do_not_hold(world, q_len, kv_len, table):
    """Wrapped round they are lengths and pages of another batch."""
    batch = attention.AttnBatch(cache(), 4)
    args = [np.array(x) for x in (q_len, kv_len, table)]
    with pytest.raises(ValueError):
        batch.refresh(*args)
    with pytest.raises(ValueError):
        hl.lora_attn_plan(batch.shape, *args)


@pytest.mark.parametrize("args", [dict(n_heads=WRAPS + 4), dict(n_heads=4, window=WRAPS), dict(n_heads=4, window=-WRAPS + 9),
                                  dict(n_heads=4, window=9, sinks=WRAPS)])
def test_refuses_a_shape_that_32_bits_do_not_hold(world, args):
    with pytest.raises(ValueError):
        attention.AttnBatch(cache(), **args)


def test_takes_whole_numbers_of_any_type(world):
    table = np.array([[1, 2]])
    for kind in (np.int64, np.uint64, np.int16, np.float64):
        for args in (([1], [20], table), (np.array([1], kind), np.array([20], kind), table.astype(kind)),
                     (torch.tensor([1]), torch.tensor([20]), torch.from_numpy(table))):
            batch = attention.AttnBatch(cache(), 4).refresh(*args)
            check_plan(batch.shape, [1], [20], table, batch._host.numpy()[:batch.info.n_staged], batch.info)
    batch = attention.AttnBatch(cache(), 4).refresh([], [], None)
    assert batch.info.n_rows == 0
