"""CPU tests of the cache's page manager and of what the page copy refuses."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import heterogeneous_adapter_batching_amd as hl
from heterogeneous_adapter_batching_amd.pages import KvCopy, KvPages

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def lists(x):
    return [list(a) for a in x]


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_manager_against_a_plain_one_under_sanitizers(tmp_path):
    exe = tmp_path / "kv_pages_sanitize"
    csrc = os.path.join(REPO, "heterogeneous_adapter_batching_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(REPO, "include"), os.path.join(csrc, "kv_pages.cpp"),
                    os.path.join(REPO, "tests", "kv_pages_sanitize.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "page manager ok" in r.stdout


def test_forks_share_pages_and_split_the_last():
    p = KvPages(8, 16, 4)
    assert lists(p.append([0], [37])) == [[], [], []]
    p.fork(0, [1, 2])
    assert p.stats() == (5, 3, 3)
    src, dst, n = p.append([0, 1, 2], [1, 1, 1])  # two copies: the third keeps the page
    assert list(src) == [2, 2] and list(dst) == [3, 4] and list(n) == [5, 5]
    table, kv = p.table([0, 1, 2])
    assert table.tolist() == [[0, 1, 3], [0, 1, 4], [0, 1, 2]] and list(kv) == [38] * 3
    assert lists(p.append([0, 1, 2], [1, 1, 1])) == [[], [], []]
    p.free([0])
    assert p.stats() == (4, 2, 5)
    src, dst, n = p.compact()
    assert (list(src), list(dst), list(n)) == ([4], [3], [7])
    assert p.table([1, 2])[0].tolist() == [[0, 1, 3], [0, 1, 2]]
    assert lists(p.compact()) == [[], [], []] and p.stats() == (4, 2, 4)


def test_a_full_last_page_is_not_split():
    p = KvPages(8, 16, 2)
    p.append([0], [32])
    p.fork(0, [1])
    assert lists(p.append([0, 1], [1, 0])) == [[], [], []]
    assert p.table([0, 1])[0].tolist() == [[0, 1, 2], [0, 1, 0]]


def test_truncated_inside_a_shared_page():
    p = KvPages(8, 16, 2)
    p.append([0], [30])
    p.fork(0, [1])
    p.truncate(0, 20)
    src, dst, n = p.append([0], [1])
    assert (list(src), list(dst), list(n)) == ([1], [2], [4])
    p.truncate(1, 0)
    assert p.stats() == (6, 0, 3)
    p.truncate(0, 16)
    assert p.table([0])[0].tolist() == [[0]]


def test_nothing_changes_when_pages_are_short():
    p = KvPages(4, 16, 3)
    p.append([0, 1], [20, 16])
    p.fork(0, [2])
    before = [x.tolist() for x in p.table([0, 1, 2])] + [p.stats()]
    for seqs, tokens in (([0, 1], [1, 1]), ([1], [33]), ([0, 2, 1], [1, 1, 1])):
        with pytest.raises(hl.LoraError) as e:
            p.append(seqs, tokens)
        assert e.value.code == hl.LORA_ECAPACITY
        assert [x.tolist() for x in p.table([0, 1, 2])] + [p.stats()] == before
    p.append([0], [1])


def test_manager_refuses():
    for args in ((0, 16, 1), (4, 16, 0), (1 << 30, 1024, 1), (-1, 16, 1)):
        with pytest.raises(hl.LoraError) as e:
            KvPages(*args)
        assert e.value.code == hl.LORA_EINVAL
    for page in (0, 3, 2048, -16):
        with pytest.raises(hl.LoraError) as e:
            KvPages(4, page, 1)
        assert e.value.code == hl.LORA_ESHAPE
    p = KvPages(4, 16, 3)
    p.append([0], [5])
    for call in (lambda: p.append([0, 0], [1, 1]), lambda: p.append([3], [1]), lambda: p.append([-1], [1]),
                 lambda: p.append([0], [-1]), lambda: p.append([0], [1 << 30]), lambda: p.fork(0, [0]),
                 lambda: p.fork(0, [1, 1]), lambda: p.fork(1, [0]), lambda: p.fork(3, [1]), lambda: p.fork(0, [3]),
                 lambda: p.truncate(0, 6), lambda: p.truncate(0, -1), lambda: p.truncate(5, 0), lambda: p.free([0, 3]),
                 lambda: p.table([3])):
        with pytest.raises(hl.LoraError) as e:
            call()
        assert e.value.code == hl.LORA_EINVAL
    for call in (lambda: p.append([0], [1, 2]), lambda: p.append([[0]], [[1]]), lambda: p.append([0], [0.5]),
                 lambda: p.truncate([0, 1], 0), lambda: p.append([0], [2 ** 32 + 1])):
        with pytest.raises(ValueError):
            call()
    assert p.table([0])[1].tolist() == [5]
    out, n = np.zeros(3, np.int32), ctypes.c_int32(0)
    assert hl._lib.lora_kv_pages_create(1, 16, 1, None) == hl.LORA_EINVAL
    assert hl._lib.lora_kv_pages_append(None, 0, None, None, None, None, None, ctypes.byref(n)) == hl.LORA_EINVAL
    assert hl._lib.lora_kv_pages_append(p._h, 1, out.ctypes.data, out.ctypes.data, None, None, None,
                                        ctypes.byref(n)) == hl.LORA_EINVAL
    assert hl._lib.lora_kv_pages_stats(None, None, None, None) == hl.LORA_EINVAL
    assert hl._lib.lora_kv_pages_destroy(None) == hl.LORA_OK
    assert p.append([], []) is not None and p.table([])[0].shape == (0, 0)


# ---------------------------------------------------------------- refusals of the copy
def kv(**change):
    f = dict(k=0x1000, v=0x2000, k_scale=None, v_scale=None, dtype=hl.LORA_KV_BF16, n_pages=10, page_tokens=16,
             n_kv_heads=2, head_dim=128, reserved=0, page_stride=4096, head_stride=2048, token_stride=128)
    f.update(change)
    return hl.lora_kv_t(**f)


def bounds(**change):
    f = dict(codes=0x3000, exps=0x4000, n_pages=10, n_kv_heads=2, head_dim=128, reserved=0)
    f.update(change)
    return hl.lora_kv_bounds_t(**f)


def array(kind, xs):
    return None if xs is None else (kind * len(xs))(*xs)


def copy(src, dst, tokens=None, caches=None, to=None, b=None, to_b=None, n=None):
    caches = [kv()] if caches is None else caches
    ids = [None if x is None else np.ascontiguousarray(x, np.int32) for x in (src, dst, tokens)]
    return hl._lib.lora_kv_copy(len(caches), array(hl.lora_kv_t, caches), array(hl.lora_kv_t, to),
                                array(hl.lora_kv_bounds_t, b), array(hl.lora_kv_bounds_t, to_b),
                                len(src) if n is None else n, *(None if x is None else x.ctypes.data for x in ids), None)


def test_copy_refuses_pages():
    for src, dst in (([10], [1]), ([-1], [1]), ([1], [10]), ([1, 2], [3, -1])):
        assert copy(src, dst) == hl.LORA_EPAGE
    for src, dst in (([1], [1]), ([1, 2], [3, 3]), ([1, 2], [2, 3]), ([1, 2, 3], [4, 5, 1])):
        assert copy(src, dst) == hl.LORA_EINVAL
    for tokens in ([17], [-1]):
        assert copy([1], [2], tokens) == hl.LORA_EINVAL
    assert copy([1, 2], [2, 3], to=[kv(v=0x9000)]) == hl.LORA_EINVAL  # the same keys
    assert copy([1], [12], to=[kv(k=0x8000, v=0x9000, n_pages=12)]) == hl.LORA_EPAGE
    assert copy([], []) == hl.LORA_OK and copy([1, 1], [2, 3], [0, 0]) == hl.LORA_OK  # nothing to launch


def test_copy_refuses_memory_written_twice_or_read_and_written():
    one, two, three = (kv(k=i << 20, v=i + 8 << 20) for i in (1, 2, 3))
    for to in ([three, three], [three, kv(k=3 << 20, v=12 << 20)], [three, kv(k=4 << 20, v=11 << 20)],
               [three, kv(k=11 << 20, v=4 << 20)]):
        assert copy([], [], caches=[one, two], to=to) == hl.LORA_EINVAL
    assert copy([], [], caches=[one, one], to=[two, three]) == hl.LORA_OK
    assert copy([1], [1], [0], caches=[one, two], to=[kv(k=4 << 20, v=5 << 20), three]) == hl.LORA_OK
    for to in ([two, one], [three, one], [two, three]):  # crosswise
        assert copy([1], [1], [0], caches=[one, two], to=to) == hl.LORA_EINVAL
        assert copy([1, 2], [2, 3], [0, 0], caches=[one, two], to=to) == hl.LORA_EINVAL
        assert copy([1, 1], [2, 3], [0, 0], caches=[one, two], to=to) == hl.LORA_OK
    b = [bounds(codes=i << 20) for i in (21, 22, 23)]
    assert copy([], [], caches=[one, one], to=[two, three], b=[b[0], b[0]], to_b=[b[1], b[1]]) == hl.LORA_EINVAL
    assert copy([], [], caches=[one, one], to=[two, three], b=[b[0], b[0]], to_b=[b[1], b[2]]) == hl.LORA_OK


@pytest.mark.parametrize("change,code", [
    (dict(k=None), hl.LORA_EINVAL), (dict(v=0x2008), hl.LORA_EINVAL), (dict(dtype=2), hl.LORA_EINVAL),
    (dict(page_tokens=12), hl.LORA_ESHAPE), (dict(page_tokens=2048), hl.LORA_ESHAPE), (dict(head_dim=96), hl.LORA_ESHAPE),
    (dict(n_kv_heads=0), hl.LORA_EINVAL), (dict(n_pages=0), hl.LORA_EINVAL), (dict(token_stride=132), hl.LORA_EINVAL),
    (dict(page_stride=-4096), hl.LORA_EINVAL), (dict(dtype=hl.LORA_KV_E4M3), hl.LORA_EINVAL),
    (dict(dtype=hl.LORA_KV_E4M3, k_scale=1, v_scale=1, head_stride=2056), hl.LORA_EINVAL)])
def test_copy_refuses_a_cache(change, code):
    assert copy([], [], caches=[kv(**change)]) == code
    assert copy([], [], caches=[kv()], to=[kv(**change)]) == code


def test_copy_refuses_caches_and_bounds_that_differ():
    assert copy([], [], caches=[kv(), kv(n_pages=11)]) == hl.LORA_ESHAPE
    assert copy([], [], caches=[kv(), kv(n_kv_heads=3)]) == hl.LORA_ESHAPE
    assert copy([], [], caches=[kv()], to=[kv(page_tokens=32)]) == hl.LORA_ESHAPE
    assert copy([], [], caches=[kv()], to=[kv(dtype=hl.LORA_KV_E4M3, k_scale=1, v_scale=1)]) == hl.LORA_ESHAPE
    assert copy([], [], b=[bounds(n_pages=9)]) == hl.LORA_ESHAPE
    assert copy([], [], b=[bounds(head_dim=64)]) == hl.LORA_ESHAPE
    assert copy([], [], b=[bounds(codes=0x3008)]) == hl.LORA_EINVAL
    assert copy([], [], b=[bounds(exps=None)]) == hl.LORA_EINVAL
    assert copy([], [], b=[bounds()], to=[kv()]) == hl.LORA_EINVAL
    assert copy([], [], to=[kv()], to_b=[bounds()]) == hl.LORA_EINVAL
    assert copy([], [], to_b=[bounds()]) == hl.LORA_EINVAL
    assert copy([1], [2], n=-1) == hl.LORA_EINVAL
    assert hl._lib.lora_kv_copy(0, None, None, None, None, 0, None, None, None, None) == hl.LORA_EINVAL
    assert hl._lib.lora_kv_copy(1, array(hl.lora_kv_t, [kv()]), None, None, None, 1, None, None, None, None) == hl.LORA_EINVAL


def test_what_is_refused_takes_no_memory():
    """Requests far beyond the cache are short of pages, and nothing is kept for them."""
    code = """
import resource, sys
sys.path.insert(0, %r)
import heterogeneous_adapter_batching_amd as hl
from heterogeneous_adapter_batching_amd.pages import KvPages
p = KvPages(100, 1, 64)
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 30),) * 2)
try:
    p.append(list(range(64)), [1 << 30] * 64)
except hl.LoraError as e:
    assert e.code == hl.LORA_ECAPACITY, e
assert p.stats() == (100, 0, 0)
print("refused")
""" % REPO
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused" in r.stdout, r.stdout + r.stderr


def test_many_children():
    """The check that no child is listed twice is linear."""
    n = 200000
    p = KvPages(10, 16, n + 1)
    p.append([n], [20])
    p.fork(n, np.arange(n))
    assert p.stats() == (8, 2, 2)
    p.free(np.arange(n))
    with pytest.raises(hl.LoraError):
        p.fork(n, np.r_[np.arange(n), 5])
    assert p.stats() == (8, 0, 2)


def test_copy_takes_gpu_caches_only():
    from heterogeneous_adapter_batching_amd.attention import KvCache
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        KvCopy([KvCache(k, k.clone())])
    with pytest.raises(ValueError):
        KvCopy([])
