"""CPU tests of the sparse attention: the plan (lora_sparse_plan), the oracle, and
refusals, which come before any HIP call."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

import heterogeneous_adapter_batching_amd as hl
import oracle
from heterogeneous_adapter_batching_amd import attention, sparse
from test_attn_batch import DEVICE, cache, world  # noqa: F401
from test_attn_plan import check_plan, make_table, shape

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def wanted(select=4, first=1, last=1):
    return hl.lora_sparse_shape_t(select, first, last, 0)


def ints(staging, off, n, width):
    return staging[off:off + n * width].reshape(n, width).tolist()


def check_sparse(s, sp, q_len, kv_len, table, bounded, staging, attn, info):
    """The plan covers every row and page once, from the definition."""
    page, group, hk = s.page_tokens, s.n_heads // s.n_kv_heads, s.n_kv_heads
    rows = [(b, kv_len[b] - q_len[b] + i) for b in range(len(q_len)) for i in range(q_len[b])]
    seen = []
    for seq, row, n, pos in ints(staging, info.off_items, info.n_items, 4):
        assert 1 <= n <= info.item_tokens
        for i in range(n):
            assert rows[row + i] == (seq, pos + i)
            scored = (pos + i) // page + 1 - sp.first - sp.last if (pos + i) // page + 1 > sp.select and pos + i >= 0 else 0
            assert scored <= info.max_scored
        seen += range(row, row + n)
    assert sorted(seen) == list(range(len(rows)))
    pad = 1
    while pad < min(group, 16):
        pad *= 2
    assert info.item_tokens * pad <= 64 and (info.item_tokens == 1 or info.item_tokens * info.max_scored <= 12288)
    if info.item_tokens == 1 and info.max_scored > 2048:  # through memory
        assert attn.workspace_floats >= hk * info.max_scored
    # attention items: every row and head over every tile once
    tiles, parts = {}, 0
    for w in ints(staging, info.off_work, info.n_work, hl.ATTN_WORK_INTS):
        seq, row0, n, it0, it1, nsplits, part, q0, n_new, kv, tok0, lead = w
        p = rows[seq][1]
        assert q0 == seq and n_new == 1 and tok0 == 0 and lead == row0 and 1 <= n <= 16 and row0 + n <= group
        assert kv == (0 if p < 0 else (min(p // page + 1, sp.select) - 1) * page + p % page + 1)
        assert kv <= attn.max_kv and -(-kv // page) <= sp.select
        tiles.setdefault((seq, row0, n, nsplits), []).append((it0, it1, part))
    covered = {r: set() for r in range(len(rows))}
    for (seq, row0, n, nsplits), spans in tiles.items():
        kv = 0 if rows[seq][1] < 0 else (min(rows[seq][1] // page + 1, sp.select) - 1) * page + rows[seq][1] % page + 1
        assert len(spans) == nsplits
        at = 0
        for it0, it1, part in sorted(spans):
            assert it0 == at
            at = it1
            if nsplits > 1:
                assert part >= 0
                parts += n
        assert at == -(-kv // 64)
        covered[seq] |= set(range(row0, row0 + n))
    assert all(c == set(range(group)) for c in covered.values())
    assert parts == info.part_rows
    assert attn.workspace_floats >= info.part_rows * hk * (s.head_dim + 2)
    want = []
    for b in range(len(q_len)):
        done = max(0, kv_len[b] - q_len[b]) if bounded is None else bounded[b]
        want += [int(table[b, i]) for i in range(kv_len[b] // page) if (i + 1) * page > done]
    assert staging[info.off_fresh:info.off_fresh + info.n_fresh].tolist() == want
    assert attn.n_staged >= info.off_fresh + info.n_fresh


CASES = [([1], [1000]), ([1, 1, 1], [16, 17, 4000]), ([40, 1, 0, 3], [700, 5, 30, 2]), ([5, 300], [2, 300]), ([0], [0]), ([], [])]


@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (8, 4), (14, 2), (16, 1), (40, 1)])
@pytest.mark.parametrize("q_len,kv_len", CASES)
@pytest.mark.parametrize("page,sp", [(16, (4, 1, 1)), (64, (2, 0, 2)), (32, (9, 2, 3)), (16, (3, 1, 2)), (128, (1, 0, 1))])
def test_plan(page, sp, q_len, kv_len, heads, kv_heads):
    s, sp = shape(heads, kv_heads, page=page), wanted(*sp)
    table = make_table(np.random.default_rng(1), kv_len, page, 1000)
    for bounded in (None, [k // 3 for k in kv_len], [0] * len(kv_len), list(kv_len)):
        staging, attn, info = hl.lora_sparse_plan(s, sp, q_len, kv_len, table, bounded)
        check_sparse(s, sp, q_len, kv_len, table, bounded, staging, attn, info)
    # the first part is lora_attn_plan's
    plain, want = hl.lora_attn_plan(s, q_len, kv_len, table)
    assert np.array_equal(staging[:len(plain)], plain)
    for name, _ in hl.lora_attn_info_t._fields_:
        if name not in ("n_staged", "workspace_floats", "shape"):
            a, b = getattr(attn, name), getattr(want, name)
            assert (list(a) if hasattr(a, "__len__") else a) == (list(b) if hasattr(b, "__len__") else b), name
    if kv_len:
        check_plan(s, q_len, kv_len, table, staging[:len(plain)], want)


def test_plan_of_many_pages_goes_through_memory():
    s = shape(4, 2, page=16, pages=100000)
    kv = 16 * 40000
    table = np.arange(40000, dtype=np.int32)[None]
    staging, attn, info = hl.lora_sparse_plan(s, wanted(8), [1], [kv], table)
    assert info.max_scored == 40000 - 2 and info.item_tokens == 1
    assert attn.workspace_floats >= 2 * info.max_scored
    check_sparse(s, wanted(8), [1], [kv], table, None, staging, attn, info)


def test_plan_refuses():
    table = np.array([[1, 2, 3]], np.int32)

    def plan(s=None, sp=None, q=(1,), kv=(40,), tab=table, **kw):
        return hl.lora_sparse_plan(s or shape(), sp or wanted(), q, kv, tab, raw=True, **kw)[0]
    assert plan() == hl.LORA_OK
    for sp in (wanted(1), wanted(0, 0, 1), wanted(4, -1, 1), wanted(4, 1, 0), wanted((1 << 30) + 1), wanted(4, 2 ** 31 - 1, 1)):
        assert plan(sp=sp) == hl.LORA_EINVAL
    assert plan(s=shape(window=4)) == hl.LORA_EINVAL and plan(s=shape(sinks=1)) == hl.LORA_EINVAL
    assert plan(s=shape(page=8), tab=np.zeros((1, 5), np.int32)) == hl.LORA_ESHAPE
    assert plan(bounded=[41]) == hl.LORA_EINVAL and plan(bounded=[-1]) == hl.LORA_EINVAL
    assert plan(bounded=[40]) == hl.LORA_OK
    assert plan(tab=np.array([[1, 2, 1000]], np.int32)) == hl.LORA_EPAGE
    assert plan(q=(-1,)) == hl.LORA_EINVAL and plan(s=shape(dim=96)) == hl.LORA_ESHAPE
    _, attn, info = hl.lora_sparse_plan(shape(), wanted(), [1], [40], table)
    for short in (1, 8):
        st, _, a, _ = hl.lora_sparse_plan(shape(), wanted(), [1], [40], table, staging_capacity=attn.n_staged - short, raw=True)
        assert st == hl.LORA_ECAPACITY and a.n_staged == attn.n_staged
    null = ctypes.byref(hl.lora_attn_info_t())
    assert hl._lib.lora_sparse_plan(None, None, 0, None, None, None, None, 0, None, 0, null, None) == hl.LORA_EINVAL


def launch(**change):
    staging, attn, info = hl.lora_sparse_plan(shape(), wanted(2), [3], [100], np.arange(7, dtype=np.int32)[None])
    L = hl.lora_sparse_launch_t(hl.lora_attn_launch_t(0x1000, attn), info)
    for k, v in change.items():
        setattr(L.info.shape if hasattr(L.info.shape, k) else L.info, k, v)
    return L


def kv(**change):
    f = dict(k=0x1000, v=0x2000, k_scale=None, v_scale=None, dtype=hl.LORA_KV_BF16, n_pages=1000, page_tokens=16,
             n_kv_heads=2, head_dim=128, reserved=0, page_stride=4096, head_stride=2048, token_stride=128)
    f.update(change)
    return hl.lora_kv_t(**f)


def bounds(**change):
    f = dict(codes=0x3000, exps=0x4000, n_pages=1000, n_kv_heads=2, head_dim=128, reserved=0)
    f.update(change)
    return hl.lora_kv_bounds_t(**f)


def call(name, L=None, c=None, b=None, q=0x1000, ldq=1024, sel=0x5000, out=0x2000, ldo=1024, scale=0.1, ws=0x6000, n=1 << 40):
    L, c, b = ctypes.byref(L or launch()), ctypes.byref(c or kv()), ctypes.byref(b or bounds())
    if name == "bounds":
        return hl._lib.lora_kv_bounds(L, c, b, None)
    if name == "select":
        return hl._lib.lora_sparse_select(L, b, q, ldq, sel, ws, n, None)
    return hl._lib.lora_sparse_attn(L, c, q, ldq, sel, out, ldo, scale, ws, n, None)


@pytest.mark.parametrize("change,code", [
    (dict(n_pages=9), hl.LORA_ESHAPE), (dict(head_dim=64), hl.LORA_ESHAPE), (dict(n_kv_heads=1), hl.LORA_ESHAPE),
    (dict(codes=None), hl.LORA_EINVAL), (dict(codes=0x3008), hl.LORA_EINVAL), (dict(exps=None), hl.LORA_EINVAL)])
def test_calls_refuse_bounds(change, code):
    assert call("bounds", b=bounds(**change)) == code and call("select", b=bounds(**change)) == code


@pytest.mark.parametrize("change", [dict(select=1), dict(first=-1), dict(last=0), dict(select=(1 << 30) + 1), dict(n_items=-1),
                                    dict(n_fresh=-1), dict(max_scored=-1), dict(item_tokens=0)])
def test_calls_refuse_a_plan_that_is_none(change):
    for name in ("bounds", "select", "attn"):
        assert call(name, L=launch(**change)) == hl.LORA_EINVAL
    dead = launch()
    dead.attn.meta = None  # as a failed lora_sparse_prepare leaves it
    for name in ("bounds", "select", "attn"):
        assert call(name, L=dead) == hl.LORA_EINVAL


def test_calls_refuse_arguments():
    bad = hl.LORA_EINVAL
    for kw in (dict(q=None), dict(q=0x1008), dict(ldq=1016), dict(ldq=1028), dict(sel=None), dict(sel=0x5002)):
        assert call("select", **kw) == bad and call("attn", **kw) == bad, kw
    for kw in (dict(out=None), dict(ldo=512), dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert call("attn", **kw) == bad, kw
    assert call("select", L=launch(item_tokens=17)) == bad  # more rows than are scored at once
    for name in ("bounds", "attn"):
        assert call(name, c=kv(n_pages=999)) == hl.LORA_ESHAPE and call(name, c=kv(k=None)) == bad
    assert hl._lib.lora_sparse_attn(None, None, 16, 8, 16, 16, 8, 1.0, None, 0, None) == bad
    assert hl._lib.lora_kv_bounds(None, None, None, None) == bad
    assert hl._lib.lora_sparse_select(None, None, 16, 8, 16, None, 0, None) == bad
    assert hl._lib.lora_sparse_prepare(None, None, 0, None, None, None, None, 0, None, 0, None, None, None) == bad


def test_calls_refuse_a_small_workspace():
    staging, attn, info = hl.lora_sparse_plan(shape(8, 2, page=16, pages=40000), wanted(600), [1], [16 * 30000],
                                              np.arange(30000, dtype=np.int32)[None])
    L = hl.lora_sparse_launch_t(hl.lora_attn_launch_t(0x1000, attn), info)
    need, c, b = int(attn.workspace_floats), kv(n_pages=40000), bounds(n_pages=40000)
    assert need > 0 and info.n_merge > 0
    for name in ("select", "attn"):
        assert call(name, L=L, c=c, b=b, n=need - 1) == hl.LORA_ECAPACITY
        assert call(name, L=L, c=c, b=b, ws=None, n=need) == hl.LORA_EINVAL
        assert call(name, L=L, c=c, b=b, ws=0x6004, n=need) == hl.LORA_EINVAL


def test_empty_batches_launch_nothing():
    staging, attn, info = hl.lora_sparse_plan(shape(), wanted(), [0], [0], None)
    L = hl.lora_sparse_launch_t(hl.lora_attn_launch_t(0x1000, attn), info)
    for name in ("bounds", "select", "attn"):
        assert call(name, L=L, q=None, sel=None, out=None) == hl.LORA_OK


def test_batch_plans_and_refuses(world, monkeypatch):  # noqa: F811
    def prepare(shape_, sp, n, q, kv_, bnd, tab, ld, staging, capacity, dev, stream, out):
        st = hl._lib.lora_sparse_plan(shape_, sp, n, q, kv_, bnd, tab, ld, staging, capacity,
                                      ctypes.byref(out._obj.attn.info), ctypes.byref(out._obj.info))
        if st == hl.LORA_OK:
            out._obj.attn.meta = dev
            ctypes.memmove(dev, staging, 4 * out._obj.attn.info.n_staged)
        return st
    import types
    monkeypatch.setattr(sparse, "_lib", types.SimpleNamespace(lora_sparse_prepare=prepare, lora_kv_bounds=None,
                                                              lora_sparse_select=None, lora_sparse_attn=None))
    batch = sparse.SparseBatch(cache(), 4, 3)
    with pytest.raises(RuntimeError):
        batch._need(0, 0, "")
    table = np.arange(8 * 600, dtype=np.int32).reshape(8, 600)
    batch.refresh([1] * 8, [9000] * 8, table)  # both buffers grow
    check_sparse(batch.shape, batch.sparse_shape, [1] * 8, [9000] * 8, table, None,
                 batch._host.numpy()[:batch.info.n_staged], batch.info, batch.sparse_info)
    batch.refresh([1], [40], table[:1], bounded=[0])
    assert batch.sparse_info.n_fresh == 2 and batch.info.n_rows == 1
    for bad in ([0, 0], [2 ** 32], [0.5]):
        with pytest.raises(ValueError):
            batch.refresh([1], [40], table[:1], bounded=bad)
    with pytest.raises(hl.LoraError):
        batch.refresh([1], [40], table[:1], bounded=[41])
    for args in ((1,), (4, -1), (4, 1, 0), (2 ** 32 + 4,), (3, 2, 2)):
        with pytest.raises(ValueError):
            sparse.SparseBatch(cache(), 4, *args)


def test_another_device_than_the_current_one(world, monkeypatch):  # noqa: F811
    """The default stream is the current device's: launched there, the work would not be the tensors' device's."""
    import types
    from heterogeneous_adapter_batching_amd import pages
    from test_attn_batch import Stream
    now = [0]
    monkeypatch.setattr(pages, "torch", types.SimpleNamespace(cuda=types.SimpleNamespace(
        is_initialized=lambda: True, current_device=lambda: now[0])))
    monkeypatch.setattr(sparse, "_lib", hl._lib)
    batch = sparse.SparseBatch(cache(), 4, 3)
    batch._use(None)
    now[0] = 1
    with pytest.raises(ValueError):
        batch._use(None)
    with pytest.raises(ValueError):
        pages.check_device(DEVICE, 0)
    batch._use(Stream(7))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_sparse_planner_under_address_and_ub_sanitizers(tmp_path):
    exe = tmp_path / "sparse_sanitize"
    csrc = os.path.join(REPO, "heterogeneous_adapter_batching_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(REPO, "include"), os.path.join(csrc, "attn_plan.cpp"),
                    os.path.join(REPO, "tests", "sparse_sanitize.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "sparse planner ok" in r.stdout


# ---------------------------------------------------------------- the oracle
def test_oracle_codes_and_exponents():
    assert [oracle.exponent_ref(x) for x in (127.0, 127.5, 1.0, 0.0, 1e38, 2.0 ** -120)] == [0, 1, -6, -100, 100, -100]
    assert list(oracle.code_ref([0.5, 1.5, -2.5, 200, -1e9, np.inf, -np.inf, np.nan], 0)) == [0, 2, -2, 127, -127, 127, -127, 0]


def test_oracle_bounds_and_scores():
    k = np.array([[1.0, -4.0, np.nan], [3.0, 2.0, np.nan]])
    codes, e = oracle.bounds_ref(k)
    assert e == -4 and codes.tolist() == [[48, 32, 0], [16, -64, 0]]
    # r = (64, -32, ..) at 2^-6: 64 * 48 + -32 * -64
    s = oracle.scores_ref([[1.0, -0.5, 0.25]], codes[None], [e])
    assert s[0] == (64 * 48 + 32 * 64) / 16
    k[0, 0] = np.inf
    codes, e = oracle.bounds_ref(k)
    assert e == -4 and codes[0, 0] == 127
    # no key inside the bounds scores more, but for the roundings
    rng = np.random.default_rng(2)
    k, q = rng.standard_normal((16, 64)), rng.standard_normal((2, 64))
    codes, e = oracle.bounds_ref(k)
    f = oracle.exponent_ref(np.abs(q).max())
    best = oracle.scores_ref(q, codes[None], [e])[0] * 2.0 ** f
    slack = 64 * (0.5 * 2.0 ** e * np.abs(q).max() + 0.5 * 2.0 ** f * (np.abs(k).max() + 2.0 ** e))
    assert (k @ q.T).max() <= best + slack


def test_oracle_select():
    codes = np.zeros((6, 2, 4), int)
    codes[:, 0, 0] = codes[:, 1, 0] = [9, 5, 7, 7, 5, 1]
    q = np.array([[127.0, 0, 0, 0]])
    assert oracle.select_ref(q, codes, [0] * 6, 5, 4, 1, 1) == [0, 2, 3, 5]
    assert oracle.select_ref(q, codes, [0] * 6, 5, 4, 0, 2) == [0, 2, 4, 5]
    assert oracle.select_ref(q, codes, [0] * 6, 3, 4, 0, 2) == [0, 1, 2, 3]
    assert oracle.select_ref(q, codes, [0, 3, 0, 0, 0, 0], 5, 3, 0, 1) == [0, 1, 5]
    assert oracle.select_ref(q, codes * 0, [0] * 6, 5, 4, 1, 1) == [0, 1, 2, 5]  # equals: the earlier
