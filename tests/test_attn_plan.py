"""CPU tests of the attention plan (lora_attn_plan), the e4m3 oracle, and the
refusals of the paged-cache calls (which return before any HIP call)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import heterogeneous_adapter_batching_amd as hl
import oracle

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TILE = 64
MOST = {hl.LORA_ATTN_NARROW: 16, hl.LORA_ATTN_WIDE: 128, hl.LORA_ATTN_PAIR: 256}  # rows of an item


def shape(heads=8, kv_heads=2, dim=128, page=16, pages=1000, dtype=hl.LORA_KV_BF16, window=0, sinks=0):
    return hl.lora_attn_shape_t(heads, kv_heads, dim, page, pages, dtype, window, sinks)


def make_table(rng, kv_len, page, pages):
    need = [-(-n // page) for n in kv_len]
    tab = np.full((len(kv_len), max([1] + need)), -77, np.int32)  # entries past the end are not read
    perm = rng.permutation(pages)[:sum(need)]
    at = 0
    for i, n in enumerate(need):
        tab[i, :n] = perm[at:at + n]
        at += n
    return tab


def span(p_lo, p_hi, window, sinks):
    """Tiles any of the positions sees, first to last."""
    tiles = set()
    for p in range(p_lo, p_hi + 1):
        tiles |= {j // TILE for j in oracle.visible_ref(p, p + 1, window, sinks)}
    return sorted(tiles)


def check_plan(s, q_len, kv_len, tab, staging, info):
    """What the kernels rely on: every row in one tile, every visible tile in
    exactly one split, splits of a tile in consecutive rows of the workspace."""
    group = s.n_heads // s.n_kv_heads

    def items(off, n):
        return staging[off:off + hl.ATTN_WORK_INTS * n].reshape(-1, hl.ATTN_WORK_INTS)
    starts = np.concatenate([[0], np.cumsum(q_len)])
    tiles, parts = {}, []
    for kind, most in MOST.items():
        for seq, row0, nrows, it0, it1, nsplits, part, q0, n_new, kv, tok0, lead in items(info.off_work[kind], info.n_work[kind]):
            assert 1 <= nrows <= most and nsplits >= 1
            assert (q0, n_new, kv) == (starts[seq], q_len[seq], kv_len[seq])
            assert (tok0, lead) == divmod(row0, group)
            tiles.setdefault((seq, row0, nrows), []).append((it0, it1, nsplits, part))
            if nsplits > 1:
                parts.append((part, part + nrows))
    for a, b in zip(sorted(parts), sorted(parts)[1:]):
        assert a[1] <= b[0]
    assert all(0 <= a and b <= info.part_rows for a, b in parts)
    assert info.workspace_floats == info.part_rows * s.n_kv_heads * (s.head_dim + 2)
    merges = {}
    for m in items(info.off_merge, info.n_merge):
        merges.setdefault(tuple(m[:3]), []).append(m)
    rows = {}
    for (seq, row0, nrows), got in tiles.items():
        rows.setdefault(seq, []).extend(range(row0, row0 + nrows))
        got.sort()
        n = got[0][2]
        assert len(got) == n and all(g[2] == n for g in got)
        assert got[0][0] == 0 and all(a[1] == b[0] for a, b in zip(got, got[1:]))
        p0 = int(kv_len[seq]) - int(q_len[seq])
        want = span(p0 + row0 // group, p0 + (row0 + nrows - 1) // group, s.window, s.sinks)
        assert got[-1][1] >= len(want)  # the list of tiles holds every visible one
        if n > 1:
            assert [g[3] for g in got] == [got[0][3] + i * nrows for i in range(n)]
            ms = merges.pop((seq, row0, nrows))
            assert all(m[5] == n and m[6] == got[0][3] for m in ms)
            assert sorted(r for m in ms for r in range(m[3], m[4])) == list(range(nrows))
    assert not merges
    for b, n in enumerate(q_len):
        assert sorted(rows.get(b, [])) == list(range(int(n) * group))
    assert np.array_equal(staging[info.off_kv_start:info.off_kv_start + len(q_len) + 1],
                          np.concatenate([[0], np.cumsum(kv_len)]))
    row = 0
    for b, n in enumerate(q_len):
        for i in range(int(n)):
            p = int(kv_len[b]) - int(n) + i
            slot = -1 if p < 0 else tab[b, p // s.page_tokens] * s.page_tokens + p % s.page_tokens
            assert staging[info.off_row_pos + row] == p and staging[info.off_row_slot + row] == slot
            row += 1
        need = -(-int(kv_len[b]) // s.page_tokens)
        staged = staging[info.off_table + b * info.ld_table:info.off_table + b * info.ld_table + need]
        assert np.array_equal(staged, tab[b, :need])


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 0), (64, 3), (130, 65), (7, 1000)])
def test_plan_covers_random_batches(window, sinks):
    rng = np.random.default_rng([window, sinks])
    for t in range(25):
        kv_heads, group = int(rng.choice([1, 2, 8])), int(rng.choice([1, 3, 4, 7]))
        page = int(rng.choice([1, 8, 64]))
        n = int(rng.integers(0, 6))
        q_len = rng.choice([0, 1, 1, 2, 17, 150, 300], n)
        kv_len = np.maximum(0, q_len + rng.choice([-3, 0, 1, 63, 64, 500], n))
        s = shape(kv_heads * group, kv_heads, 64, page, 4000, window=window, sinks=sinks)
        tab = make_table(rng, kv_len, page, 4000)
        staging, info = hl.lora_attn_plan(s, q_len, kv_len, tab)
        assert (info.n_seq, info.n_rows, info.n_tokens) == (n, q_len.sum(), kv_len.sum())
        assert info.max_kv == max([0, *kv_len])
        check_plan(s, q_len, kv_len, tab, staging, info)


def test_plan_splits_long_contexts_and_counts_a_window():
    rng = np.random.default_rng(1)
    tab = make_table(rng, [100000], 64, 2000)
    _, full = hl.lora_attn_plan(shape(page=64, pages=2000), [1], [100000], tab)
    assert full.n_merge == 1 and full.n_work[hl.LORA_ATTN_NARROW] >= 64
    staging, few = hl.lora_attn_plan(shape(page=64, pages=2000, window=1000, sinks=4), [1], [100000], tab)
    it = staging[few.off_work[0]:few.off_work[0] + hl.ATTN_WORK_INTS * few.n_work[0]].reshape(-1, hl.ATTN_WORK_INTS)
    assert (it[:, 4] - it[:, 3]).sum() <= 1000 // TILE + 3  # the window's tiles and one of sinks


def test_plan_of_nothing():
    staging, info = hl.lora_attn_plan(shape(), [], [], None)
    assert info.n_rows == 0 and list(info.n_work) == [0, 0, 0]
    staging, info = hl.lora_attn_plan(shape(), [2, 0], [0, 0], None)  # rows that see nothing still have an item
    assert info.n_work[0] == 1 and info.max_kv == 0


@pytest.mark.parametrize("change,code", [
    (dict(dim=80), hl.LORA_ESHAPE), (dict(dim=0), hl.LORA_ESHAPE), (dict(dim=256), hl.LORA_ESHAPE),
    (dict(heads=7), hl.LORA_ESHAPE), (dict(heads=0), hl.LORA_EINVAL), (dict(kv_heads=0), hl.LORA_EINVAL),
    (dict(page=0), hl.LORA_ESHAPE), (dict(page=24), hl.LORA_ESHAPE), (dict(page=2048), hl.LORA_ESHAPE),
    (dict(pages=0), hl.LORA_EINVAL), (dict(pages=2 ** 31 - 1), hl.LORA_EINVAL), (dict(dtype=2), hl.LORA_EINVAL),
    (dict(heads=4097, kv_heads=1), hl.LORA_ESHAPE), (dict(window=-1), hl.LORA_EINVAL), (dict(sinks=-1), hl.LORA_EINVAL)])
def test_plan_refuses_shapes(change, code):
    st, _, _ = hl.lora_attn_plan(shape(**change), [1], [1], np.zeros((1, 1), np.int32), raw=True)
    assert st == code


def test_plan_refuses_batches():
    tab = np.zeros((2, 2), np.int32)
    assert hl.lora_attn_plan(shape(), [-1, 1], [1, 1], tab, raw=True)[0] == hl.LORA_EINVAL
    assert hl.lora_attn_plan(shape(), [1, 1], [1, -1], tab, raw=True)[0] == hl.LORA_EINVAL
    assert hl.lora_attn_plan(shape(), [1, 1], [1, 33], tab, raw=True)[0] == hl.LORA_EINVAL  # 33 tokens, 2 pages of 16
    assert hl.lora_attn_plan(shape(), [1, 1], [1, 2 ** 30 + 1], tab, raw=True)[0] == hl.LORA_EINVAL
    assert hl.lora_attn_plan(shape(), [2 ** 30, 2 ** 30], [1, 1], tab, raw=True)[0] == hl.LORA_EINVAL
    assert hl.lora_attn_plan(shape(), [1], [1], None, raw=True)[0] == hl.LORA_EINVAL
    for page in (-1, 1000, 2 ** 31 - 1):
        bad = np.array([[0, 5], [3, page]], np.int32)
        assert hl.lora_attn_plan(shape(), [1, 1], [32, 17], bad, raw=True)[0] == hl.LORA_EPAGE
        assert hl.lora_attn_plan(shape(), [1, 1], [32, 16], bad, raw=True)[0] == hl.LORA_OK  # not read
    st, _, info = hl.lora_attn_plan(shape(), [1, 1], [1, 32], tab, staging_capacity=3, raw=True)
    assert st == hl.LORA_ECAPACITY and info.n_staged > 3
    info = hl.lora_attn_info_t()
    one = np.ones(1, np.int32)
    sh = shape()
    assert hl._lib.lora_attn_plan(None, 1, one.ctypes.data, one.ctypes.data, None, 0, None, 0,
                                  ctypes.byref(info)) == hl.LORA_EINVAL
    assert hl._lib.lora_attn_plan(ctypes.byref(sh), 1, None, one.ctypes.data, None, 0, None, 0,
                                  ctypes.byref(info)) == hl.LORA_EINVAL
    assert hl._lib.lora_attn_plan(ctypes.byref(sh), 1, one.ctypes.data, one.ctypes.data, None, 0, None, 0,
                                  None) == hl.LORA_EINVAL


# ---------------------------------------------------------------- refusals of the GPU calls (nothing is launched)
def _launch(q_len=(3,), kv_len=(20,), **kw):
    s = shape(**kw)
    tab = np.arange(2 * len(q_len), dtype=np.int32).reshape(len(q_len), 2)
    _, info = hl.lora_attn_plan(s, list(q_len), list(kv_len), tab)
    return hl.lora_attn_launch_t(0x1000, info)


def _kv(**change):
    f = dict(k=0x10000, v=0x20000, k_scale=None, v_scale=None, dtype=hl.LORA_KV_BF16, n_pages=1000, page_tokens=16,
             n_kv_heads=2, head_dim=128, reserved=0, page_stride=4096, head_stride=2048, token_stride=128)
    f.update(change)
    return hl.lora_kv_t(**f)


BAD_KV = [(dict(k=None), hl.LORA_EINVAL), (dict(v=0x20004), hl.LORA_EINVAL), (dict(n_pages=999), hl.LORA_ESHAPE),
          (dict(page_tokens=32), hl.LORA_ESHAPE), (dict(n_kv_heads=1), hl.LORA_ESHAPE),
          (dict(head_dim=64), hl.LORA_ESHAPE), (dict(dtype=hl.LORA_KV_E4M3), hl.LORA_ESHAPE),
          (dict(page_stride=4100), hl.LORA_EINVAL), (dict(head_stride=-8), hl.LORA_EINVAL),
          (dict(token_stride=4), hl.LORA_EINVAL)]


def _attn(L, kv, q=0x1000, ldq=1024, out=0x2000, ldo=1024, scale=0.1, ws=0x4000, ws_floats=1 << 40):
    return hl._lib.lora_attn(ctypes.byref(L), ctypes.byref(kv), q, ldq, out, ldo, scale, ws, ws_floats, None)


def _write(L, kv, **change):
    f = dict(q=0x1000, k=0x2000, v=0x3000, ldq=1024, ldk=256, ldv=256, rope=0x4000, q_out=0x5000, ld_out=1024,
             dtype=hl.LORA_F32, rope_len=20, rope_dim=128, reserved=0)
    f.update(change)
    return hl._lib.lora_kv_write(ctypes.byref(L), ctypes.byref(kv),
                                 ctypes.byref(hl.lora_kv_write_args_t(**f)), None)


def _read(L, kv, k=0x1000, v=0x2000, ld=256):
    return hl._lib.lora_kv_read(ctypes.byref(L), ctypes.byref(kv), k, v, ld, None)


@pytest.mark.parametrize("change,code", BAD_KV)
def test_calls_refuse_a_cache_that_is_not_the_plans(change, code):
    L, kv = _launch(), _kv(**change)
    assert _attn(L, kv) == code and _write(L, kv) == code and _read(L, kv) == code


def test_calls_refuse_arguments():
    L, kv, bad = _launch(), _kv(), hl.LORA_EINVAL
    for kw in (dict(q=None), dict(q=0x1008), dict(ldq=1016), dict(ldq=1028), dict(out=None), dict(ldo=512),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _attn(L, kv, **kw) == bad, kw
    for kw in (dict(k=None), dict(v=0x3001), dict(ldk=248), dict(ldv=260), dict(q_out=None), dict(ld_out=8),
               dict(dtype=2), dict(rope=None), dict(rope_dim=0), dict(rope_len=19), dict(rope=0x4004)):
        assert _write(L, kv, **kw) == bad, kw
    for d in (8, 144, -16):
        assert _write(L, kv, rope_dim=d) == hl.LORA_ESHAPE
    for kw in (dict(k=None), dict(v=0x2002), dict(ld=128), dict(ld=257)):
        assert _read(L, kv, **kw) == bad, kw
    assert hl._lib.lora_attn(None, ctypes.byref(kv), 16, 8, 16, 8, 1.0, None, 0, None) == bad
    assert hl._lib.lora_kv_write(ctypes.byref(L), None, None, None) == bad
    assert hl._lib.lora_kv_read(ctypes.byref(L), None, 16, 16, 8, None) == bad
    e4m3 = _launch(dtype=hl.LORA_KV_E4M3)
    assert _attn(e4m3, _kv(dtype=hl.LORA_KV_E4M3)) == bad  # no scales
    assert _attn(e4m3, _kv(dtype=hl.LORA_KV_E4M3, k_scale=1, v_scale=1, token_stride=136)) == bad


def test_attn_refuses_a_small_workspace():
    s = shape(page=64, pages=2000)
    _, info = hl.lora_attn_plan(s, [1], [100000], make_table(np.random.default_rng(0), [100000], 64, 2000))
    L = hl.lora_attn_launch_t(0x1000, info)
    kv = _kv(n_pages=2000, page_tokens=64, page_stride=16384, head_stride=8192)
    need = int(info.workspace_floats)
    assert need > 0
    assert _attn(L, kv, ws_floats=need - 1) == hl.LORA_ECAPACITY
    assert _attn(L, kv, ws=None, ws_floats=need) == hl.LORA_EINVAL
    assert _attn(L, kv, ws=0x4004, ws_floats=need) == hl.LORA_EINVAL


def test_empty_batches_launch_nothing():
    _, info = hl.lora_attn_plan(shape(), [0], [0], None)
    L = hl.lora_attn_launch_t(0x1000, info)
    assert _attn(L, _kv(), q=None, out=None) == hl.LORA_OK
    assert _write(L, _kv(), k=None, v=None) == hl.LORA_OK
    assert _read(L, _kv(), k=None, v=None) == hl.LORA_OK


def test_cache_refuses_tensors():
    from heterogeneous_adapter_batching_amd.attention import KvCache
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for bad in ((k, k[:3]), (k, k.half()), (k.half(), k.half()), (k[0], k[0]), (k, k, torch.zeros(4, 2, 16), None),
                (k.transpose(2, 3), k.transpose(2, 3)), (k, k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3))):
        with pytest.raises(ValueError):
            KvCache(*bad)
    f8 = k.to(torch.float8_e4m3fn)
    scale = torch.zeros(4, 2, 16, dtype=torch.uint8)
    for bad in ((f8, f8), (f8, f8, scale, None), (f8, f8, scale, scale[:3]), (f8, f8, scale, scale.float())):
        with pytest.raises(ValueError):
            KvCache(*bad)
    KvCache(f8, f8, scale, scale)


# ---------------------------------------------------------------- the oracle
def test_oracle_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_values(), want, equal_nan=True)
    rng = np.random.default_rng(3)
    v = oracle.e4m3_values()[:127]
    y = np.concatenate([v, (v[1:] + v[:-1]) / 2, rng.uniform(0, 448, 5000), 2.0 ** rng.uniform(-12, 8, 5000)])
    y = np.float32(np.concatenate([y, -y]))
    got = oracle.e4m3_nearest(y)
    assert np.array_equal(got, torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_quantise_picks_the_least_power():
    x = np.array([[448.0, 1.0], [449.0, 0.0], [0.0, 0.0], [3.0, -2.0], [3.4e38, 1.0], [np.inf, 1.0], [1e-40, 0.0]])
    codes, e = oracle.quantise_ref(x)
    assert list(e) == [0, 1, -100, -7, 119, -8, -100]
    assert codes[5, 0] == 0x7F and oracle.e4m3_values()[codes[5, 1]] * 2.0 ** -8 == 1.0


def test_oracle_attend_matches_torch_softmax():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    out, _, _ = oracle.attend_ref(q, k, v, 5, 0, 0, 0.5)
    kk, vv = (torch.from_numpy(t).repeat_interleave(2, 1) for t in (k, v))
    s = 0.5 * torch.einsum("nhd,jhd->hnj", torch.from_numpy(q), kk)
    s.masked_fill_(torch.arange(5) > torch.arange(2, 5)[:, None], float("-inf"))
    want = torch.einsum("hnj,jhd->nhd", s.softmax(-1), vv)
    assert np.allclose(out, want.numpy(), rtol=1e-12, atol=1e-12)
    assert oracle.visible_ref(5, 6, 2, 1) == [0, 4, 5] and oracle.visible_ref(-1, 0, 0, 0) == []


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_attn_planner_under_address_and_ub_sanitizers(tmp_path):
    exe = tmp_path / "attn_sanitize"
    csrc = os.path.join(REPO, "heterogeneous_adapter_batching_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-I", os.path.join(REPO, "include"), os.path.join(csrc, "attn_plan.cpp"),
                    os.path.join(REPO, "tests", "attn_sanitize.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "attention planner ok" in r.stdout
