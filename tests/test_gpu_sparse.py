"""The bounds of pages, the choice of pages by them and the attention over the
chosen pages on the GPU, against the oracle.  Bounds and choice are whole numbers
and have to be equal.  The attention's tolerance is that of test_gpu_attn.py, over
the tokens of the chosen pages."""
import numpy as np
import pytest
import torch

import heterogeneous_adapter_batching_amd as hl
import oracle
from heterogeneous_adapter_batching_amd.attention import KvCache
from heterogeneous_adapter_batching_amd.sparse import KvBounds, SparseBatch
from test_gpu_attn import check, make_cache, make_table, tokens, values
from test_gpu_kv_copy import make_bounds

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def page_values(cache, pages):
    at = torch.from_numpy(np.asarray(pages, np.int64)).cuda()
    return values(cache.k[at], None if cache.k_scale is None else cache.k_scale[at])


def check_bounds(cache, bounds, pages, before):
    """The listed pages have their bounds, the others what they had."""
    codes, exps = bounds.codes.cpu().numpy(), bounds.exps.cpu().numpy()
    x = page_values(cache, pages)
    for i, page in enumerate(pages):
        for h in range(cache.n_kv_heads):
            want, e = oracle.bounds_ref(x[i, h])
            assert exps[page, h] == e + 127, (page, h)
            assert np.array_equal(codes[page, h], want), (page, h)
    rest = np.setdiff1d(np.arange(cache.n_pages), pages)
    assert np.array_equal(codes[rest], before[0].cpu().numpy()[rest])
    assert np.array_equal(exps[rest], before[1].cpu().numpy()[rest])


def expected_choice(batch, bounds, table, q, q_len, kv_len):
    s, sp = batch.shape, batch.sparse_shape
    group, out = s.n_heads // s.n_kv_heads, []
    codes, exps = bounds.codes.cpu().numpy(), bounds.exps.cpu().numpy().astype(int) - 127
    x, row = q.double().cpu().numpy().reshape(-1, s.n_kv_heads, group, s.head_dim), 0
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        for i in range(n):
            own = (m - n + i) // s.page_tokens
            ids = table[b, :max(own, 0) + 1]
            out.append([[int(ids[j]) for j in oracle.select_ref(x[row, h], codes[ids, h], exps[ids, h], own, sp.select,
                                                               sp.first, sp.last)] if own >= 0 else []
                        for h in range(s.n_kv_heads)])
            row += 1
    want = np.full((row, s.n_kv_heads, sp.select), -1, np.int64)
    for r, heads in enumerate(out):
        for h, ids in enumerate(heads):
            want[r, h, :len(ids)] = ids
    return want


def expected_out(cache, q, chosen, q_len, kv_len, heads, scale):
    """(out, tolerance) over the chosen pages' tokens, of which the last page's are seen up to the row's own."""
    group, page, d, hk = heads // cache.n_kv_heads, cache.page_tokens, cache.head_dim, cache.n_kv_heads
    out, tol = np.zeros((2, len(chosen), heads, d))
    tol += 1e-37  # of rows that see nothing, as in test_gpu_attn.py
    k, v = (values(t, e).astype(np.float64) for t, e in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    qq = q.double().cpu().numpy().reshape(-1, heads, d)
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(q_len, kv_len)] + [np.zeros(0, int)]).astype(int)
    for r in range(len(chosen)):
        for h in range(hk):
            ids = chosen[r, h][chosen[r, h] >= 0]
            if not len(ids):
                continue
            n = (len(ids) - 1) * page + pos[r] % page + 1
            kk, vv = (x[ids, h].reshape(-1, d)[:n, None] for x in (k, v))
            mine = slice(h * group, (h + 1) * group)
            o, spread, reach = oracle.attend_ref(qq[r:r + 1, mine], kk, vv, n, 0, 0, scale)
            slack = U + 2 * ((d + 4) * 2.0 ** -24 * reach[..., None] + 2.0 ** -20)
            err = slack * spread * 1.01 + 2.0 ** -22 * np.abs(o)
            out[r, mine], tol[r, mine] = o[0], (err + U * (np.abs(o) + err) + 1e-37)[0]
    return out, tol


def normal(rng, *size):
    return torch.from_numpy(rng.standard_normal(size).astype(np.float32)).bfloat16().cuda()


def run_case(seqs, heads, kv_heads, dim, page, dtype, select, first=1, last=1, token_major=False, seed=0, attend=True,
             bounded=None, cache=None, q=None):
    rng = np.random.default_rng([seed, heads, dim, page])
    q_len, kv_len = [s[0] for s in seqs], [s[1] for s in seqs]
    pages = int(sum(-(-n // page) for n in kv_len)) + 3
    cache = cache or make_cache(rng, pages, kv_heads, page, dim, dtype, token_major)
    table = make_table(rng, kv_len, page, cache.n_pages)
    rows = sum(q_len)
    q = normal(rng, rows, heads * dim) if q is None else q
    bounds = make_bounds(rng, cache)
    before = bounds.codes.clone(), bounds.exps.clone()
    batch = SparseBatch(cache, heads, select, first, last)
    bounded = [0] * len(seqs) if bounded is None else bounded
    batch.refresh(q_len, kv_len, table, bounded=bounded)
    print(f"case {seqs} heads {heads}/{kv_heads} dim {dim} page {page} {dtype} select {select} {first} {last}", flush=True)
    batch.bounds(bounds)
    torch.cuda.synchronize()
    fresh = [int(table[b, i]) for b in range(len(seqs)) for i in range(bounded[b] // page, kv_len[b] // page)]
    check_bounds(cache, bounds, fresh, before)
    chosen = torch.full((rows + 1, kv_heads, select), 77, dtype=torch.int32, device="cuda")
    batch.select(q, bounds, chosen)
    torch.cuda.synchronize()
    want = expected_choice(batch, bounds, table, q, q_len, kv_len)
    assert np.array_equal(chosen[:rows].cpu().numpy(), want)
    assert (chosen[rows] == 77).all()
    if attend:
        out = torch.full((rows + 1, heads * dim), 7.0, dtype=torch.bfloat16, device="cuda")
        batch.sparse(q, out, dim ** -0.5, chosen)
        torch.cuda.synchronize()
        check(out[:rows], *expected_out(cache, q, want, q_len, kv_len, heads, dim ** -0.5))
        assert (out[rows] == 7).all()
    return batch, cache, bounds, table, q, chosen


SEQS = [(1, 1), (1, 16), (1, 17), (1, 500), (3, 131), (20, 300), (0, 40), (1, 130)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (4, 2), (3, 1), (14, 2), (8, 1), (16, 1)])
def test_groups(heads, kv_heads, dim, dtype):
    run_case(SEQS, heads, kv_heads, dim, 16, dtype, 5, 1, 2)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,select,first,last", [(16, 1, 0, 1), (16, 3, 1, 2), (32, 4, 0, 1), (64, 2, 1, 1), (64, 3, 0, 2),
                                                    (128, 2, 0, 1), (1024, 1, 0, 1), (16, 40, 2, 3), (16, 12, 5, 4)])
def test_pages(page, select, first, last, dtype):
    run_case(SEQS + [(2, 1500), (1, 2100)], 8, 2, 128, page, dtype, select, first, last)
    run_case([(5, 700), (1, 64)], 2, 2, 64, page, dtype, select, first, last, token_major=True)


@pytest.mark.parametrize("heads", [17, 33, 64])
def test_more_heads_than_a_tile(heads):
    run_case([(1, 300), (3, 90)], heads, 1, 64, 16, "bf16", 4)


def test_rows_before_the_first_token():
    *_, chosen = run_case([(5, 2), (3, 0), (40, 20), (1, 1)], 4, 2, 64, 16, "bf16", 3)
    assert (chosen[:3] == -1).all() and (chosen[5:8] == -1).all() and (chosen[8:28] == -1).all()


def test_bounds_of_new_pages_only():
    run_case([(40, 100), (1, 32), (1, 33), (7, 7), (16, 48)], 2, 2, 128, 16, "bf16", 3, bounded=[60, 31, 32, 0, 32], attend=False)
    run_case([(3, 200), (1, 64)], 2, 2, 128, 64, "e4m3", 3, bounded=[130, 64], attend=False)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
def test_bounds_of_every_kind_of_value(dim, dtype):
    """Infinities, NaN of both signs, columns of NaN, borders of exponents, subnormal and huge pages, zeros."""
    rng = np.random.default_rng([dim])
    n, page = 24, 32
    cache = make_cache(rng, n, 2, page, dim, dtype)
    if dtype == "bf16":
        x = torch.from_numpy(rng.standard_normal((n, 2, page, dim)).astype(np.float32))
        for i, size in enumerate((1e-39, 1e-30, 1e30, 1e38, 127.0, 2.0 ** 100)):
            x[i] *= size
        x[6:8].clamp_(-1, 1)
        x[6, :, 0, 0], x[7, :, 3, 5] = 127 / 64, -128 / 64
        x[8] = 0
        x[9, 0, 5, 7], x[9, 1, 5, 7] = float("inf"), float("-inf")
        x[10, 0, 5, 7], x[10, 1, :, 9] = float("nan"), float("nan")
        x[11] = float("nan")
        x[12] = float("inf")
        x[13, 0, :, 3], x[13, 1, 1:, 3] = float("-inf"), float("nan")
        x[14] = x[14].abs()
        x[15] = -x[15].abs()
        x = x.bfloat16().cuda()
        negative = x.view(torch.int16)
        negative[10, 0, 9, 11], negative[10, 0, 9, 12] = -1, -64  # NaN with a sign
        negative[16, 0, 2, 1] = 0x7F81 - 0  # a signalling one
        cache.k.copy_(x)
    else:
        codes = cache.k.view(torch.uint8)
        codes[8] = 0
        codes[10, 0, 5, 7], codes[10, 1, :, 9], codes[11], codes[12, 0, 3, 3] = 0x7F, 0xFF, 0xFF, 0xFF
        cache.k_scale[1], cache.k_scale[2], cache.k_scale[3, :, ::2] = 27, 246, 200
    table = rng.permutation(n).astype(np.int32)[None]
    bounds = make_bounds(rng, cache)
    before = bounds.codes.clone(), bounds.exps.clone()
    batch = SparseBatch(cache, 2, 2).refresh([0], [n * page], table, bounded=[0])
    batch.bounds(bounds)
    torch.cuda.synchronize()
    check_bounds(cache, bounds, list(range(n)), before)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 1024])
@pytest.mark.parametrize("dim,kv_heads,n", [(64, 3, 7), (128, 1, 3), (64, 1, 1), (128, 5, 9)])
def test_bounds_of_pages_that_share_a_wave(dim, kv_heads, n, page, dtype):
    """Numbers of pages and heads that leave the last wave part of them; one page with NaN beside others."""
    rng = np.random.default_rng([dim, page, n])
    cache = make_cache(rng, n + 2, kv_heads, page, dim, dtype, token_major=n == 7)
    table = rng.permutation(n + 2).astype(np.int32)[None, :n]
    codes = cache.k.view(torch.uint8 if dtype == "e4m3" else torch.int16)
    codes[int(table[0, n // 2]), 0, 5, 7] = 0x7F if dtype == "e4m3" else 0x7FC0
    bounds = make_bounds(rng, cache)
    before = bounds.codes.clone(), bounds.exps.clone()
    batch = SparseBatch(cache, kv_heads, 2).refresh([0], [n * page], table, bounded=[0])
    batch.bounds(bounds)
    torch.cuda.synchronize()
    check_bounds(cache, bounds, [int(p) for p in table[0]], before)


@pytest.mark.parametrize("dim,page,dtype", [(128, 64, "bf16"), (64, 16, "e4m3"), (64, 16, "bf16"), (128, 16, "e4m3"),
                                            (64, 32, "e4m3")])
def test_bounds_of_many_pages(dim, page, dtype):
    """A call of 160 MB of keys and more: the same pages many times over."""
    rng = np.random.default_rng([dim, page])
    n, hk = 20, 8
    each = page * hk * dim * (2 if dtype == "bf16" else 1)
    cache = make_cache(rng, n, hk, page, dim, dtype)
    table = np.resize(rng.permutation(n).astype(np.int32), (1, 165000000 // each))
    bounds = make_bounds(rng, cache)
    before = bounds.codes.clone(), bounds.exps.clone()
    batch = SparseBatch(cache, hk, 2).refresh([0], [table.shape[1] * page], table, bounded=[0])
    batch.bounds(bounds)
    torch.cuda.synchronize()
    check_bounds(cache, bounds, list(range(n)), before)


def test_choice_of_every_kind_of_query():
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.standard_normal((12, 4 * 64)).astype(np.float32))
    for i, size in enumerate((1e-39, 1e-30, 1e30, 3e38)):
        q[i] *= size
    q[4] = 0
    q[5, 3], q[5, 130] = float("inf"), float("-inf")
    q[6, 3], q[6, 70:75] = float("nan"), float("nan")
    q[7] = float("nan")
    q[8, ::2] = 127 / 64
    q[9] = q[9].abs()
    q[10] = -q[10].abs()
    run_case([(12, 400)], 4, 2, 64, 16, "bf16", 5, q=q.bfloat16().cuda(), attend=False)


def test_equals_go_to_the_earlier_page():
    rng = np.random.default_rng(4)
    cache = make_cache(rng, 70, 1, 16, 64, "bf16", fill=1.0)
    for seqs, select in (([(1, 1000)], 7), ([(20, 1010)], 9), ([(1, 1000)], 62)):
        run_case(seqs, 2, 1, 64, 16, "bf16", select, cache=cache, attend=False)
    # two values of score only
    cache.k.copy_(torch.from_numpy(rng.integers(0, 2, (70, 1, 1, 1)).astype(np.float32)).bfloat16().cuda().expand(70, 1, 16, 64))
    for select in (4, 20, 33, 50):
        run_case([(1, 1000), (6, 80)], 2, 1, 64, 16, "bf16", select, cache=cache, attend=False)


@pytest.mark.parametrize("heads,kv_heads,new", [(2, 1, 1), (4, 2, 3), (20, 1, 1)])
def test_pages_past_what_lds_holds(heads, kv_heads, new):
    """Scores go through memory."""
    rng = np.random.default_rng(5)
    n = 13000
    cache = make_cache(rng, n + 8, kv_heads, 16, 64, "bf16")
    table = rng.permutation(n + 8).astype(np.int32)[None, :n]
    q = normal(rng, new, heads * 64)
    bounds = KvBounds.empty(cache)
    batch = SparseBatch(cache, heads, 100).refresh([new], [16 * n - 3], table, bounded=[0])
    assert batch.sparse_info.item_tokens == 1 and batch.sparse_info.max_scored > 12288
    batch.bounds(bounds)
    chosen, out = batch.empty_selected(), torch.zeros_like(q)
    batch.select(q, bounds, chosen)
    batch.sparse(q, out, 0.125, chosen)
    torch.cuda.synchronize()
    codes, exps = bounds.codes.cpu().numpy(), bounds.exps.cpu().numpy().astype(int) - 127
    for page in rng.integers(0, n, 20):
        want, e = oracle.bounds_ref(page_values(cache, [table[0, page]])[0, 0])
        assert np.array_equal(codes[table[0, page], 0], want) and exps[table[0, page], 0] == e
    want = expected_choice(batch, bounds, table, q, [new], [16 * n - 3])
    assert np.array_equal(chosen.cpu().numpy(), want)
    check(out, *expected_out(cache, q, want, [new], [16 * n - 3], heads, 0.125))


@pytest.mark.parametrize("heads,kv_heads,new,kv", [(8, 8, 70, 16 * 2400), (2, 2, 300, 16 * 2500), (6, 1, 1, 16 * 2050)])
def test_many_pages(heads, kv_heads, new, kv):
    """Tokens on either side of what LDS holds of one, and of several at once."""
    rng = np.random.default_rng(kv)
    n = kv // 16
    cache = make_cache(rng, n, kv_heads, 16, 64, "bf16")
    table, q = rng.permutation(n).astype(np.int32)[None], normal(rng, new, heads * 64)
    bounds = KvBounds.empty(cache)
    batch = SparseBatch(cache, heads, 40, 2, 3).refresh([new], [kv], table, bounded=[0])
    batch.bounds(bounds)
    chosen = batch.empty_selected()
    batch.select(q, bounds, chosen)
    torch.cuda.synchronize()
    assert np.array_equal(chosen.cpu().numpy(), expected_choice(batch, bounds, table, q, [new], [kv]))


def test_more_items_than_a_launch_takes():
    """16500 tokens of 128 kv heads: two launches, the same choice for the same query."""
    rng = np.random.default_rng(11)
    rows, some = 16500, 12
    cache = make_cache(rng, 8, 128, 16, 64, "bf16")
    table = np.tile(rng.permutation(8).astype(np.int32)[:5], (rows, 1))
    few = normal(rng, some, 128 * 64)
    q = few.repeat(rows // some, 1)
    bounds = KvBounds.empty(cache)
    batch = SparseBatch(cache, 128, 3).refresh([1] * rows, [75] * rows, table, bounded=[0] + [75] * (rows - 1))
    assert batch.sparse_info.n_items == rows
    batch.bounds(bounds)
    chosen = batch.empty_selected()
    chosen.fill_(-2)
    batch.select(q, bounds, chosen)
    torch.cuda.synchronize()
    assert torch.equal(chosen, chosen[:some].repeat(rows // some, 1, 1))
    want = expected_choice(batch, bounds, table, few, [1] * some, [75] * some)
    assert np.array_equal(chosen[:some].cpu().numpy(), want)


def test_split_contexts():
    batch, *_ = run_case([(1, 3000), (2, 1500), (1, 40)], 8, 2, 128, 64, "bf16", 30)
    assert batch.sparse_info.n_merge > 0
    run_case([(1, 3000), (2, 1500)], 4, 2, 64, 16, "e4m3", 120, 2, 3)


# more than 2048 items: a wave to each
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,page,heads,kv_heads,n", [(128, 16, 8, 8, 260), (64, 32, 8, 4, 530), (128, 64, 14, 2, 1030),
                                                       (64, 16, 20, 1, 1030)])
def test_many_tokens(dim, page, heads, kv_heads, n, dtype):
    batch, *_ = run_case([(n, n + 90), (1, 1), (4, 2), (1, 37)], heads, kv_heads, dim, page, dtype, 3)
    assert batch.sparse_info.n_work * kv_heads >= 2048
    run_case([(n, n), (1, 300)], heads, kv_heads, dim, page, dtype, 4, 0, 2, token_major=True)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_many_tokens_and_long_ones(dtype):
    """Items that are split among many that are not."""
    batch, *_ = run_case([(1100, 1100)] + [(1, 4000)] * 3, 2, 2, 64, 16, dtype, 200)
    assert batch.sparse_info.n_merge > 0 and batch.sparse_info.n_work * 2 >= 2048


def test_what_is_not_seen_does_not_matter():
    """NaN and infinities in pages that are not chosen, in unused pages, and past the row in its own page."""
    rng = np.random.default_rng(6)
    batch, cache, bounds, table, q, chosen = run_case([(3, 330), (1, 200)], 4, 2, 64, 16, "bf16", 4)
    out, again = torch.zeros_like(q), torch.zeros_like(q)
    batch.sparse(q, out, 0.125, chosen)
    used = chosen.cpu().numpy()
    for h in range(2):
        for p in range(cache.n_pages):
            if p not in used[:, h]:
                cache.k[p, h], cache.v[p, h] = float("nan"), float("inf")
    cache.k[int(table[0, 20]), :, 10:] = float("nan")
    cache.v[int(table[1, 12]), :, 8:] = float("nan")
    batch.sparse(q, again, 0.125, chosen)
    torch.cuda.synchronize()
    assert torch.isfinite(again).all() and torch.equal(out, again)


def test_all_pages_selected_is_the_dense_attention():
    rng = np.random.default_rng(7)
    seqs = [(1, 500), (9, 70), (1, 1)]
    batch, cache, bounds, table, q, chosen = run_case(seqs, 8, 2, 128, 16, "bf16", 40)
    dense = torch.zeros_like(q)
    batch.attn(q, dense, 128 ** -0.5)
    torch.cuda.synchronize()
    want, tol = expected_out(cache, q, chosen[:11].cpu().numpy(), *zip(*seqs), 8, 128 ** -0.5)
    check(dense, want, tol)


def test_same_bits_again_and_in_another_batch():
    batch, cache, bounds, table, q, chosen = run_case(SEQS, 8, 2, 128, 16, "bf16", 5, 1, 2)
    rows = q.shape[0]
    out, again = torch.zeros_like(q), torch.zeros_like(q)
    batch.sparse(q, out, 0.1, chosen)
    for _ in range(3):
        other = torch.zeros_like(chosen)
        batch.select(q, bounds, other)
        batch.sparse(q, again, 0.1, other)
        torch.cuda.synchronize()
        assert torch.equal(other[:rows], chosen[:rows]) and torch.equal(out, again)
    one = SparseBatch(cache, 8, 5, 1, 2).refresh([1], [500], table[3:4])
    other = one.empty_selected()
    one.select(q[3:4], bounds, other)
    torch.cuda.synchronize()
    assert torch.equal(other[0], chosen[3])


def test_pages_beyond_32_bit_offsets():
    rng = np.random.default_rng(8)
    stride, n = 1 << 28, 10
    pool = [torch.zeros(stride * (n - 1) + 2 * 16 * 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k, v = (p.as_strided((n, 2, 16, 64), (stride, 16 * 64, 64, 1)) for p in pool)
    for t in (k, v):
        t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
    run_case([(2, 110)], 4, 2, 64, 16, "bf16", 3, cache=KvCache(k, v))


def test_a_step_on_a_stream_and_in_a_graph():
    """Write, bounds, select and attention of one step, replayed with other inputs."""
    rng = np.random.default_rng(9)
    cache = make_cache(rng, 80, 2, 16, 128, "bf16")
    q_len, kv_len = [1, 1, 20], [700, 96, 60]
    table = make_table(rng, kv_len, 16, 80)
    x, q = torch.randn(2, 22, 256, device="cuda"), torch.randn(22, 512, device="cuda")
    qo = torch.zeros(22, 512, dtype=torch.bfloat16, device="cuda")
    out, bounds = torch.zeros_like(qo), make_bounds(rng, cache)
    batch, side = SparseBatch(cache, 4, 3), torch.cuda.Stream()
    batch.refresh(q_len, kv_len, table, bounded=[0, 0, 0])
    batch.bounds(bounds)
    side.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        batch.write(x[0], x[1], q, qo, stream=stream)
        batch.bounds(bounds, stream=stream)
        batch.select(qo, bounds, chosen, stream=stream)
        batch.sparse(qo, out, 0.1, chosen, stream=stream)

    def verify():
        torch.cuda.synchronize()
        want = expected_choice(batch, bounds, table, qo, q_len, kv_len)
        assert np.array_equal(chosen.cpu().numpy(), want)
        for b in range(3):  # what the pages hold now
            for i in range((kv_len[b] - q_len[b]) // 16, kv_len[b] // 16):
                codes, e = oracle.bounds_ref(page_values(cache, [table[b, i]])[0, 1])
                assert np.array_equal(bounds.codes[int(table[b, i]), 1].cpu().numpy(), codes)
        check(out, *expected_out(cache, qo, want, q_len, kv_len, 4, 0.1))
    batch.refresh(q_len, kv_len, table, stream=side)
    chosen = batch.empty_selected()
    step(side)
    verify()
    batch.refresh(q_len, kv_len, table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        g = torch.Generator().manual_seed(i)
        x.copy_(torch.randn(x.shape, generator=g))
        q.copy_(torch.randn(q.shape, generator=g))
        chosen.zero_()
        out.zero_()
        graph.replay()
        verify()


def test_batch_refuses():
    cache = KvCache.empty(10, 2, 16, 64)
    batch = SparseBatch(cache, 4, 3)
    bounds, q = KvBounds.empty(cache), torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError):
        batch.bounds(bounds)
    batch.refresh([3], [20], np.array([[1, 2]], np.int32))
    chosen = batch.empty_selected()
    other = KvBounds.empty(KvCache.empty(11, 2, 16, 64))
    for call in (lambda: batch.bounds(other), lambda: batch.select(q, other, chosen), lambda: batch.select(q[:2], bounds, chosen),
                 lambda: batch.select(q, bounds, chosen[:2]), lambda: batch.select(q, bounds, chosen.long()),
                 lambda: batch.select(q, bounds, chosen.cpu()), lambda: batch.select(q, bounds, chosen[:, :1]),
                 lambda: batch.sparse(q, q.clone(), 0.1, chosen.transpose(1, 2)), lambda: batch.sparse(q.half(), q, 0.1, chosen),
                 lambda: batch.sparse(q, q.clone(), 0.1, chosen, cache=KvCache.empty(11, 2, 16, 64)),
                 lambda: KvBounds(cache, bounds.codes.cpu(), bounds.exps), lambda: KvBounds(cache, bounds.codes[:9], bounds.exps),
                 lambda: KvBounds(cache, bounds.codes, bounds.exps.int()), lambda: KvBounds(cache, bounds.codes.float(), bounds.exps)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(hl.LoraError):
        batch.sparse(q, q.clone(), 0.0, chosen)
    with pytest.raises(hl.LoraError):
        SparseBatch(KvCache.empty(10, 2, 8, 64), 4, 3).refresh([1], [20], np.array([[1, 2, 3]], np.int32))


def test_choice_is_as_good_as_keys_that_stand_out():
    """A key that matches the query is found wherever its page lies."""
    rng = np.random.default_rng(10)
    cache = make_cache(rng, 64, 1, 16, 128, "bf16")
    table = rng.permutation(64).astype(np.int32)[None, :60]
    q = normal(rng, 1, 256)
    bounds = KvBounds.empty(cache)
    batch = SparseBatch(cache, 2, 4).refresh([1], [60 * 16], table, bounded=[0])
    for place in (1, 17, 40, 58):
        cache.k.copy_(torch.from_numpy(rng.standard_normal(cache.k.shape).astype(np.float32)))
        cache.k[int(table[0, place]), 0, 7] = 4 * q[0, 128:]
        batch.bounds(bounds)
        chosen = batch.empty_selected()
        batch.select(q, bounds, chosen)
        assert int(table[0, place]) in chosen[0, 0].tolist()


def test_values_of_sequences_come_back():
    """tokens() of the shared helpers agrees with what the choice addresses."""
    rng = np.random.default_rng(11)
    batch, cache, bounds, table, q, chosen = run_case([(1, 100)], 2, 2, 64, 16, "e4m3", 9)
    k, _ = tokens(cache, table, 0, 100)
    ids = chosen[0, 0][chosen[0, 0] >= 0].cpu().numpy()
    got = page_values(cache, ids)[:, 0].reshape(-1, 64)[:100]
    assert np.array_equal(got, k[:, 0])
