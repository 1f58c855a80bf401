"""The paged cache's write and read and the attention over it on the GPU,
against the fp64 oracle.

Tolerances.  Attention: with u = 2^-8 (half a bf16 step), the weights are
rounded to bf16 (relative u each, summed as rounded, so an output moves by at
most u times the weighted spread of v about it), the scores carry fp32
rounding: a dot product of dim terms and its scaling err by at most (dim + 4) *
2^-24 of the sum of |terms| (`reach`), twice (numerator and sum), the base-2
exponential and its argument by 2^-20; the output is rounded once more.  The
write's bf16: one rounding, of a turn that errs by 3 * 2^-24 of its terms.
Quantised values without a turn and everything read back are exact."""
import numpy as np
import pytest
import torch

import heterogeneous_adapter_batching_amd as hl
import oracle
from heterogeneous_adapter_batching_amd.attention import AttnBatch, KvCache, rope_table

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def make_cache(rng, pages, kv_heads, page, dim, dtype, token_major=False, fill=None):
    """A cache of random values on the GPU, its values as float64 [pages, kv_heads, page, dim]."""
    shape = (pages, page, kv_heads, dim) if token_major else (pages, kv_heads, page, dim)
    order = (0, 2, 1, 3) if token_major else (0, 1, 2, 3)

    def one():
        x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
        if fill is not None:
            x.fill_(fill)
        return (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn) if dtype == "e4m3" else x.bfloat16()
    k, v = one().cuda().permute(order), one().cuda().permute(order)
    if dtype == "bf16":
        return KvCache(k, v)
    ke, ve = (torch.from_numpy(rng.integers(118, 123, (pages, kv_heads, page)).astype(np.uint8)).cuda() for _ in "kv")
    return KvCache(k, v, ke, ve)


def values(codes, exps):
    x = codes.float().cpu().double().numpy()
    return x if exps is None else x * 2.0 ** (exps.cpu().numpy().astype(np.float64)[..., None] - 127)


def tokens(cache, table, b, n):
    """(k, v) of sequence b's first n tokens, float64 [n, kv_heads, dim]."""
    out = []
    for codes, exps in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        need = -(-n // cache.page_tokens)
        at = torch.from_numpy(table[b, :need].astype(np.int64)).cuda()
        x = values(codes[at], None if exps is None else exps[at])
        out.append(x.transpose(0, 2, 1, 3).reshape(-1, cache.n_kv_heads, cache.head_dim)[:n])
    return out


def make_table(rng, kv_len, page, pages):
    need = [-(-int(n) // page) for n in kv_len]
    assert sum(need) <= pages
    tab = np.zeros((len(kv_len), max([1] + need)), np.int32)
    perm, at = rng.permutation(pages), 0
    for i, n in enumerate(need):
        tab[i, :n] = perm[at:at + n]
        at += n
    return tab


def expected(cache, table, q, q_len, kv_len, heads, window, sinks, scale, kv=None):
    """(out, tolerance) [rows, heads, dim] in fp64."""
    out, tol, row = [], [], 0
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        k, v = tokens(cache, table, b, int(m)) if kv is None else kv[b]
        qq = q[row:row + n].double().cpu().numpy().reshape(n, heads, cache.head_dim)
        o, spread, reach = oracle.attend_ref(qq, k, v, int(m), window, sinks, scale)
        slack = U + 2 * ((cache.head_dim + 4) * 2.0 ** -24 * reach[..., None] + 2.0 ** -20)
        err = slack * spread * 1.01 + 2.0 ** -22 * np.abs(o)
        out.append(o)
        tol.append(err + U * (np.abs(o) + err) + 1e-37)
        row += n
    return np.concatenate(out), np.concatenate(tol)


def check(got, want, tol):
    got = got.double().cpu().numpy().reshape(want.shape)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - want) / tol) if want.size else 0.0
    assert worst <= 1.0, worst


def run_case(seqs, heads, kv_heads, dim, page, dtype, window=0, sinks=0, token_major=False, scale=None, seed=0):
    rng = np.random.default_rng([seed, heads, dim, page])
    q_len, kv_len = np.array([s[0] for s in seqs]), np.array([s[1] for s in seqs])
    pages = int(sum(-(-int(n) // page) for n in kv_len)) + 3
    cache = make_cache(rng, pages, kv_heads, page, dim, dtype, token_major)
    table = make_table(rng, kv_len, page, pages)
    rows = int(q_len.sum())
    q = torch.from_numpy(rng.standard_normal((rows, heads * dim)).astype(np.float32)).bfloat16().cuda()
    out = torch.full_like(q, float("nan"))
    scale = dim ** -0.5 if scale is None else scale
    batch = AttnBatch(cache, heads, window, sinks).refresh(q_len, kv_len, table)
    print(f"case {seqs} heads {heads}/{kv_heads} dim {dim} page {page} {dtype} window {window}/{sinks}", flush=True)
    batch.attn(q, out, scale)
    torch.cuda.synchronize()
    want, tol = expected(cache, table, q, q_len, kv_len, heads, window, sinks, scale)
    check(out, want, tol)
    return batch, cache, table, q, out


# (new tokens, cached tokens with them) of each sequence
DECODE = [(1, 1), (1, 2), (1, 31), (1, 32), (1, 33), (1, 64), (1, 65), (1, 200)]
CHUNKS = [(5, 5), (17, 17), (3, 70), (40, 129), (1, 64), (0, 9), (130, 300)]
LONG = [(1, 3000), (2, 1500), (33, 2000)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,page", [(4, 4, 16), (8, 1, 1), (7, 1, 64), (6, 2, 8)])
def test_single_tokens(heads, kv_heads, page, dim, dtype):
    run_case(DECODE, heads, kv_heads, dim, page, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,page", [(2, 2, 16), (8, 1, 32), (3, 1, 1), (14, 2, 128)])
def test_chunks(heads, kv_heads, page, dim, dtype):
    run_case(CHUNKS, heads, kv_heads, dim, page, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("seqs", [DECODE, CHUNKS])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (33, 1), (64, 4), (50, 70), (4096, 4)])
def test_window_and_sinks(window, sinks, seqs, dtype):
    run_case(seqs, 4, 2, 64 if window == 33 else 128, 16, dtype, window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 4)])
def test_split_contexts(window, sinks, dtype):
    batch, *_ = run_case(LONG, 8, 2, 128, 64, dtype, window, sinks)
    assert batch.info.n_merge > 0
    run_case(LONG, 4, 2, 64, 16, dtype, window, sinks)


@pytest.mark.parametrize("heads,kv_heads", [(64, 1), (5, 1), (33, 1), (32, 32)])
def test_groups(heads, kv_heads):
    run_case([(1, 77), (3, 100), (2, 2)], heads, kv_heads, 64, 16, "bf16")


def test_many_heads_to_a_kv_head():
    run_case([(1, 77), (2, 100), (1, 2100)], 300, 1, 64, 16, "bf16")


# row tiles over 32 tiles of tokens and more
OVER = [(70, 2300), (300, 2433), (1, 40), (33, 33)]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,window,sinks", [(1, 0, 0), (16, 0, 0), (64, 2200, 5), (4, 2050, 130)])
def test_chunks_over_long_contexts(page, window, sinks, dim, dtype):
    batch, cache, table, q, out = run_case(OVER, 4, 1, dim, page, dtype, window, sinks)
    assert batch.info.n_work[hl.LORA_ATTN_PAIR] > 0
    again = torch.zeros_like(out)
    for _ in range(2):
        batch.attn(q, again, dim ** -0.5)
        torch.cuda.synchronize()
        assert torch.equal(out, again)


def test_long_contexts_of_a_token_major_cache():
    batch, *_ = run_case(OVER, 6, 2, 128, 32, "bf16", token_major=True)
    assert batch.info.n_work[hl.LORA_ATTN_PAIR] > 0


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 16])
def test_values_that_no_row_sees_over_long_contexts(page, dtype):
    """As the test of masked values below, for row tiles of the kernel for long contexts."""
    rng = np.random.default_rng([page, 4])
    n, kv, window, sinks, dim, heads = 100, 2600, 2100, 70, 128, 4
    pages = -(-kv // page) + 2
    cache = make_cache(rng, pages, 1, page, dim, dtype)
    table = make_table(rng, [kv], page, pages)
    kvs = [tokens(cache, table, 0, kv)]
    hidden = np.arange(sinks, kv - n - window + 1)
    assert len(hidden) > 300
    for t in (cache.k, cache.v):
        at = (torch.from_numpy(table[0][hidden // page].astype(np.int64)).cuda(), 0,
              torch.from_numpy(hidden % page).cuda())
        if dtype == "e4m3":
            t.view(torch.uint8)[at] = 0x7F
        else:
            t[at] = float("nan")
    q = torch.from_numpy(rng.standard_normal((n, heads * dim)).astype(np.float32)).bfloat16().cuda()
    out = torch.zeros_like(q)
    batch = AttnBatch(cache, heads, window, sinks).refresh([n], [kv], table)
    assert batch.info.n_work[hl.LORA_ATTN_PAIR] > 0
    batch.attn(q, out, 0.09)
    torch.cuda.synchronize()
    check(out, *expected(cache, table, q, [n], [kv], heads, window, sinks, 0.09, kvs))
    last = cache.v[int(table[0, (kv - 1) // page]), :, (kv - 1) % page]  # only the last new token sees it
    (last.view(torch.uint8) if dtype == "e4m3" else last).fill_(0x7F if dtype == "e4m3" else float("nan"))
    batch.attn(q, out, 0.09)
    torch.cuda.synchronize()
    check(out[:n - 1], *(x[:n - 1] for x in expected(cache, table, q, [n], [kv], heads, window, sinks, 0.09, kvs)))
    assert torch.isnan(out[n - 1]).all()


def test_token_major_cache_and_strided_rows():
    run_case(CHUNKS, 4, 2, 128, 16, "bf16", token_major=True)
    rng = np.random.default_rng(9)
    cache = make_cache(rng, 40, 2, 16, 128, "e4m3", token_major=True)
    q_len, kv_len = [20, 1], [100, 300]
    table = make_table(rng, kv_len, 16, 40)
    wide = torch.from_numpy(rng.standard_normal((23, 4 * 128 + 64)).astype(np.float32)).bfloat16().cuda()
    into = torch.full((25, 4 * 128 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    q, out = wide[:, 32:32 + 512], into[:, 8:8 + 512]
    batch = AttnBatch(cache, 4).refresh(q_len, kv_len, table)
    batch.attn(q, out, 0.1)
    torch.cuda.synchronize()
    check(out[:21], *expected(cache, table, q[:21], q_len, kv_len, 4, 0, 0, 0.1))
    assert (into[:, :8] == 7).all() and (into[:, 520:] == 7).all() and (into[21:] == 7).all()


def test_rows_that_see_nothing_are_zero():
    """More new tokens than the cache holds: the first rows come before token 0."""
    rng = np.random.default_rng(2)
    cache = make_cache(rng, 8, 2, 16, 64, "bf16")
    q_len, kv_len = [4, 3, 40, 1], [2, 0, 3, 0]
    table = make_table(rng, kv_len, 16, 8)
    q = torch.from_numpy(rng.standard_normal((48, 256)).astype(np.float32)).bfloat16().cuda()
    out = torch.full_like(q, float("nan"))
    AttnBatch(cache, 4).refresh(q_len, kv_len, table).attn(q, out, 0.125)
    torch.cuda.synchronize()
    check(out, *expected(cache, table, q, q_len, kv_len, 4, 0, 0, 0.125))
    assert (out[:2] == 0).all() and (out[4:7] == 0).all() and (out[7:44] == 0).all() and (out[47] == 0).all()


def test_large_and_equal_scores():
    run_case([(1, 300), (20, 150)], 4, 2, 128, 16, "bf16", scale=3.0)     # a few weights dominate
    run_case([(1, 300), (20, 150)], 4, 2, 128, 16, "bf16", scale=1e-6)    # all weights alike
    rng = np.random.default_rng(5)
    cache = make_cache(rng, 12, 1, 16, 64, "bf16", fill=-3e4)
    table = make_table(rng, [150], 16, 12)
    q = torch.full((1, 64), 300.0, dtype=torch.bfloat16, device="cuda")   # scores near -6e8: none underflows to an empty row
    out = torch.zeros_like(q)
    AttnBatch(cache, 1).refresh([1], [150], table).attn(q, out, 1.0)
    assert torch.equal(out, torch.full_like(out, -3e4))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,n", [(2, 1), (2, 6), (4, 70)])
def test_values_that_no_row_sees_do_not_matter(heads, n, dtype):
    """Infinities and NaN past the end, between the sinks and the window, and in later new tokens."""
    rng = np.random.default_rng([heads, n])
    page, window, sinks, kv = 16, 90, 5, 400
    cache = make_cache(rng, 30, 2, page, 64, dtype)
    table = make_table(rng, [kv], page, 30)
    kvs = [tokens(cache, table, 0, kv)]
    nan = 0x7F if dtype == "e4m3" else None

    def poison(t, i, value):
        at = t[int(table[0, i // page]), :, i % page]
        if nan is None:
            at.fill_(value)
        else:
            at.view(torch.uint8).fill_(nan)
    for t in (cache.k, cache.v):
        used = torch.zeros(30, dtype=torch.bool)
        used[torch.from_numpy(table[0].astype(np.int64))] = True
        (t.view(torch.uint8) if nan else t)[~used.cuda()] = nan if nan else float("nan")
        for i in range(kv, len(table[0]) * page):
            poison(t, i, float("inf"))
        for i in range(sinks, kv - n - window + 1):
            poison(t, i, float("nan") if i % 3 else float("-inf"))
    q = torch.from_numpy(rng.standard_normal((n, heads * 64)).astype(np.float32)).bfloat16().cuda()
    out = torch.zeros_like(q)
    batch = AttnBatch(cache, heads, window, sinks).refresh([n], [kv], table)
    batch.attn(q, out, 0.2)
    torch.cuda.synchronize()
    check(out, *expected(cache, table, q, [n], [kv], heads, window, sinks, 0.2, kvs))
    if n > 1:  # the last new token: every row before it stays as it was, its own is not finite
        before = out.clone()
        poison(cache.k, kv - 1, float("nan"))
        poison(cache.v, kv - 1, float("inf"))
        batch.attn(q, out, 0.2)
        torch.cuda.synchronize()
        check(out[:n - 1], *(x[:n - 1] for x in expected(cache, table, q, [n], [kv], heads, window, sinks, 0.2, kvs)))
        assert not torch.isfinite(out[n - 1]).any()
        assert torch.isfinite(before).all()


def test_same_bits_again_and_in_another_batch():
    batch, cache, table, q, out = run_case(LONG + CHUNKS, 8, 2, 128, 64, "bf16")
    again = torch.zeros_like(out)
    for _ in range(3):
        batch.attn(q, again, 128 ** -0.5)
        torch.cuda.synchronize()
        assert torch.equal(out, again)


def test_pages_beyond_32_bit_offsets():
    """Pages half a gibi-element apart: the last ones start past 2^32 bytes and 2^31 elements."""
    rng = np.random.default_rng(8)
    stride, pages = 1 << 28, 10
    pool = [torch.empty(stride * (pages - 1) + 2 * 16 * 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k, v = (p.as_strided((pages, 2, 16, 64), (stride, 16 * 64, 64, 1)) for p in pool)
    for t in (k, v):
        t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
    cache = KvCache(k, v)
    table = np.array([[9, 8, 0], [7, 1, 2]], np.int32)
    q = torch.from_numpy(rng.standard_normal((11, 256)).astype(np.float32)).bfloat16().cuda()
    out = torch.zeros_like(q)
    batch = AttnBatch(cache, 4).refresh([1, 10], [48, 40], table)
    batch.attn(q, out, 0.125)
    torch.cuda.synchronize()
    check(out, *expected(cache, table, q, [1, 10], [48, 40], 4, 0, 0, 0.125))
    new = torch.from_numpy(rng.standard_normal((2, 11, 128)).astype(np.float32)).cuda()
    batch.write(new[0], new[1])
    ko, vo = (torch.zeros(88, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    batch.read(ko, vo)
    for got, x in ((ko, new[0]), (vo, new[1])):
        assert torch.equal(got[47], x[0].bfloat16()) and torch.equal(got[78:88], x[1:].bfloat16())


def test_other_streams_and_graphs():
    rng = np.random.default_rng(6)
    cache = make_cache(rng, 80, 2, 16, 128, "bf16")
    q_len, kv_len = [1, 1, 9], [700, 90, 60]
    table = make_table(rng, kv_len, 16, 80)
    q = torch.from_numpy(rng.standard_normal((11, 512)).astype(np.float32)).bfloat16().cuda()
    new = torch.from_numpy(rng.standard_normal((2, 11, 256)).astype(np.float32)).cuda()
    out, qo = torch.zeros_like(q), torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    batch = AttnBatch(cache, 4)
    with torch.cuda.stream(side):
        batch.refresh(q_len, kv_len, table)
        batch.write(new[0], new[1], q.float(), qo)
        batch.attn(qo, out, 0.1)
    side.synchronize()
    assert torch.equal(qo, q)
    check(out, *expected(cache, table, q, q_len, kv_len, 4, 0, 0, 0.1))

    q32 = q.float()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        write = batch.prepare_write(new[0], new[1], q32, qo)
        attn = batch.prepare_attn(qo, out, 0.1)
        write()
        attn()
    for i in range(4):
        new.copy_(torch.randn(new.shape, generator=torch.Generator().manual_seed(i)))
        q32.copy_(torch.randn(q32.shape, generator=torch.Generator().manual_seed(50 + i)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(out, *expected(cache, table, q32.bfloat16(), q_len, kv_len, 4, 0, 0, 0.1))


def test_one_plan_serves_many_caches_and_refreshes():
    rng = np.random.default_rng(12)
    caches = [make_cache(rng, 200, 2, 16, 64, "bf16") for _ in range(2)]
    batch = AttnBatch(caches[0], 4)
    out = torch.zeros(300, 256, dtype=torch.bfloat16, device="cuda")
    q = torch.from_numpy(rng.standard_normal((300, 256)).astype(np.float32)).bfloat16().cuda()
    runs = [batch.prepare_attn(q, out, 0.1, cache=c) for c in caches]
    with pytest.raises(RuntimeError):
        runs[0]()
    for q_len, kv_len in (([1], [5]), ([200, 1, 1], [260, 1500, 1100]), ([3, 1], [3, 8])):
        table = make_table(rng, kv_len, 16, 200)
        batch.refresh(q_len, kv_len, table)
        for run, cache in zip(runs, caches):
            run()
            torch.cuda.synchronize()
            n = sum(q_len)
            check(out[:n], *expected(cache, table, q[:n], q_len, kv_len, 4, 0, 0, 0.1))


def test_batch_refuses():
    cache = KvCache.empty(10, 2, 16, 64)
    batch = AttnBatch(cache, 4).refresh([3], [20], np.array([[1, 2]], np.int32))
    q = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    for bad in (q.half(), q[:, :128], q.cpu(), torch.zeros(256, 3, dtype=torch.bfloat16, device="cuda").T):
        with pytest.raises(ValueError):
            batch.attn(bad, q, 0.1)
    with pytest.raises(ValueError):
        batch.attn(q[:2], q, 0.1)
    with pytest.raises(ValueError):
        batch.attn(q, q.clone(), 0.1, cache=KvCache.empty(11, 2, 16, 64))
    for scale in (0.0, float("nan")):
        with pytest.raises(hl.LoraError):
            batch.attn(q, q.clone(), scale)
    kv = torch.zeros(3, 128, device="cuda")
    for args in ((kv, kv, q), (kv.half(), kv.half()), (kv, kv.bfloat16()), (kv[:2], kv), (kv, kv, q, torch.zeros_like(q))):
        with pytest.raises(ValueError):
            batch.write(*args)
    with pytest.raises(hl.LoraError):
        batch.write(kv, kv, rope=rope_table(19, 64))
    with pytest.raises(ValueError):
        batch.read(torch.zeros(19, 128, dtype=torch.bfloat16, device="cuda"),
                   torch.zeros(20, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(hl.LoraError) as e:
        batch.refresh([1], [20], np.array([[1, 10]], np.int32))
    assert e.value.code == hl.LORA_EPAGE
    with pytest.raises(RuntimeError):
        batch.attn(q, q.clone(), 0.1)


# ---------------------------------------------------------------- write and read
def write_case(source, dtype, dim, heads, kv_heads, page, rope_dim, seqs, seed=0):
    rng = np.random.default_rng([seed, dim, heads, rope_dim])
    q_len, kv_len = np.array([s[0] for s in seqs]), np.array([s[1] for s in seqs])
    pages = int(sum(-(-int(n) // page) for n in kv_len)) + 2
    cache = make_cache(rng, pages, kv_heads, page, dim, dtype)
    table = make_table(rng, kv_len, page, pages)
    rows = int(q_len.sum())
    x = torch.from_numpy(rng.standard_normal((rows, (heads + 2 * kv_heads) * dim)).astype(np.float32)
                         * 2.0 ** rng.integers(-6, 6, (rows, 1)).astype(np.float32))
    x = x.to(torch.float32 if source == "f32" else torch.bfloat16).cuda()
    q, k, v = x.split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
    q_out = torch.full((rows, heads * dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    rope = rope_table(int(kv_len.max()), rope_dim) if rope_dim else None
    before = [None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    batch = AttnBatch(cache, heads).refresh(q_len, kv_len, table)
    batch.write(k, v, q, q_out, rope)
    torch.cuda.synchronize()
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(q_len, kv_len)])
    seq = np.repeat(np.arange(len(q_len)), q_len)
    if rope_dim:  # the table's own cosines and sines: what is tested is the turn
        t = rope.cpu().double().numpy()[pos.clip(0)]
        angle = np.arctan2(t[:, rope_dim // 2:], t[:, :rope_dim // 2])
    parts = []
    for part, n in ((q, heads), (k, kv_heads), (v, kv_heads)):
        y = part.double().cpu().numpy().reshape(rows, n, dim)
        parts.append((y, oracle.turn_ref(y, angle) if rope_dim and part is not v else y))
    return batch, cache, table, before, pos, seq, q_out, parts


def bf16_tolerance(want, terms):
    # a turn's two products and their sum err by 3 * 2^-24 of the terms (and the cosines, fp32
    # of themselves, by 2^-24); one rounding to bf16
    err = 4 * 2.0 ** -24 * terms
    return err + U * (np.abs(want) + err) + 1e-39


SEQS = [(1, 1), (3, 3), (1, 40), (20, 33), (2, 17)]


@pytest.mark.parametrize("source", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,heads,kv_heads,page,rope_dim",
                         [(128, 8, 2, 16, 128), (64, 3, 3, 1, 64), (128, 4, 1, 8, 48), (64, 5, 1, 64, 0), (128, 7, 1, 32, 0)])
def test_write(dim, heads, kv_heads, page, rope_dim, dtype, source):
    batch, cache, table, before, pos, seq, q_out, parts = write_case(source, dtype, dim, heads, kv_heads, page, rope_dim,
                                                                     SEQS)
    x, want = parts[0]
    terms = np.maximum(np.abs(x), np.abs(np.roll(x, rope_dim // 2, -1)) if rope_dim else 0)
    terms = 2 * np.maximum(terms, np.abs(x).max(-1, keepdims=True) if rope_dim else 0)
    got = q_out.double().cpu().numpy().reshape(want.shape)
    assert np.all(np.abs(got - want) <= bf16_tolerance(want, terms))
    page_of, place = table[seq, pos // page], pos % page
    written = np.zeros(cache.k.shape[:3], bool)
    written[page_of, :, place] = True
    for t, exps, old, old_exps, (x, want) in ((cache.k, cache.k_scale, before[0], before[2], parts[1]),
                                              (cache.v, cache.v_scale, before[1], before[3], parts[2])):
        raw, raw_old = (y.contiguous().view(torch.uint8).cpu().numpy().reshape(*y.shape[:3], -1) for y in (t, old))
        assert np.array_equal(raw[~written], raw_old[~written])
        got = values(t, exps)[page_of, :, place]
        if dtype == "bf16":
            big = 2 * np.abs(x).max(-1, keepdims=True)
            assert np.all(np.abs(got - want) <= bf16_tolerance(want, big))
            continue
        assert np.array_equal(exps.cpu().numpy()[~written], old_exps.cpu().numpy()[~written])
        codes, e = oracle.quantise_ref(want)
        e_got = exps.cpu().numpy()[page_of, :, place].astype(int) - 127
        if not rope_dim or x is want:
            assert np.array_equal(e_got, e) and np.array_equal(raw[page_of, :, place], codes)
            continue
        # a turned row: its power may differ only where its maximum is on the border
        top = np.abs(want).max(-1)
        assert np.all((e_got == e) | (np.abs(top / (448 * 2.0 ** np.minimum(e, e_got)) - 1) < 1e-5))
        step = 2.0 ** (e_got[..., None] - 9.0)  # the least step; half a step of a value is 2^-4 of it
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), step / 2) * (1 + 1e-5) + 1e-6 * np.abs(x).max())


@pytest.mark.parametrize("source", ["f32", "bf16"])
def test_write_quantises_every_kind_of_value(source):
    """Borders between codes, ties, subnormal codes, zeros, infinities and NaN, tiny and huge rows."""
    v = oracle.e4m3_values()[:127]
    base = np.concatenate([v, (v[1:] + v[:-1]) / 2, -v, np.nextafter(v[1:].astype(np.float32), np.float32(0))])
    base = np.resize(base, (len(base) // 128 + 1) * 128)
    rows = [base * 2.0 ** e for e in (0, -100, 50, -30, 7)]
    special = np.zeros((6, 128))
    special[0, :4] = [np.inf, -np.inf, np.nan, 3.0]
    special[1] = 3.3e38
    special[2] = 1e-42
    special[3, 5] = -448.0 * 2.0 ** -100
    special[4] = np.nan
    special[5, 0] = 448.5
    x = np.concatenate([r.reshape(-1, 128) for r in rows] + [special]).astype(np.float32)
    x = torch.from_numpy(x).cuda()
    if source == "bf16":
        x = x.bfloat16()
    n = x.shape[0]
    cache = KvCache.empty(-(-n // 16), 1, 16, 128, torch.float8_e4m3fn)
    table = np.arange(-(-n // 16), dtype=np.int32)[None]
    AttnBatch(cache, 1).refresh([n], [n], table).write(x, x)
    torch.cuda.synchronize()
    codes, e = oracle.quantise_ref(x.double().cpu().numpy())
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert np.array_equal(s.cpu().numpy().reshape(-1)[:n].astype(int) - 127, e)
        got = t.view(torch.uint8).cpu().numpy().reshape(-1, 128)[:n]
        got = np.where(got & 0x7F == 0x7F, 0x7F, got)  # NaN of either sign
        zero = oracle.e4m3_values()[codes] == 0
        assert np.array_equal(got[~zero], codes[~zero]) and np.all(got[zero] & 0x7F == 0)


def test_write_skips_rows_before_the_first_token():
    rng = np.random.default_rng(3)
    cache = make_cache(rng, 4, 1, 16, 64, "bf16")
    old = cache.k.clone()
    x = torch.randn(5, 64, device="cuda")
    q_out = torch.full((5, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = torch.randn(5, 128, device="cuda")
    batch = AttnBatch(cache, 2).refresh([5], [2], np.array([[3]], np.int32))
    batch.write(x, x, q, q_out, rope_table(2, 64))
    torch.cuda.synchronize()
    assert (q_out[:3] == 0).all() and torch.equal(q_out[3], q[3].bfloat16())  # position 0 is not turned
    assert torch.equal(cache.k[3, 0, 0], x[3].bfloat16())
    cache.k[3, 0, :2] = old[3, 0, :2]
    assert torch.equal(cache.k, old)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,kv_heads,page", [(64, 3, 1), (128, 2, 16), (64, 1, 128), (128, 8, 8)])
def test_read_is_exact(dim, kv_heads, page, dtype):
    rng = np.random.default_rng([dim, page])
    kv_len = [1, 0, 17, 128, 200, 0]
    pages = sum(-(-n // page) for n in kv_len) + 1
    cache = make_cache(rng, pages, kv_heads, page, dim, dtype, token_major=page == 16)
    table = make_table(rng, kv_len, page, pages)
    into = [torch.full((sum(kv_len) + 2, kv_heads * dim + 8), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ko, vo = (t[:, :kv_heads * dim] for t in into)
    AttnBatch(cache, kv_heads).refresh([0] * len(kv_len), kv_len, table).read(ko, vo)
    torch.cuda.synchronize()
    row = 0
    for b, n in enumerate(kv_len):
        k, v = tokens(cache, table, b, n)
        for got, want in ((ko, k), (vo, v)):
            assert np.array_equal(got[row:row + n].double().cpu().numpy(), want.reshape(n, kv_heads * dim))
        row += n
    for t in into:
        assert (t[row:] == 7).all() and (t[:, kv_heads * dim:] == 7).all()


def test_read_gives_every_code_at_every_scale():
    cache = KvCache.empty(220, 1, 2, 128, torch.float8_e4m3fn)
    cache.k.view(torch.uint8).copy_(torch.arange(256, dtype=torch.uint8).view(1, 1, 2, 128).expand(220, 1, 2, 128))
    cache.v.copy_(cache.k)
    e = torch.arange(27, 247, dtype=torch.uint8)
    cache.k_scale.copy_(e.view(220, 1, 1).expand(220, 1, 2))
    cache.v_scale.copy_(cache.k_scale)
    ko, vo = (torch.zeros(440, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    AttnBatch(cache, 1).refresh([0], [440], np.arange(220, dtype=np.int32)[None]).read(ko, vo)
    torch.cuda.synchronize()
    want = oracle.e4m3_values()[None] * 2.0 ** (np.arange(27, 247)[:, None] - 127.0)
    for got in (ko, vo):
        assert np.array_equal(got.double().cpu().numpy().reshape(220, 256), want, equal_nan=True)


# ---------------------------------------------------------------- all of it together
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attention_layer_example(dtype):
    """The example's layer against its plain form.  bf16: the base projections,
    the cache, the turned q, the weights and the attention's output are rounded
    once each, by 2^-9 rms at most, and the errors add up over two projections in
    a row: 8 * 2^-9.  An e4m3 value is off by half of 2^-3 of it at most, 2^-4."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    out, held = mod.run(torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16, 8)
    cache_off = 2.0 ** -4 if dtype == "e4m3" else 2 * 2.0 ** -9
    assert held <= cache_off + 2 * 2.0 ** -9
    assert out <= (2 * cache_off if dtype == "e4m3" else 0) + 8 * 2.0 ** -9
