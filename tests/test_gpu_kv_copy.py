"""The copy of a cache's pages on the GPU: the bytes asked for, and no others."""
import numpy as np
import pytest
import torch

import heterogeneous_adapter_batching_amd as hl
from heterogeneous_adapter_batching_amd.attention import KvCache
from heterogeneous_adapter_batching_amd.pages import KvCopy, KvPages
from heterogeneous_adapter_batching_amd.sparse import KvBounds
from test_gpu_attn import make_cache

pytestmark = pytest.mark.gpu


def raw(cache):
    """The cache's tensors as bytes: k, v [pages, heads, tokens, bytes] and scales."""
    k, v = (t.contiguous().view(torch.uint8).reshape(*t.shape[:3], -1) for t in (cache.k, cache.v))
    return [x.clone() for x in (k, v, cache.k_scale, cache.v_scale) if x is not None]


def make_bounds(rng, cache):
    """Bounds of other keys: the largest first."""
    codes = np.sort(rng.integers(-127, 128, (cache.n_pages, cache.n_kv_heads, 2, cache.head_dim)), 2)[:, :, ::-1]
    return KvBounds(cache, torch.from_numpy(codes.astype(np.int8)).cuda(),
                    torch.from_numpy(rng.integers(90, 160, (cache.n_pages, cache.n_kv_heads)).astype(np.uint8)).cuda())


def check(before_src, before_dst, after, src, dst, tokens, page):
    for s, want, got in zip(before_src, before_dst, after):
        want = want.clone()
        for a, b, n in zip(src, dst, tokens):
            want[b, :, :n] = s[a, :, :n]
        assert torch.equal(got, want)


def run_case(pairs, caches, bounds=None, to=None, to_bounds=None, whole=False, seed=0, one_source=False):
    rng = np.random.default_rng([seed, pairs])
    page, n = caches[0].page_tokens, caches[0].n_pages
    if to is None:
        order = rng.permutation(n)
        src, dst = order[:pairs], order[pairs:2 * pairs]
    else:
        src, dst = rng.integers(0, n, pairs), rng.permutation(to[0].n_pages)[:pairs]
    if one_source:
        src = np.full(pairs, src[0])
    tokens = np.full(pairs, page) if whole else rng.integers(0, page + 1, pairs)
    into, into_bounds = to or caches, to_bounds if to else bounds
    before = [(raw(c), raw(d)) for c, d in zip(caches, into)]
    held = [(b.codes.clone(), b.exps.clone(), d.codes.clone(), d.exps.clone()) for b, d in zip(bounds, into_bounds)] \
        if bounds else []
    print(f"copy {pairs} pairs, {len(caches)} caches, page {page}, whole {whole}", flush=True)
    KvCopy(caches, bounds, to, to_bounds).copy(src, dst, None if whole else tokens)
    torch.cuda.synchronize()
    for (s, d), c in zip(before, into):
        check(s, d, raw(c), src, dst, tokens, page)
    for (codes, exps, want, want_exps), d in zip(held, into_bounds or []):
        for a, b, n in zip(src, dst, tokens):
            if n == page:
                want[b], want_exps[b] = codes[a], exps[a]
        assert torch.equal(d.codes, want) and torch.equal(d.exps, want_exps)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,kv_heads,page", [(128, 8, 16), (64, 3, 1), (128, 1, 1), (64, 2, 64), (128, 5, 8), (64, 33, 4),
                                               (128, 2, 1024), (64, 9, 32), (128, 40, 2)])
def test_copy(dim, kv_heads, page, dtype):
    rng = np.random.default_rng([dim, kv_heads, page])
    for pairs, whole in ((1, False), (7, False), (9, True)):
        run_case(pairs, [make_cache(rng, 20, kv_heads, page, dim, dtype)], whole=whole)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("dim,page,pairs,layers", [(128, 1024, 16, 7), (64, 64, 230, 14)])
def test_large_copies(dim, page, pairs, layers, dtype):
    """200 MB and more, of few pairs and of many."""
    caches = [KvCache.empty(2 * pairs + 1, 8, page, dim, dtype) for _ in range(layers)]
    for c in caches:
        for t in (c.k, c.v):
            t.view(torch.uint8).random_(generator=torch.Generator("cuda").manual_seed(pairs))
        for t in (c.k_scale, c.v_scale):
            if t is not None:
                t.random_(100, 150)
    assert 2 * layers * pairs * 8 * page * dim * caches[0].k.element_size() >= 200e6
    run_case(pairs, caches, whole=True)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_layers_strides_and_bounds(dtype):
    """More caches and pairs than one launch takes; layouts that change between caches."""
    rng = np.random.default_rng(3)
    caches = [make_cache(rng, 500, 2, 16, 64, dtype, token_major=i in (3, 4, 20)) for i in range(21)]
    run_case(240, caches, bounds=[make_bounds(rng, c) for c in caches])
    run_case(193, caches[:2], bounds=[make_bounds(rng, c) for c in caches[:2]], whole=True)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_to_other_caches(dtype):
    rng = np.random.default_rng(4)
    caches = [make_cache(rng, 12, 3, 32, 128, dtype) for _ in range(2)]
    to = [make_cache(rng, 30, 3, 32, 128, dtype, token_major=True) for _ in range(2)]
    bounds, to_bounds = [make_bounds(rng, c) for c in caches], [make_bounds(rng, c) for c in to]
    run_case(25, caches, bounds, to, to_bounds)
    run_case(10, caches, to=to, whole=True)


def test_bounds_to_others_of_the_same_cache():
    """The same caches on both sides, bounds of different memory; few pairs and many."""
    rng = np.random.default_rng(11)
    cache = make_cache(rng, 80, 2, 16, 64, "bf16")
    for pairs in (5, 30):
        order = rng.permutation(80)
        src, dst = order[:pairs], order[pairs:2 * pairs]
        a, b = make_bounds(rng, cache), make_bounds(rng, cache)
        before, codes, exps = raw(cache), b.codes.clone(), b.exps.clone()
        kept = a.codes.clone()
        copy = KvCopy([cache], [a], [cache], [b])
        copy._args = (copy._args[0], copy._args[0], *copy._args[2:])  # one array for both sides
        copy.copy(src, dst)
        torch.cuda.synchronize()
        check(before, before, raw(cache), src, dst, [16] * pairs, 16)
        codes[dst], exps[dst] = a.codes[src], a.exps[src]
        assert torch.equal(b.codes, codes) and torch.equal(b.exps, exps) and torch.equal(a.codes, kept)


def test_bounds_that_both_caches_share():
    """Whole pages that keep their numbers, and parts of pages, whose bounds stay where they are."""
    rng = np.random.default_rng(12)
    one, two = (make_cache(rng, 12, 2, 16, 64, "e4m3") for _ in range(2))
    bounds = make_bounds(rng, one)
    codes, exps = bounds.codes.clone(), bounds.exps.clone()
    copy = KvCopy([one], [bounds], [two], [bounds])
    for src, dst, n in (([1, 2, 5], [1, 2, 5], [16, 16, 16]), ([1, 2, 5], [2, 3, 6], [5, 15, 1])):
        source, before = raw(one), raw(two)
        copy.copy(src, dst, n)
        torch.cuda.synchronize()
        check(source, before, raw(two), src, dst, n, 16)
        assert torch.equal(bounds.codes, codes) and torch.equal(bounds.exps, exps)
    with pytest.raises(hl.LoraError):
        copy.copy([1, 2], [2, 3])


def test_one_page_to_many():
    rng = np.random.default_rng(5)
    run_case(9, [make_cache(rng, 20, 2, 16, 128, "bf16")], one_source=True)


def test_pages_beyond_32_bit_offsets():
    rng = np.random.default_rng(6)
    stride, pages = 1 << 28, 10
    pool = [torch.zeros(stride * (pages - 1) + 2 * 16 * 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k, v = (p.as_strided((pages, 2, 16, 64), (stride, 16 * 64, 64, 1)) for p in pool)
    for t in (k, v):
        t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
    run_case(5, [KvCache(k, v)], whole=True)


def test_replayed_in_a_graph_with_lists_that_are_gone():
    rng = np.random.default_rng(7)
    cache = make_cache(rng, 40, 2, 16, 128, "e4m3")
    copy = KvCopy([cache])
    graph = torch.cuda.CUDAGraph()
    src, dst, n = np.array([1, 2, 3], np.int32), np.array([11, 12, 13], np.int32), np.array([16, 5, 1], np.int32)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        copy.copy(src, dst, n)
    pairs = list(zip(src.tolist(), dst.tolist(), n.tolist()))
    src[:], dst[:], n[:] = 7, 8, 9
    for i in range(3):
        fresh = make_cache(rng, 40, 2, 16, 128, "e4m3")
        for a, b in ((cache.k, fresh.k), (cache.v, fresh.v), (cache.k_scale, fresh.k_scale), (cache.v_scale, fresh.v_scale)):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        before = raw(cache)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(before, before, raw(cache), *zip(*pairs), 16)


def test_on_a_named_stream():
    rng = np.random.default_rng(8)
    cache = make_cache(rng, 8, 2, 16, 64, "bf16")
    before = raw(cache)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    KvCopy([cache]).copy([1], [2], [3], stream=side)
    side.synchronize()
    check(before, before, raw(cache), [1], [2], [3], 16)


def test_refuses():
    cache = KvCache.empty(10, 2, 16, 64)
    copy = KvCopy([cache])
    for args in (([1], [1]), ([1], [10]), ([1], [2], [17])):
        with pytest.raises(hl.LoraError):
            copy.copy(*args)
    for args in (([1], [1, 2]), ([1], [2], [1, 1]), ([[1]], [[2]]), ([1.5], [2])):
        with pytest.raises(ValueError):
            copy.copy(*args)
    other = KvCache.empty(11, 2, 16, 64)
    for args in (([cache], [KvBounds.empty(other)]), ([cache], None, [cache, cache]), ([cache], None, None, [KvBounds.empty(cache)]),
                 ([cache], [KvBounds.empty(cache)], [other])):
        with pytest.raises(ValueError):
            KvCopy(*args)


def test_a_beam_forks_and_is_compacted():
    """The manager's lists through the copy: every sequence reads back what was written to it."""
    from heterogeneous_adapter_batching_amd.attention import AttnBatch
    rng = np.random.default_rng(9)
    caches = [make_cache(rng, 64, 2, 16, 64, "bf16") for _ in range(2)]
    pages, copy, batch = KvPages(64, 16, 6), KvCopy(caches), AttnBatch(caches[0], 2)
    held = {s: [torch.empty(0, 128, dtype=torch.bfloat16, device="cuda") for _ in caches] for s in range(6)}

    def step(seqs, tokens):
        copy.copy(*pages.append(seqs, tokens))
        table, kv = pages.table(seqs)
        batch.refresh(tokens, kv, table)
        for i, c in enumerate(caches):
            x = torch.randn(sum(tokens), 128, device="cuda").bfloat16()
            batch.write(x, -x, cache=c)
            for s, part in zip(seqs, x.split(tokens)):
                held[s][i] = torch.cat([held[s][i], part])

    def read(seqs):
        table, kv = pages.table(seqs)
        batch.refresh([0] * len(seqs), kv, table)
        for i, c in enumerate(caches):
            ko, vo = (torch.empty(int(kv.sum()), 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
            batch.read(ko, vo, cache=c)
            want = torch.cat([held[s][i] for s in seqs])
            assert torch.equal(ko, want) and torch.equal(vo, -want)
    step([0], [37])
    pages.fork(0, [1, 2, 3])
    for s in (1, 2, 3):
        held[s] = list(held[0])
    step([0, 1, 2, 3], [1, 1, 20, 1])
    read([0, 1, 2, 3])
    pages.truncate(2, 33)
    held[2] = [x[:33] for x in held[2]]
    pages.free([0])
    step([4, 2], [50, 2])
    copy.copy(*pages.compact())
    read([1, 2, 3, 4])
    assert pages.stats()[2] == 64 - pages.stats()[0]
