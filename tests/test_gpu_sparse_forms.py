"""The choice of pages in all of its kernels' forms: items of one token and of several,
over up to 512 pages a wave and more, with scores in LDS and in memory, in one part of
the workspace and several.  Each case says which form it means and checks that the
plan takes it.  Against the oracle, for the rows on either side of items' and parts'
borders and some others; bounds are drawn, half of the pages with another's, so that
scores tie."""
import numpy as np
import pytest
import torch

import oracle
from heterogeneous_adapter_batching_amd.attention import KvCache
from heterogeneous_adapter_batching_amd.sparse import KvBounds, SparseBatch
from test_gpu_sparse import normal

pytestmark = pytest.mark.gpu
LDS_KEYS, ONE_KEYS, SLAB_KEYS = 12288, 2048, 1 << 24  # of several tokens, of one, and of one part of the workspace


def draw_bounds(rng, cache):
    n, hk, d = cache.n_pages, cache.n_kv_heads, cache.head_dim
    codes = np.sort(rng.integers(-127, 128, (n, hk, 2, d), dtype=np.int64), 2)[:, :, ::-1].astype(np.int8)
    exps = rng.integers(125, 129, (n, hk)).astype(np.uint8)
    twin = rng.permutation(n)
    half = twin[:n // 2]
    codes[half], exps[half] = codes[twin[n - n // 2:]], exps[twin[n - n // 2:]]
    return KvBounds(cache, torch.from_numpy(np.ascontiguousarray(codes)).cuda(), torch.from_numpy(exps).cuda()), codes, exps


def run(q_len, kv_len, heads, kv_heads, dim, select, first=1, last=1, page=16, shared=False, seed=0):
    """Returns the plan's sparse info; shared: the sequences' pages are those of one."""
    rng = np.random.default_rng([seed, heads, dim, len(q_len)])
    need = [-(-n // page) for n in kv_len]
    pages = (max(need) if shared else sum(need)) + 2
    cache = KvCache.empty(pages, kv_heads, page, dim)
    order, at = rng.permutation(pages).astype(np.int32), 0
    table = np.zeros((len(kv_len), max(need)), np.int32)
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += 0 if shared else n
    bounds, codes, exps = draw_bounds(rng, cache)
    rows, group = sum(q_len), heads // kv_heads
    q = normal(rng, rows, heads * dim)
    batch = SparseBatch(cache, heads, select, first, last).refresh(q_len, kv_len, table)
    info = batch.sparse_info
    print(f"{rows} rows of {len(q_len)}, heads {heads}/{kv_heads} of {dim}, {info.max_scored} scored, {info.item_tokens} to an item",
          flush=True)
    chosen = torch.full((rows + 1, kv_heads, select), 77, dtype=torch.int32, device="cuda")
    batch.select(q, bounds, chosen)
    torch.cuda.synchronize()
    got = chosen.cpu().numpy()
    assert (got[rows] == 77).all()
    seq = np.repeat(np.arange(len(q_len)), q_len)
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(q_len, kv_len)])
    step = info.item_tokens
    part = max(1, SLAB_KEYS // max(1, info.max_scored * kv_heads))
    some = np.r_[0:min(3, rows), max(0, rows - 3):rows, np.arange(1, 4) * step - 1, np.arange(1, 4) * step,
                 np.arange(1, 4) * part - 1, np.arange(1, 4) * part, rng.integers(0, rows, 12)]
    x = q.double().cpu().numpy().reshape(rows, kv_heads, group, dim)
    for r in np.unique(some[some < rows]):
        own = int(pos[r]) // page
        ids = table[seq[r], :max(own, 0) + 1]
        for h in range(kv_heads) if group < 9 else (0, kv_heads - 1):
            want = np.full(select, -1)
            if own >= 0:
                best = oracle.select_ref(x[r, h], codes[ids, h], exps[ids, h].astype(int) - 127, own, select, first, last)
                want[:len(best)] = ids[best]
            assert np.array_equal(got[r, h], want), (r, h)
    return info


# heads, kv heads, new tokens, pages, tokens to an item: one, two and four tiles of 16 rows, one and several tokens to a wave
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,new,pages,tokens", [
    (64, 8, 603, 300, 8),      # four tiles
    (32, 8, 603, 300, 8),      # two
    (24, 8, 603, 60, 8),
    (16, 8, 2053, 282, 16),    # a wave chooses for two tokens
    (32, 32, 519, 70, 32),     # for four
    (32, 32, 1100, 64, 64),    # for eight
    (14, 2, 1300, 100, 5),
    (24, 2, 1100, 100, 4),     # 12 heads: a tile to a token
    (40, 2, 1100, 100, 4),     # 20 heads: two tiles one after the other
    (33, 1, 2060, 90, 4)])     # 33: three
def test_several_tokens(heads, kv_heads, new, pages, tokens, dim):
    info = run([new], [16 * pages - 3], heads, kv_heads, dim, 13, 2, 1)
    assert info.item_tokens == tokens and 1 < info.max_scored * tokens <= LDS_KEYS


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,new,pages,tokens", [
    (64, 8, 520, 1500, 8), (16, 8, 700, 600, 8), (8, 8, 530, 1530, 8), (32, 8, 300, 2400, 4), (12, 2, 530, 5000, 2)])
def test_several_tokens_over_more_pages_than_a_wave_holds(heads, kv_heads, new, pages, tokens, dim):
    info = run([new], [16 * pages - 3], heads, kv_heads, dim, 100, 1, 2)
    assert info.item_tokens == tokens and info.max_scored > 512 and info.max_scored * tokens <= LDS_KEYS


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(64, 8), (7, 7), (32, 32)])
def test_chunks_with_single_tokens_and_short_ones(heads, kv_heads, dim):
    q_len = [600, 1, 1, 0, 30, 5, 40]
    info = run(q_len, [5000, 7000, 40, 90, 20, 2, 700], heads, kv_heads, dim, 20, 1, 3)
    assert info.item_tokens > 1 and info.max_scored > 400


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 1), (20, 1), (6, 3)])
def test_single_tokens_in_lds(heads, kv_heads, dim):
    info = run([1] * 5, [16 * n - 5 for n in (2040, 600, 513, 40, 2)], heads, kv_heads, dim, 30, 1, 2)
    assert info.item_tokens == 1 and 1900 < info.max_scored <= ONE_KEYS


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,longest", [(8, 1, 2400), (40, 2, 5200), (6, 3, 9000), (4, 1, 17000), (17, 1, 40000)])
def test_single_tokens_through_memory(heads, kv_heads, longest, dim):
    """17000 and 40000 pages: more than the choosing waves hold."""
    info = run([1, 1, 2, 1], [16 * n - 5 for n in (longest, 600, 2500, 4)], heads, kv_heads, dim, 200, 2, 1)
    assert info.item_tokens == 1 and info.max_scored > ONE_KEYS


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 8, 64), (16, 2, 128)])
def test_more_scores_than_one_part_of_the_workspace(heads, kv_heads, dim):
    n = 700 if kv_heads == 8 else 2600
    info = run([1] * n, [16 * 7100 - (151 * i) % 113000 for i in range(n)], heads, kv_heads, dim, 40, 1, 1, shared=True)
    assert info.item_tokens == 1 and info.max_scored * kv_heads * n > 2 * SLAB_KEYS


@pytest.mark.parametrize("heads,kv_heads,new", [(16, 8, 90), (3, 1, 40)])
def test_a_chunk_through_memory(heads, kv_heads, new):
    """Too many pages for several tokens of an item: one each, also of the short sequences beside it."""
    info = run([new, 20, 1], [16 * 7000 - 3, 900, 100], heads, kv_heads, 128, 50, 1, 2)
    assert info.item_tokens == 1 and info.max_scored > LDS_KEYS // 2
