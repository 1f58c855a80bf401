"""Attention on the GPU at the edges of its numbers, against what the formula
gives: NaN scores, windows longer than any sequence, scores far from zero, values
near the largest, weights next to each other."""
import numpy as np
import pytest
import torch

import oracle
from heterogeneous_adapter_batching_amd.attention import AttnBatch
from test_gpu_attn import U, check, expected, make_cache, make_table, run_case, tokens

pytestmark = pytest.mark.gpu

# (new tokens, cached tokens with them): narrow items of one and of several splits, wide ones, pair ones
SIZES = [(1, 40), (1, 3000), (70, 90), (33, 2000), (300, 2433)]


def case(n, kv, dtype, seed, heads=4, kv_heads=1, dim=64, page=16, **more):
    rng = np.random.default_rng([seed, n, kv])
    pages = -(-kv // page) + 2
    cache = make_cache(rng, pages, kv_heads, page, dim, dtype, **more)
    table = make_table(rng, [kv], page, pages)
    q = torch.from_numpy(rng.standard_normal((n, heads * dim)).astype(np.float32)).bfloat16().cuda()
    print(f"case {n} over {kv} {dtype}", flush=True)
    return cache, table, q


def attend(cache, table, q, kv, scale, heads=4):
    out = torch.zeros_like(q)
    AttnBatch(cache, heads).refresh([q.shape[0]], [kv], table).attn(q, out, scale)
    torch.cuda.synchronize()
    return out


def set_tokens(t, table, which, value):
    """Every element of tokens `which` of the one sequence becomes `value` (e4m3: its code)."""
    page = t.shape[2]
    at = (torch.from_numpy(table[0][which // page].astype(np.int64)).cuda(), slice(None),
          torch.from_numpy(which % page).cuda())
    if t.dtype == torch.float8_e4m3fn:
        t.view(torch.uint8)[at] = torch.tensor([value]).to(t.dtype).view(torch.uint8).item()
    else:
        t[at] = value


@pytest.mark.parametrize("n,kv", SIZES)
def test_a_query_that_is_nan_gives_nan(n, kv):
    cache, table, q = case(n, kv, "bf16", 1)
    kvs = [tokens(cache, table, 0, kv)]
    q[n // 2, 64:128] = float("nan")  # one head of one row
    out = attend(cache, table, q, kv, 0.125)
    assert torch.isnan(out[n // 2, 64:128]).all()
    out[n // 2, 64:128] = q[n // 2, 64:128] = 0
    want, tol = expected(cache, table, q, [n], [kv], 4, 0, 0, 0.125, kvs)
    want[n // 2, 1] = 0
    check(out, want, tol)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("kv", [1, 33, 34, 65, 97, 129])
def test_a_newest_key_that_is_nan_gives_nan(kv, dtype):
    """One token over kv: the newest key may be all that a wave sees."""
    cache, table, q = case(1, kv, dtype, 2)
    set_tokens(cache.k, table, np.array([kv - 1]), float("nan"))
    assert torch.isnan(attend(cache, table, q, kv, 0.125)).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,kv", SIZES)
@pytest.mark.parametrize("late", [False, True])
def test_keys_that_are_nan_give_nan(n, kv, late, dtype):
    """Half of the keys that every row sees: some parts of a split row see nothing else."""
    cache, table, q = case(n, kv, dtype, 3)
    seen = kv - n + 1
    set_tokens(cache.k, table, np.arange(seen // 2, seen) if late else np.arange((seen + 1) // 2), float("nan"))
    assert torch.isnan(attend(cache, table, q, kv, 0.125)).all()


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 5), (2 ** 30, 2 ** 31 - 1), (20, 2 ** 31 - 1)])
def test_windows_and_sinks_longer_than_any_sequence(window, sinks):
    """Rows before the first token among them, which see nothing."""
    run_case([(40, 35), (1, 70), (3, 0), (150, 140), (1, 2000)], 4, 2, 64, 16, "bf16", window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,kv", SIZES)
@pytest.mark.parametrize("query", [1e7, -1e7, 3.1e7, 1e9, -1e12, 1e25])
def test_scores_far_from_zero(n, kv, query, dtype):
    """Scores of 1e11 and more, where a step of fp32 is thousands: rows average
    the values of the tokens with the largest score, however far from zero it
    is.  Odd tokens have half of the even ones' score.  The weights are equal, so
    what is left is the sum's rounding and the output's."""
    cache, table, q = case(n, kv, dtype, 4)
    set_tokens(cache.k, table, np.arange(kv), -104.0)
    set_tokens(cache.k, table, np.arange(1, kv, 2), -52.0)
    if dtype == "e4m3":
        cache.k_scale.fill_(127)
    _, v = tokens(cache, table, 0, kv)
    q.fill_(query)
    got = attend(cache, table, q, kv, 0.125).double().cpu().numpy().reshape(n, 4, 64)
    assert np.isfinite(got).all()
    for i in range(n):
        seen = np.arange(kv - n + i + 1)
        best = seen[seen % 2 == (0 if query < 0 or len(seen) == 1 else 1)]
        want = v[best, 0].mean(0)
        err = (len(best) + 8) * 2.0 ** -23 * np.abs(v[best, 0]).mean(0)
        assert np.all(np.abs(got[i] - want) <= err + U * (np.abs(want) + err)), i


HUGE = 3.3e38  # near the largest bf16 value; an e4m3 cache goes to 448 * 2^119


def huge_values(cache, rng):
    """Values near the largest that the cache holds, of one sign in most elements."""
    x = rng.uniform(0.3, 1.0, cache.v.shape) * np.where(np.arange(cache.v.shape[3]) % 4 == 3, -1, 1)
    if cache.v_scale is None:
        cache.v.copy_(torch.from_numpy((HUGE * x).astype(np.float32)))
    else:
        cache.v.copy_(torch.from_numpy((448 * x).astype(np.float32)).to(torch.float8_e4m3fn))
        cache.v_scale.fill_(127 + 119)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,kv", SIZES + [(1, 2), (2, 130), (40, 400)])
@pytest.mark.parametrize("scale", [1e-6, 0.125, 2.0])
def test_values_near_the_largest(n, kv, scale, dtype):
    """A weighted mean is no larger than its largest value, whatever its sum is."""
    cache, table, q = case(n, kv, dtype, 5)
    huge_values(cache, np.random.default_rng(6))
    out = attend(cache, table, q, kv, scale)
    check(out, *expected(cache, table, q, [n], [kv], 4, 0, 0, scale))


@pytest.mark.parametrize("n,kv,every", [(1, 128, 32), (1, 3000, 32), (1, 3000, 256), (33, 2000, 64), (300, 2433, 128)])
def test_values_near_the_largest_in_every_part(n, kv, every):
    """Equal weights, one token in each wave's or split's part and none beside it."""
    cache, table, q = case(n, kv, "bf16", 7)
    huge_values(cache, np.random.default_rng(8))
    set_tokens(cache.k, table, np.arange(kv), -8.0)
    set_tokens(cache.k, table, np.arange(0, kv, every), 8.0)
    q.fill_(1.0)
    out = attend(cache, table, q, kv, 0.125)
    check(out, *expected(cache, table, q, [n], [kv], 4, 0, 0, 0.125))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n,kv,window", [(1, 200, 0), (4, 90, 0), (1, 3000, 0), (2, 900, 300)])
def test_weights_of_few_rows_keep_16_bits(n, kv, window, dim, dtype):
    """Up to 16 rows to a kv head: a weight enters the product in two bf16 parts, so
    it is off by 2^-16 of it at most (2^-8 of what the first part leaves, which is
    2^-8 of the weight).  The rest is as in the other tests' tolerance, and the
    fp32 sum of kv products (2^-24 of the terms each)."""
    cache, table, q = case(n, kv, dtype, 9, dim=dim)
    scale = dim ** -0.5
    out = torch.zeros_like(q)
    batch = AttnBatch(cache, 4, window, 3).refresh([n], [kv], table)
    assert batch.info.n_work[0] > 0 and sum(batch.info.n_work) == batch.info.n_work[0]
    batch.attn(q, out, scale)
    torch.cuda.synchronize()
    k, v = tokens(cache, table, 0, kv)
    want, spread, reach = oracle.attend_ref(q.double().cpu().numpy().reshape(n, 4, dim), k, v, kv, window, 3, scale)
    slack = 2.0 ** -16 + 2 * ((dim + 4) * 2.0 ** -24 * reach[..., None] + 2.0 ** -20)
    err = slack * spread * 1.01 + (kv + 64) * 2.0 ** -24 * (spread + np.abs(want))
    check(out, want, err + U * (np.abs(want) + err))
