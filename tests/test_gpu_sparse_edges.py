"""Sparse attention at the edges of its numbers, in all of its kernels' forms: items
shared by four waves, items of a wave each, and items split over their tokens.  The
pages that rows see are drawn here, so that nothing depends on the choice.
Tolerances: test_gpu_sparse.py's, and those of test_gpu_attn_edges.py where named."""
import numpy as np
import pytest
import torch

from heterogeneous_adapter_batching_amd.sparse import SparseBatch
from test_gpu_attn import U, check, make_cache, make_table, values
from test_gpu_attn_edges import huge_values, set_tokens
from test_gpu_sparse import expected_out, normal

pytestmark = pytest.mark.gpu
HEADS, PAGE = 3, 16

# (new, cached) tokens of each sequence, pages of a row, whether every item has a wave, whether some are split
SHARED = ([(40, 130), (1, 37), (1, 1), (4, 2)], 5, False, False)
SOLO = ([(2100, 2190), (1, 37), (1, 1), (4, 2)], 5, True, False)
SPLIT = ([(12, 1500), (1, 2500)], 40, False, True)
SOLO_SPLIT = ([(1500, 700), (700, 760)] + [(1, 9000)] * 3, 300, True, True)
FORMS = [SHARED, SOLO, SPLIT, SOLO_SPLIT]
NAMES = ["shared", "solo", "split", "solo_split"]
forms = pytest.mark.parametrize("form", FORMS, ids=NAMES)
# (items of e4m3 heads of 64 never have a wave each)
kinds = pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "bf16"), (128, "e4m3"), (64, "e4m3")])


class Case:
    def __init__(self, form, dim, dtype, seed):
        seqs, self.select, solo, split = form
        rng = self.rng = np.random.default_rng([seed, dim, len(seqs)])
        self.q_len, self.kv_len, self.dim = [s[0] for s in seqs], [s[1] for s in seqs], dim
        need = sum(-(-n // PAGE) for n in self.kv_len)
        self.cache = make_cache(rng, need + 3, 1, PAGE, dim, dtype)
        self.table = make_table(rng, self.kv_len, PAGE, need + 3)
        self.rows = sum(self.q_len)
        self.pos = np.concatenate([np.arange(m - n, m) for n, m in zip(self.q_len, self.kv_len)])
        self.seq = np.repeat(np.arange(len(seqs)), self.q_len)
        self.q = normal(rng, self.rows, HEADS * dim)
        self.pages = np.full((self.rows, 1, self.select), -1, np.int32)  # numbers in the sequence
        for r, p in enumerate(self.pos):
            own = p // PAGE
            if own >= 0:
                seen = np.sort(rng.permutation(own)[:self.select - 1])
                self.pages[r, 0, :len(seen) + 1] = np.r_[seen, own]
        self.ids = np.where(self.pages < 0, -1, self.table[self.seq[:, None, None], self.pages.clip(0)])
        # rows that are looked at one by one: some of many
        self.some = np.arange(self.rows) if self.rows < 100 else np.unique(
            np.r_[np.arange(20), rng.integers(0, self.rows, 100), np.arange(self.rows - 20, self.rows)])
        self.batch = SparseBatch(self.cache, HEADS, self.select).refresh(self.q_len, self.kv_len, self.table)
        info = self.batch.sparse_info
        assert (info.n_work >= 2048) == solo and (info.n_merge > 0) == split
        self.chosen = torch.from_numpy(self.ids.astype(np.int32)).cuda()

    def run(self, scale=0.125, q=None):
        out = torch.full_like(self.q, 7.0)
        print(f"{self.rows} rows, select {self.select}, dim {self.dim}", flush=True)
        self.batch.sparse(self.q if q is None else q, out, scale, self.chosen)
        torch.cuda.synchronize()
        return out.view(self.rows, HEADS, self.dim)

    def expected(self, scale=0.125):
        """(out, tolerance) of the rows `some`."""
        at = self.some  # each as a sequence of one new token
        return expected_out(self.cache, self.q[torch.from_numpy(at).cuda()], self.ids[at], [1] * len(at), self.pos[at] + 1,
                            HEADS, scale)

    def tokens(self, r):
        """Numbers of the tokens that row r sees."""
        pages = self.pages[r, 0][self.pages[r, 0] >= 0]
        t = (pages[:, None] * PAGE + np.arange(PAGE)).ravel()
        return t[t <= self.pos[r]]

    def slots(self, r):
        """(page, slot) of these."""
        t = self.tokens(r)
        return self.table[self.seq[r], t // PAGE], t % PAGE


@forms
@kinds
def test_a_query_that_is_nan_gives_nan(form, dim, dtype):
    c = Case(form, dim, dtype, 1)
    rows = [r for r in (0, 1, c.rows // 2, c.rows - 1) if c.pos[r] >= 0]
    q = c.q.clone().view(c.rows, HEADS, dim)
    q[rows, 1] = float("nan")
    out = c.run(q=q.view(c.rows, -1))
    assert torch.isnan(out[rows, 1]).all()
    want, tol = c.expected()
    out[rows, 1] = 0
    want[np.isin(c.some, rows), 1] = 0
    check(out[c.some], want, tol)


@forms
@kinds
@pytest.mark.parametrize("which", ["k", "v"])
def test_what_is_not_finite_reaches_the_rows_that_see_it(form, dim, dtype, which):
    """NaN and infinities in some tokens' keys (or values): rows that see one are not finite (of NaN they
    are NaN), the others, of the same pages at times, are as if there were none."""
    c = Case(form, dim, dtype, 2)
    clean, tol = c.expected()
    t = getattr(c.cache, which)
    bad = np.zeros((c.cache.n_pages, PAGE), bool)
    last = int(np.argmax(c.kv_len))
    picked = [(last, c.kv_len[last] - 1), (last, c.kv_len[last] - 2), (0, c.kv_len[0] - 1), (0, 40), (0, c.kv_len[0] // 2)]
    for i, (b, token) in enumerate(picked):
        page, slot = int(c.table[b, token // PAGE]), token % PAGE
        bad[page, slot] = True
        if dtype == "e4m3":
            t.view(torch.uint8)[page, 0, slot] = 0x7F
        else:
            t[page, 0, slot] = float("nan") if i % 2 == 0 or which == "k" else float("-inf")
    for b, n in enumerate(c.kv_len):  # and past the end, which nobody sees
        if n % PAGE:
            page = int(c.table[b, n // PAGE])
            if dtype == "e4m3":
                t.view(torch.uint8)[page, 0, n % PAGE:] = 0xFF
            else:
                t[page, 0, n % PAGE:] = float("inf")
    hit = np.array([c.pos[r] >= 0 and bool(bad[c.slots(r)].any()) for r in c.some])
    assert hit.any() and not hit.all()
    out = c.run()[c.some]
    assert not torch.isfinite(out[hit]).any()
    check(out[~hit], clean[~hit], tol[~hit])


@forms
@kinds
@pytest.mark.parametrize("query", [1e7, -3.1e7, 1e25])
def test_scores_far_from_zero(form, dim, dtype, query):
    """As in test_gpu_attn_edges.py: rows average the values of the tokens with the largest score."""
    c = Case(form, dim, dtype, 4)
    for b, n in enumerate(c.kv_len):
        set_tokens(c.cache.k, c.table[b:b + 1], np.arange(n), -104.0)
        set_tokens(c.cache.k, c.table[b:b + 1], np.arange(1, n, 2), -52.0)
    if dtype == "e4m3":
        c.cache.k_scale.fill_(127)
    c.q.fill_(query)
    got = c.run().double().cpu().numpy()
    assert np.isfinite(got).all()
    v = values(c.cache.v, c.cache.v_scale)[:, 0]
    for r in c.some:
        if c.pos[r] < 0:
            assert not got[r].any()
            continue
        best = c.tokens(r) % 2 == (0 if query < 0 or c.pos[r] == 0 else 1)
        x = v[tuple(i[best] for i in c.slots(r))]
        want, err = x.mean(0), (len(x) + 8) * 2.0 ** -23 * np.abs(x).mean(0)
        assert np.all(np.abs(got[r] - want) <= err + U * (np.abs(want) + err)), r


@forms
@kinds
@pytest.mark.parametrize("scale", [0.125, 2.0])
def test_values_near_the_largest(form, dim, dtype, scale):
    """A weighted mean is no larger than its largest value, whatever its sum is."""
    c = Case(form, dim, dtype, 5)
    huge_values(c.cache, np.random.default_rng(6))
    check(c.run(scale)[c.some], *c.expected(scale))
