"""Pages, norms in the write, bounds, choice and sparse attention as a server calls
them: two layers' caches, prompts, forks that split pages, tokens taken back,
sequences that end, a cache that is compacted.  After each step every sequence's
keys and values are the ones it has written, the new ones are the oracle's within
the tolerances of test_gpu_kv_norm.py, bounds and choice are the oracle's, and the
attention is within that of test_gpu_attn.py."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from heterogeneous_adapter_batching_amd.attention import rope_table
from heterogeneous_adapter_batching_amd.pages import KvCopy, KvPages
from heterogeneous_adapter_batching_amd.sparse import KvBounds, SparseBatch
from test_gpu_attn import check, make_cache, tokens
from test_gpu_kv_norm import U, normed, turned
from test_gpu_sparse import expected_choice, expected_out

pytestmark = pytest.mark.gpu
PAGE, PAGES, SEQS, LAYERS, EPS = 16, 48, 7, 2, 1e-5


class Server:
    def __init__(self, heads, kv_heads, dim, dtype, select):
        self.rng = np.random.default_rng([heads, dim])
        self.heads, self.kv_heads, self.dim, self.dtype = heads, kv_heads, dim, dtype
        self.caches = [make_cache(self.rng, PAGES, kv_heads, PAGE, dim, dtype) for _ in range(LAYERS)]
        self.bounds = [KvBounds.empty(c) for c in self.caches]
        self.pages, self.copy = KvPages(PAGES, PAGE, SEQS), KvCopy(self.caches, self.bounds)
        self.batch = SparseBatch(self.caches[0], heads, select)
        self.rope = rope_table(400, dim)
        self.weights = [torch.from_numpy((1 + 0.3 * self.rng.standard_normal(dim)).astype(np.float32)).cuda() for _ in "qk"]
        empty = np.zeros((0, kv_heads, dim))
        self.held = [[(empty, empty) for _ in range(SEQS)] for _ in range(LAYERS)]  # what each sequence has written

    def fork(self, parent, children):
        self.pages.fork(parent, children)
        for layer in self.held:
            for c in children:
                layer[c] = layer[parent]

    def truncate(self, seq, n):
        self.pages.truncate(seq, n)
        for layer in self.held:
            layer[seq] = tuple(x[:n] for x in layer[seq])

    def free(self, seqs):
        self.pages.free(seqs)
        for layer in self.held:
            for s in seqs:
                layer[s] = tuple(x[:0] for x in layer[s])

    def step(self, seqs, new):
        self.copy.copy(*self.pages.append(seqs, new))
        table, kv_len = self.pages.table(seqs)
        self.batch.refresh(new, kv_len, table)
        rows, h, hk, d = sum(new), self.heads, self.kv_heads, self.dim
        found = []
        for cache, bounds in zip(self.caches, self.bounds):
            x = torch.from_numpy(self.rng.standard_normal((rows, (h + 2 * hk) * d)).astype(np.float32)).cuda()
            q, k, v = x.split([h * d, hk * d, hk * d], 1)
            q_out, out = (torch.full((rows, h * d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            chosen = self.batch.empty_selected()
            self.batch.write(k, v, q, q_out, self.rope, cache, q_norm=self.weights[0], k_norm=self.weights[1], eps=EPS)
            self.batch.bounds(bounds, cache)
            self.batch.select(q_out, bounds, chosen)
            self.batch.sparse(q_out, out, d ** -0.5, chosen, cache)
            found.append((q, k, v, q_out, chosen, out))
        torch.cuda.synchronize()
        pos = np.concatenate([np.arange(m - n, m) for n, m in zip(new, kv_len)])
        angles = self.rope.cpu().double().numpy()[pos]
        angles = np.arctan2(angles[:, d // 2:], angles[:, :d // 2])
        for layer, (cache, bounds, (q, k, v, q_out, chosen, out)) in enumerate(zip(self.caches, self.bounds, found)):
            row = 0
            for i, (s, n) in enumerate(zip(seqs, new)):
                got = tokens(cache, table, i, kv_len[i])
                for x, before in zip(got, self.held[layer][s]):
                    assert len(x) == len(before) + n and np.array_equal(x[:len(before)], before), (layer, s)
                self.held[layer][s] = got
                self.check_new(q_out, q, angles, row, n, self.weights[0], h, q_out[row:row + n].double().cpu().numpy())
                self.check_new(None, k, angles, row, n, self.weights[1], hk, got[0][kv_len[i] - n:])
                want = v[row:row + n].double().cpu().numpy().reshape(n, hk, d)
                slack = U * np.abs(want) if self.dtype == "bf16" else self.step_of(want)
                assert np.all(np.abs(got[1][kv_len[i] - n:] - want) <= slack)
                for j in range(kv_len[i] // PAGE):
                    for head in range(hk):
                        codes, e = oracle.bounds_ref(got[0][j * PAGE:(j + 1) * PAGE, head])
                        page = int(table[i, j])
                        assert np.array_equal(bounds.codes[page, head].cpu().numpy(), codes), (layer, s, j)
                        assert int(bounds.exps[page, head]) == e + 127
                row += n
            want = expected_choice(self.batch, bounds, table, q_out, new, kv_len)
            assert np.array_equal(chosen.cpu().numpy(), want)
            want, tol = expected_out(cache, q_out, want, new, kv_len, h, d ** -0.5)
            check(out, want, tol)

    def step_of(self, want):
        """Half a step of e4m3 at a token and head's scale, the least power of two that holds it."""
        e = np.ceil(np.log2(np.abs(want).max(-1, keepdims=True) / 448))
        return np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** (e - 9) / 2)

    def check_new(self, is_q, x, angles, row, n, weight, heads, got):
        x = x[row:row + n].double().cpu().numpy().reshape(n, heads, self.dim)
        want, err = normed(x, weight.double().cpu().numpy(), EPS, False)
        want, err = turned(want, err, angles[row:row + n])
        if is_q is not None or self.dtype == "bf16":
            slack = U * (np.abs(want) + err)
        else:
            slack = self.step_of(np.abs(want) + err)
        assert np.all(np.abs(got.reshape(want.shape) - want) <= err + slack)


@pytest.mark.parametrize("heads,kv_heads,dim,dtype", [(8, 2, 64, "bf16"), (4, 4, 128, "e4m3"), (6, 1, 128, "bf16"),
                                                      (8, 8, 64, "e4m3")])
def test_a_server_of_forking_requests(heads, kv_heads, dim, dtype):
    s = Server(heads, kv_heads, dim, dtype, select=3)
    s.step([0, 1], [70, 37])                    # prompts
    s.fork(0, [2, 3])                           # samples of them, whose last pages split
    s.fork(1, [4])
    s.step([0, 1, 2, 3, 4], [1] * 5)
    shared = s.pages.stats()[1]
    assert shared > 0
    for _ in range(2):
        s.step([4, 2, 0, 3, 1], [1] * 5)
    s.truncate(2, 40)                           # back into a page that others hold
    s.step([2, 3, 1], [30, 1, 16])              # and a prompt's chunk beside single tokens
    s.free([0, 4])
    s.free([0])
    before = s.pages.stats()
    moves = s.pages.compact()
    assert len(moves[0]) > 0 and s.pages.stats()[2] == PAGES - before[0]
    s.copy.copy(*moves)
    s.step([1, 2, 3], [1, 2, 1])
    s.step([5, 3, 1], [95, 1, 1])               # a prompt into the pages that were freed
    s.free([1, 2, 3])
    s.fork(5, [6])
    s.truncate(5, 0)                            # the fork is the only holder: nothing splits
    s.step([6], [1])
    s.free([6])
    assert s.pages.stats() == (PAGES, 0, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_shared_prompt_example(dtype):
    """Runs; over all pages it is lora_attn's sum in another order: each output is off by
    its rounding to bf16 (2^-8 at most) and, on both sides, by 2^-12 of what its tokens' values reach."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prompt.py")
    spec = importlib.util.spec_from_file_location("shared_prompt", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    off, used, alone = mod.run(dtype, 300, 6, 4)
    assert np.isfinite(off) and used < alone
    assert mod.run(dtype, 300, 6, 300)[0] <= 2 * U
