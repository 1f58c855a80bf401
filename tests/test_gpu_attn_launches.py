"""Batches of more workgroups than one launch holds (2^23 of them): the same results
for the same rows, wherever the launches part, against the oracle for some."""
import numpy as np
import pytest
import torch

from heterogeneous_adapter_batching_amd.sparse import SparseBatch
from test_gpu_attn import check, expected, make_cache
from test_gpu_sparse import expected_out, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_more_rows_than_a_launch_takes(dtype):
    """65600 single tokens of 128 kv heads; sparse with a wave to an item (bf16) or four, and dense."""
    rng = np.random.default_rng(21)
    rows, some, heads, dim, kv = 65600, 16, 128, 64, 75
    assert rows * heads > 1 << 23 and rows % some == 0
    cache = make_cache(rng, 8, heads, 16, dim, dtype)
    table = np.tile(rng.permutation(8).astype(np.int32)[:5], (rows, 1))
    few = normal(rng, some, heads * dim)
    q = few.repeat(rows // some, 1)
    batch = SparseBatch(cache, heads, 3).refresh([1] * rows, [kv] * rows, table)
    pick = np.stack([np.sort(rng.permutation(4)[:2]) for _ in range(some * heads)])
    pick = table[0][np.c_[pick, np.full(len(pick), 4)]].reshape(some, heads, 3).astype(np.int32)
    chosen = torch.from_numpy(pick).cuda().repeat(rows // some, 1, 1)
    out = torch.full((rows + 1, heads * dim), 7.0, dtype=torch.bfloat16, device="cuda")
    print(f"{rows} rows of {heads} heads, {dtype}", flush=True)
    batch.sparse(q, out, 0.125, chosen)
    torch.cuda.synchronize()
    check(out[:some], *expected_out(cache, few, pick, [1] * some, [kv] * some, heads, 0.125))
    assert torch.equal(out[:rows].view(rows // some, -1), out[:some].reshape(1, -1).expand(rows // some, -1))
    out[:rows].fill_(7.0)
    batch.attn(q, out, 0.125)
    torch.cuda.synchronize()
    check(out[:some], *expected(cache, table[:some], few, [1] * some, [kv] * some, heads, 0, 0, 0.125))
    assert torch.equal(out[:rows].view(rows // some, -1), out[:some].reshape(1, -1).expand(rows // some, -1))
    assert (out[rows] == 7).all()
