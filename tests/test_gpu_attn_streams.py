"""The attention's buffers on streams that the caller names, while the current
stream is busy with memory that it has let go of."""
import numpy as np
import pytest
import torch

from heterogeneous_adapter_batching_amd.attention import AttnBatch
from test_gpu_attn import check, expected, make_cache, make_table

pytestmark = pytest.mark.gpu


def keep_busy(floats):
    """Work on the current stream that writes to a block which the allocator takes for free."""
    x = torch.empty(floats, dtype=torch.float32, device="cuda")
    for _ in range(20):
        x.normal_()


@pytest.mark.parametrize("grow", [False, True])
def test_a_named_stream_beside_a_busy_one(grow):
    rng = np.random.default_rng(1)
    q_len, kv_len = [1] * 6 + [40], [3000] * 6 + [90]
    cache = make_cache(rng, 1200, 2, 16, 64, "bf16")
    table = make_table(rng, kv_len, 16, 1200)
    q = torch.from_numpy(rng.standard_normal((46, 256)).astype(np.float32)).bfloat16().cuda()
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    batch = AttnBatch(cache, 4)
    if grow:
        batch.refresh([1], [20], table[:1], stream=side)
    sizes = [1 << 12, 1 << 14, 1 << 16, 1 << 18, 1 << 20, 1 << 22]
    for n in sizes:
        keep_busy(n)
    batch.refresh(q_len, kv_len, table, stream=side)
    assert batch.info.n_merge > 0
    for n in sizes:
        keep_busy(n)
    batch.attn(q, out, 0.125, stream=side)
    torch.cuda.synchronize()
    check(out, *expected(cache, table, q, q_len, kv_len, 4, 0, 0, 0.125))
