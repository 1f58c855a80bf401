"""The write with norms of queries and keys on the GPU, against the fp64 oracle.

Tolerances, with e = 2^-24.  A norm without centring: scaling by a power of two
is exact; the sum of squares is a tree of 3 + 4 additions over rounded squares
(8 e), the mean's division and the addition of eps round once each (eps times a
power of two twice is exact), the root's reciprocal takes half of that (5 e) and
errs by 2 e itself, two products round: 9 e of the value, taken as 16 e.
Centred, the mean errs by 9 e of the largest |x| and the difference by e of
itself: with s the head's deviation (and eps), a value moves by 9 e top / s of
the weight directly, and by twice that of itself through the deviation.
A turn adds 4 e of its two terms and passes their errors on; one rounding to
bf16 adds 2^-8 of the value, one to e4m3 half a step: 2^-4 of the value, or half
of the least step where the code is subnormal."""
import numpy as np
import pytest
import torch

import oracle
from heterogeneous_adapter_batching_amd.attention import AttnBatch, KvCache, rope_table
from test_gpu_attn import make_cache, make_table, values

pytestmark = pytest.mark.gpu
E, U = 2.0 ** -24, 2.0 ** -8


def normed(x, w, eps, centred):
    """(value, error) of the norm in fp32, from the oracle and the bounds above."""
    want = oracle.norm_ref(x, w, eps, centred)
    err = 16 * E * np.abs(want)
    if centred:
        s = np.sqrt(x.var(-1, keepdims=True) + eps)
        ratio = 9 * E * np.abs(x).max(-1, keepdims=True) / s
        err = err + ratio * (np.abs(w) + 2 * np.abs(want))
    return want, err + 1e-38


def turned(want, err, angles):
    half = angles.shape[1]
    both = np.abs(want) + err
    out, size = oracle.turn_ref(want, angles), both.copy()
    size[..., :half] = size[..., half:2 * half] = both[..., :half] + both[..., half:2 * half]
    move = err.copy()
    move[..., :half] = move[..., half:2 * half] = err[..., :half] + err[..., half:2 * half]
    return out, move + 4 * E * size


def run_case(seqs, heads, kv_heads, dim, page, dtype, source, rope_dim, weights="f32", per_head=False, centred=False,
             eps=1e-6, q_norm=True, k_norm=True, x=None, seed=0, with_q=True):
    rng = np.random.default_rng([seed, heads, dim, page])
    q_len, kv_len = np.array([s[0] for s in seqs]), np.array([s[1] for s in seqs])
    pages = int(sum(-(-int(n) // page) for n in kv_len)) + 2
    cache = make_cache(rng, pages, kv_heads, page, dim, dtype)
    before = cache.k.clone()
    table, rows = make_table(rng, kv_len, page, pages), int(q_len.sum())
    if x is None:
        x = rng.standard_normal((rows, (heads + 2 * kv_heads) * dim)) * 2.0 ** rng.integers(-6, 6, (rows, 1))
        x = x + (rng.standard_normal((rows, 1)) if centred else 0)
    x = torch.from_numpy(x.astype(np.float32)).to(torch.float32 if source == "f32" else torch.bfloat16).cuda()
    q, k, v = x.split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
    q_out = torch.full((rows, heads * dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    kind = torch.float32 if weights == "f32" else torch.bfloat16
    w = [torch.from_numpy((1 + 0.3 * rng.standard_normal((n, dim) if per_head else dim)).astype(np.float32)).to(kind).cuda()
         for n in (heads, kv_heads)]
    rope = rope_table(int(max(1, kv_len.max())), rope_dim) if rope_dim else None
    print(f"case {seqs} {heads}/{kv_heads} dim {dim} page {page} {dtype} {source} {weights} rope {rope_dim} centred "
          f"{centred} per head {per_head} norms {q_norm} {k_norm}", flush=True)
    batch = AttnBatch(cache, heads).refresh(q_len, kv_len, table)
    batch.write(k, v, q if with_q else None, q_out if with_q else None, rope, q_norm=w[0] if q_norm else None,
                k_norm=w[1] if k_norm else None, eps=eps, centred=centred)
    torch.cuda.synchronize()
    pos = np.concatenate([np.arange(m - n, m) for n, m in zip(q_len, kv_len)])
    seq = np.repeat(np.arange(len(q_len)), q_len)
    found = []
    for part, n, weight, used in ((q, heads, w[0], q_norm), (k, kv_heads, w[1], k_norm)):
        y = part.double().cpu().numpy().reshape(rows, n, dim)
        want, err = normed(y, weight.double().cpu().numpy(), eps, centred) if used else (y, np.zeros_like(y))
        if rope_dim:
            t = rope.cpu().double().numpy()[pos.clip(0)]
            want, err = turned(want, err, np.arctan2(t[:, rope_dim // 2:], t[:, :rope_dim // 2]))
        found.append((want, err))
    held = pos >= 0
    if with_q:
        want, err = found[0]
        got = q_out.double().cpu().numpy().reshape(want.shape)
        assert np.all(np.abs(got - want)[held] <= (err + U * (np.abs(want) + err) + 1e-39)[held])
        assert np.all(got[~held] == 0)
    else:
        assert torch.isnan(q_out).all()
    want, err = found[1][0][held], found[1][1][held]
    page_of, place = table[seq, pos // page][held], (pos % page)[held]
    got = values(cache.k, cache.k_scale)[page_of, :, place]
    if dtype == "bf16":
        assert np.all(np.abs(got - want) <= err + U * (np.abs(want) + err) + 1e-39)
    else:
        e = cache.k_scale.cpu().numpy()[page_of, :, place].astype(int) - 127
        top, slack = np.abs(want).max(-1), err.max(-1)
        # the least power that holds the largest value, up to its error
        assert np.all((448 * 2.0 ** e >= top - slack) | (e == 119))
        assert np.all((448 * 2.0 ** (e - 1.0) < top + slack) | (e == -100))
        step = 2.0 ** (e[..., None] - 9.0)
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * (np.abs(want) + err), step / 2) + err)
    # v is as without norms, and nothing else is written
    vs = v.double().cpu().numpy().reshape(rows, kv_heads, dim)[held]
    got = values(cache.v, cache.v_scale)[page_of, :, place]
    if dtype == "bf16":
        assert np.array_equal(got, torch.from_numpy(vs).bfloat16().double().numpy())
    written = np.zeros(cache.k.shape[:3], bool)
    written[page_of, :, place] = True
    raw, old = (t.view(torch.uint8).cpu().numpy().reshape(*written.shape, -1) for t in (cache.k, before))
    assert np.array_equal(raw[~written], old[~written])
    return batch, cache, q_out


SEQS = [(1, 1), (3, 3), (1, 40), (20, 33), (2, 17)]


@pytest.mark.parametrize("centred", [False, True])
@pytest.mark.parametrize("source", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,heads,kv_heads,page,rope_dim",
                         [(128, 8, 2, 16, 128), (64, 3, 3, 1, 64), (128, 4, 1, 8, 48), (64, 5, 1, 64, 0), (128, 7, 1, 32, 0)])
def test_norms(dim, heads, kv_heads, page, rope_dim, dtype, source, centred):
    run_case(SEQS, heads, kv_heads, dim, page, dtype, source, rope_dim, centred=centred,
             weights="bf16" if heads % 2 else "f32", per_head=kv_heads != 1)


@pytest.mark.parametrize("q_norm,k_norm,with_q", [(True, False, True), (False, True, True), (False, True, False)])
def test_one_norm_alone(q_norm, k_norm, with_q):
    run_case(SEQS, 6, 2, 64, 16, "bf16", "f32", 64, q_norm=q_norm, k_norm=k_norm, with_q=with_q, per_head=True)


def test_rows_before_the_first_token():
    run_case([(5, 2), (3, 0), (1, 1)], 4, 2, 128, 16, "e4m3", "f32", 128)


@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-5, 1.0])
def test_heads_of_every_size(eps):
    """Elements whose squares pass fp32's range, subnormal ones, zeros, one alone."""
    rng = np.random.default_rng(4)
    x = np.empty((12, 4 * 64))
    for i, size in enumerate((1e38, 1e25, 1e10, 1.0, 1e-4, 1e-10, 1e-20, 1e-35, 1e-42)):
        x[i] = rng.uniform(-1, 1, 256) * size
    x[9] = 0
    x[10] = 0
    x[10, ::64] = [3e38, 1.0, 1e-20, -5.0]
    x[11] = 7.0
    run_case([(12, 12)], 2, 1, 64, 16, "bf16", "f32", 64, eps=eps, x=x)
    x[9:] = 1e20  # equal elements, eps far below a step of their squares
    _, cache, q_out = run_case([(1, 1)], 2, 1, 64, 16, "bf16", "f32", 0, eps=eps, x=x[11:], centred=True)
    assert (q_out == 0).all()
    run_case([(1, 1)], 2, 1, 64, 16, "bf16", "f32", 0, eps=eps, x=x[9:10] * 0, centred=True)


def test_infinities_and_nan_stay_in_their_head():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((3, 4 * 64)).astype(np.float32)).cuda()
    x[0, 5], x[1, 70], x[2, 130] = float("inf"), float("nan"), float("-inf")
    cache = KvCache.empty(1, 1, 16, 64)
    q_out, w = torch.empty(3, 128, dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    batch = AttnBatch(cache, 2).refresh([3], [3], np.zeros((1, 1), np.int32))
    batch.write(x[:, 128:192], x[:, 192:], x[:, :128], q_out, q_norm=w, k_norm=w)
    torch.cuda.synchronize()
    assert torch.isnan(q_out[0, 5]) and (q_out[0, :5] == 0).all() and torch.isfinite(q_out[0, 64:]).all()
    assert torch.isnan(q_out[1, 64:]).all() and torch.isfinite(q_out[1, :64]).all()
    assert torch.isnan(cache.k[0, 0, 2, 2]) and (cache.k[0, 0, 2, 3:] == 0).all() and torch.isfinite(cache.k[0, 0, :2]).all()


def test_the_write_without_norms_is_as_before():
    """The two entry points agree where no norm applies: v, and a k without one."""
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.standard_normal((40, 8 * 128)).astype(np.float32)).cuda()
    q, k, v = x.split([512, 256, 256], 1)
    table, rope = np.array([[2, 0, 1]], np.int32), rope_table(40, 128)
    got = []
    for norm in (None, torch.ones(128, device="cuda")):
        cache = KvCache.empty(3, 2, 16, 128, torch.float8_e4m3fn)
        for t in (cache.k, cache.v):
            t.view(torch.uint8).zero_()
        q_out = torch.empty(40, 512, dtype=torch.bfloat16, device="cuda")
        AttnBatch(cache, 4).refresh([40], [40], table).write(k, v, q, q_out, rope, q_norm=norm)
        got.append([t.view(torch.uint8).clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_replayed_in_a_graph_on_another_stream():
    rng = np.random.default_rng(7)
    cache = make_cache(rng, 12, 2, 16, 128, "bf16")
    table = make_table(rng, [30, 60], 16, 12)
    x = torch.from_numpy(rng.standard_normal((7, 8 * 128)).astype(np.float32)).cuda()
    q, k, v = x.split([512, 256, 256], 1)
    q_out, w = torch.empty(7, 512, dtype=torch.bfloat16, device="cuda"), torch.rand(4, 128, device="cuda")
    rope = rope_table(60, 128)
    batch = AttnBatch(cache, 4).refresh([1, 6], [30, 60], table)
    eager = batch.prepare_write(k, v, q, q_out, rope, q_norm=w, k_norm=w[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        batch.write(k, v, q, q_out, rope, q_norm=w, k_norm=w[0])
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)))
        eager()
        torch.cuda.synchronize()
        want = [t.clone() for t in (q_out, cache.k, cache.v)]
        for t in (q_out, cache.k, cache.v):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, want[0])
        pos = [(table[0, 29 // 16], 29 % 16)] + [(table[1, p // 16], p % 16) for p in range(54, 60)]
        for page, slot in pos:
            assert torch.equal(cache.k[page, :, slot], want[1][page, :, slot])
            assert torch.equal(cache.v[page, :, slot], want[2][page, :, slot])
