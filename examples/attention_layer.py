"""One attention layer that serves requests with different adapters, from prompts
to tokens:

  base projections (torch) -> lora_apply adds every row's q, k and v delta
  -> lora_kv_write turns q and k and puts k and v into the paged cache
  -> lora_attn, prompts' chunks and single tokens in one call
  -> lora_apply adds the output projection's delta

and at the end lora_kv_read takes the cache back out.  Everything is compared
with the layer written out plainly in 64 bits.

    python examples/attention_layer.py [--cache bf16|e4m3] [--steps N]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from heterogeneous_adapter_batching_amd.attention import AttnBatch, KvCache, rope_table  # noqa: E402
from heterogeneous_adapter_batching_amd.session import Batch, Rows  # noqa: E402

D, HEADS, KV_HEADS, DIM, PAGE, PAGES = 512, 8, 2, 64, 16, 96
RANKS = [8, 16, 32, 64]         # one adapter each
MAX_ROWS, POSITIONS = 256, 1024
WIDTHS = {"q": (D, HEADS * DIM), "k": (D, KV_HEADS * DIM), "v": (D, KV_HEADS * DIM), "o": (HEADS * DIM, D)}


class Layer:
    def __init__(self, cache_type, seed=0):
        rng = torch.Generator().manual_seed(seed)
        self.base, self.adapters, self.rows = {}, {}, {}
        for name, (n_in, n_out) in WIDTHS.items():
            self.base[name] = (torch.randn(n_in, n_out, generator=rng) * n_in ** -0.5).bfloat16().cuda()
            for side, n in (("A", n_in), ("B", n_out)):
                # adapter rows one after the other: offset of row j of adapter a
                pool = (torch.randn(len(RANKS), max(RANKS), n, generator=rng) * D ** -0.5).bfloat16().cuda()
                off = torch.arange(len(RANKS) * max(RANKS), dtype=torch.int64, device="cuda") * n
                self.adapters[name, side] = pool
                self.rows[name, side] = Rows(pool, off, len(RANKS), max(RANKS), n, n)
        self.cache = KvCache.empty(PAGES, KV_HEADS, PAGE, DIM, cache_type)
        self.rope = rope_table(POSITIONS, DIM)
        self.lora = Batch(MAX_ROWS, RANKS, D, D)
        self.attn = AttnBatch(self.cache, HEADS)

    def project(self, x, names):
        """fp32 outputs of the base projections with every row's delta."""
        ys = [(x @ self.base[n]).float() for n in names]
        self.lora.apply([(x, self.rows[n, "A"], self.lora.new_v(max(RANKS)), self.rows[n, "B"], y, 1.0)
                         for n, y in zip(names, ys)])
        return ys

    def step(self, x, row_adapter, q_len, kv_len, table):
        """x: bf16 [rows, D], the new tokens of every request on end."""
        self.lora.refresh(np.asarray(row_adapter, np.int32))
        self.attn.refresh(q_len, kv_len, table)
        q, k, v = self.project(x, "qkv")
        turned, out = (torch.empty(x.shape[0], HEADS * DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.attn.write(k, v, q, turned, self.rope)
        self.attn.attn(turned, out, DIM ** -0.5)
        return self.project(out, "o")[0]


def plain(layer, x, adapter):
    """The layer's output for one request's whole x [n, D], in 64 bits on the CPU; and its k, v."""
    def project(x, name):
        A, B = (layer.adapters[name, s][adapter, :RANKS[adapter]].double().cpu() for s in "AB")
        return x @ layer.base[name].double().cpu() + x @ A.T @ B

    def turn(u):
        cos, sin = layer.rope[:n].double().cpu()[:, None].split(DIM // 2, 2)
        a, b = u.split(DIM // 2, 2)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], 2)
    x, n = x.double().cpu(), x.shape[0]
    q, k, v = (project(x, name).reshape(n, -1, DIM) for name in "qkv")
    q, k = turn(q), turn(k)
    group = HEADS // KV_HEADS
    s = (q.transpose(0, 1) @ k.repeat_interleave(group, 1).permute(1, 2, 0)) * DIM ** -0.5
    s += torch.full((n, n), -torch.inf, dtype=torch.float64).triu(1)
    o = torch.softmax(s, -1) @ v.repeat_interleave(group, 1).transpose(0, 1)
    return project(o.transpose(0, 1).reshape(n, -1), "o"), k, v


def run(cache_type, steps, seed=0):
    """Relative error of the outputs, and of what is read back from the cache."""
    rng = np.random.default_rng(seed)
    layer = Layer(cache_type, seed)
    free = list(rng.permutation(PAGES))
    requests = []  # adapter, x so far, outputs so far, pages
    for step in range(steps):
        # every request there is gets a token; now and then one joins with its prompt
        new = [torch.randn(1, D).bfloat16().cuda() for _ in requests]
        if step % 3 == 0 and len(requests) < 6:
            requests.append([int(rng.integers(len(RANKS))), torch.empty(0, D, dtype=torch.bfloat16, device="cuda"), [], []])
            new.append(torch.randn(int(rng.integers(2, 90)), D).bfloat16().cuda())
        for r, x in zip(requests, new):
            r[1] = torch.cat([r[1], x])
            while len(r[3]) * PAGE < r[1].shape[0]:
                r[3].append(free.pop())
        q_len, kv_len = [x.shape[0] for x in new], [r[1].shape[0] for r in requests]
        table = np.zeros((len(requests), max(len(r[3]) for r in requests)), np.int32)
        for i, r in enumerate(requests):
            table[i, :len(r[3])] = r[3]
        y = layer.step(torch.cat(new), np.repeat([r[0] for r in requests], q_len), q_len, kv_len, table)
        for r, part in zip(requests, y.split(q_len)):
            r[2].append(part)
    k_out, v_out = (torch.empty(sum(kv_len), KV_HEADS * DIM, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    layer.attn.read(k_out, v_out)
    off = total = held_off = held = 0.0
    for (adapter, x, outs, _), k, v in zip(requests, k_out.split(kv_len), v_out.split(kv_len)):
        want, want_k, want_v = plain(layer, x, adapter)
        off += float((torch.cat(outs).double().cpu() - want).square().sum())
        total += float(want.square().sum())
        for got, w in ((k, want_k), (v, want_v)):
            held_off += float((got.double().cpu() - w.reshape(len(w), -1)).square().sum())
            held += float(w.square().sum())
    return (off / total) ** 0.5, (held_off / held) ** 0.5


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    p.add_argument("--steps", type=int, default=20)
    args = p.parse_args()
    out, held = run(torch.float8_e4m3fn if args.cache == "e4m3" else torch.bfloat16, args.steps)
    print(f"{args.steps} steps, {args.cache} cache: outputs off by {out:.2e}, k and v in the cache by {held:.2e} (relative, 2-norm)")


if __name__ == "__main__":
    main()
