"""Several answers to one long prompt, over shared pages of a paged cache:

  KvPages hands out pages, shares the prompt's among the answers, and says which
  last pages have to be copied; lora_kv_copy copies them in every layer's cache
  -> lora_kv_write_norm norms and turns q and k of every head and writes k and v
  -> lora_kv_bounds, lora_sparse_select, lora_sparse_attn: each new token attends
     over the pages that score highest for it, in every second layer; the
     others' attention is lora_attn over all of them
  -> answers end, their pages are free, and the cache is compacted

    python examples/shared_prompt.py [--cache bf16|e4m3] [--prompt N] [--steps N] [--select N]

Printed is how far the sparse attention over `select` pages is from the one over
all of them (the inputs are random: no page matters more than others), and that
over all of them from lora_attn."""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from heterogeneous_adapter_batching_amd.attention import KvCache, rope_table  # noqa: E402
from heterogeneous_adapter_batching_amd.pages import KvCopy, KvPages  # noqa: E402
from heterogeneous_adapter_batching_amd.sparse import KvBounds, SparseBatch  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE, LAYERS, ANSWERS = 16, 4, 128, 16, 4, 4


class Model:
    """The attention's part of LAYERS layers; projections are random numbers."""

    def __init__(self, cache_type, pages, positions, select, seed=0):
        self.rng = torch.Generator().manual_seed(seed)
        self.caches = [KvCache.empty(pages, KV_HEADS, PAGE, DIM, cache_type) for _ in range(LAYERS)]
        self.bounds = [KvBounds.empty(c) for c in self.caches]
        self.pages, self.copies = KvPages(pages, PAGE, 1 + ANSWERS), KvCopy(self.caches, self.bounds)
        self.batch = SparseBatch(self.caches[0], HEADS, select)
        self.rope = rope_table(positions, DIM)
        self.q_norm, self.k_norm = (torch.rand(LAYERS, DIM, generator=self.rng).cuda() + 0.5 for _ in "qk")

    def step(self, seqs, new):
        """`new` tokens of each sequence through all layers: the last sparse layer's output, and the dense one's there."""
        self.copies.copy(*self.pages.append(seqs, new))
        table, kv_len = self.pages.table(seqs)
        self.batch.refresh(new, kv_len, table)
        rows = sum(new)
        chosen = self.batch.empty_selected()
        outs = [torch.empty(rows, HEADS * DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for i, (cache, bounds) in enumerate(zip(self.caches, self.bounds)):
            x = torch.randn(rows, (HEADS + 2 * KV_HEADS) * DIM, generator=self.rng).cuda()
            q, k, v = x.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1)
            turned = torch.empty(rows, HEADS * DIM, dtype=torch.bfloat16, device="cuda")
            self.batch.write(k, v, q, turned, self.rope, cache, q_norm=self.q_norm[i], k_norm=self.k_norm[i])
            self.batch.attn(turned, outs[1], DIM ** -0.5, cache)
            if i % 2:
                self.batch.bounds(bounds, cache)
                self.batch.select(turned, bounds, chosen)
                self.batch.sparse(turned, outs[0], DIM ** -0.5, chosen, cache)
        return [o.float() for o in outs]


def run(cache_type, prompt, steps, select):
    """(relative distance of the sparse outputs from the dense ones, pages in use at the end, pages without sharing)."""
    per_answer = -(-(prompt + steps) // PAGE)
    pages = -(-prompt // PAGE) + ANSWERS * (steps // PAGE + 2)
    model = Model(cache_type, pages, prompt + steps, select)
    model.step([0], [prompt])
    answers = list(range(1, 1 + ANSWERS))
    model.pages.fork(0, answers)
    model.pages.free([0])
    off = total = 0.0
    for step in range(steps):
        if step == steps // 2:  # one answer ends; the pages that are left move together
            model.pages.free([answers.pop(0)])
            model.copies.copy(*model.pages.compact())
        sparse, dense = model.step(answers, [1] * len(answers))
        off += float((sparse - dense).square().sum())
        total += float(dense.square().sum())
    free = model.pages.stats()[0]
    return (off / total) ** 0.5, pages - free, len(answers) * per_answer


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    p.add_argument("--prompt", type=int, default=2000)
    p.add_argument("--steps", type=int, default=40)
    p.add_argument("--select", type=int, default=32)
    args = p.parse_args()
    kind = torch.float8_e4m3fn if args.cache == "e4m3" else torch.bfloat16
    off, used, alone = run(kind, args.prompt, args.steps, args.select)
    every = run(kind, args.prompt, args.steps, args.prompt)[0]
    print(f"{args.steps} steps after a prompt of {args.prompt}, {args.cache} cache: {used} pages in use, {alone} without sharing")
    print(f"attention over {args.select} pages is {off:.2e} off the one over all, that over all chosen pages {every:.2e} "
          "(relative, 2-norm)")


if __name__ == "__main__":
    main()
