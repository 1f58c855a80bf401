"""The operators around the paged cache as they are measured: the write with norms
of queries and keys, the copy of pages, the bounds of pages' keys, the choice of
pages by them for each new token, and the attention over the chosen pages.

`run` computes them in plain torch where `own` is false, and through the
framework's entry points where it is true.  A batch is made of `seqs`
sequences with new_lo..new_hi new tokens each and `singles` more with one new
token; each has past_lo..past_hi tokens in the cache already (all lengths
spread over their logarithm, and fixed by the case, not by the seed).  `heads`
query heads share `kv_heads` key and value heads of `dim` elements; the cache
holds pages of `page` tokens, in bf16 or in e4m3 with a power of two per token
and head.  A copy moves `pairs` pages (their first tokens, or all of them) in
each of `layers` caches.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EXP_LO, EXP_HI = -100, 119   # exponents a cache's scale may have
BOUND_MAX, BOUND_EXP = 127.0, 100  # largest bound, and exponent of bounds
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a 64-request batch of a d = 8192 layer with norms of q and k, straight
        # from the projections' fp32 outputs
        _case("norm_decode", "norm", seqs=64, past=(1, 2048), heads=64, kv_heads=8, page=16, source="f32", rotary=128),
        # a prefill batch of lognormal-like prompt lengths at d = 4096, centred, a weight of its own for each
        # head, quantised as it is written
        _case("norm_prefill", "norm", seqs=16, new=(128, 2048), heads=32, kv_heads=32, page=64, cache="e4m3", rotary=64,
              centred=True, per_head=True),
        # the smallest call: a request forks inside its last page, one layer
        _case("copy_one", "copy", pairs=1, layers=1, spare=63, heads=8, kv_heads=8, page=16),
        # 64 requests of a beam go on from others' last pages, all layers of a model
        _case("copy_fork", "copy", pairs=64, layers=32, spare=128, heads=8, kv_heads=8, page=16),
        # a fragmented quantised cache is compacted, bounds and all
        _case("copy_compact", "copy", pairs=700, layers=4, spare=648, heads=8, kv_heads=8, page=64, cache="e4m3",
              whole=True, bounded=True),
        # the pages that a prefill batch has filled, every head with keys of its own
        _case("bounds_prefill", "bounds", seqs=16, new=(128, 2048), heads=32, kv_heads=32, page=16),
        # sequences brought back into a quantised cache
        _case("bounds_back", "bounds", seqs=48, past=(256, 16384), heads=64, kv_heads=8, page=64, cache="e4m3"),
        # the choice for one decode step over long ragged contexts in small pages
        _case("select_decode", "select", seqs=32, past=(2048, 32768), heads=64, kv_heads=8, page=16, select=128, last=2),
        # the choice for every token of a chunk of a long prompt
        _case("select_chunk", "select", seqs=1, new=(512, 512), past=(16000, 16000), heads=32, kv_heads=8, page=32,
              select=64, last=4),
        # one request's token over a long context, choice and attention
        _case("sparse_one", "sparse", seqs=1, past=(32000, 32000), heads=32, kv_heads=8, page=64, select=16),
        # one decode step over long ragged contexts of a quantised cache
        _case("sparse_decode", "sparse", seqs=32, past=(2048, 32768), heads=64, kv_heads=8, page=64, cache="e4m3",
              select=32, last=2),
        # chunks of two long prompts and single tokens beside them: the largest
        _case("sparse_chunk", "sparse", seqs=2, new=(400, 512), past=(16000, 32768), singles=8, heads=64, kv_heads=8,
              page=64, select=16, last=2),
    ]


def _case(name, op, *, seqs=0, new=(1, 1), past=(0, 0), singles=0, heads, kv_heads, dim=128, page, cache="bf16",
          source="bf16", rotary=0, centred=False, per_head=False, pairs=0, layers=1, spare=0, whole=False, bounded=False,
          select=0, first=1, last=1, lengths=0):
    c = {"name": name, "op": op, "seqs": seqs, "new_lo": new[0], "new_hi": new[1], "past_lo": past[0],
         "past_hi": past[1], "singles": singles, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
         "cache": cache, "source": source, "rotary": rotary, "centred": centred, "per_head": per_head, "pairs": pairs,
         "layers": layers, "spare": spare, "whole": whole, "bounded": bounded, "select": select, "first": first,
         "last": last, "lengths": lengths}
    if name is None:
        del c["name"]
    return c


def _spread(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1))) - 1)))


def draw(rng):
    kind = rng.choice(("norm", "copy", "bounds", "select", "sparse", "sparse"))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 32))
    group = rng.choice((1, 2, 4, 7, 8)) if kv_heads <= 8 else 1
    dim = rng.choice((64, 128, 128))
    base = dict(heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 32, 64, 128)),
                cache=rng.choice(("bf16", "e4m3")), lengths=rng.randrange(1, 1 << 30))
    if kind == "norm":
        return _case(None, "norm", seqs=_spread(rng, 1, 16), new=(1, _spread(rng, 1, 2048)),
                     past=(0, _spread(rng, 1, 4096)), singles=_spread(rng, 1, 128), source=rng.choice(("f32", "bf16")),
                     rotary=rng.choice((0, dim // 2, dim)), centred=rng.random() < 0.3, per_head=rng.random() < 0.3,
                     **base)
    if kind == "copy":
        base["page"] = rng.choice((1, 8, 16, 32, 64, 128))
        bounded = rng.random() < 0.3 and base["page"] >= 16
        layers = _spread(rng, 1, 8)
        room = int(2e8 // (layers * kv_heads * base["page"] * 4 * dim))
        return _case(None, "copy", pairs=max(1, min(_spread(rng, 1, 500), room)), layers=layers,
                     spare=_spread(rng, 1, 200), whole=rng.random() < 0.5, bounded=bounded, **base)
    if kind == "bounds":  # a page at least to each sequence
        if rng.random() < 0.5:
            return _case(None, "bounds", seqs=_spread(rng, 1, 32), past=(base["page"], _spread(rng, 256, 8192)), **base)
        return _case(None, "bounds", seqs=_spread(rng, 1, 16), new=(base["page"], _spread(rng, 256, 2048)),
                     past=(0, _spread(rng, 1, 4096)), singles=_spread(rng, 1, 64), **base)
    first, last = rng.choice((0, 1, 1, 2)), rng.choice((1, 1, 2, 4))
    page = base["page"]
    select = first + last + _spread(rng, 0, 2048 // page)
    mask = dict(select=select, first=first, last=last)
    if rng.random() < 0.5:
        top = _spread(rng, 256, 32768)
        # bytes that are read, and that the cache takes
        room = min(4e8 // (kv_heads * select * page * 4 * dim), 3e9 // (kv_heads * top * 4 * dim))
        return _case(None, kind, seqs=max(1, min(_spread(rng, 1, 64), int(room))), past=(_spread(rng, 1, top), top),
                     **base, **mask)
    top = _spread(rng, 256, 16384)
    # elements of the chosen keys of every row, which the plain form holds
    room = int(4e8 // (kv_heads * select * page * dim))
    new = max(2, min(_spread(rng, 2, 512), room))
    return _case(None, kind, seqs=max(1, min(_spread(rng, 1, 3), room // new)), new=(max(1, new // 3), new),
                 past=(0, top), singles=rng.choice((0, 0, 3)), **base, **mask)


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence."""
    rng = random.Random("%d %d %d" % (case["lengths"], case["new_hi"], case["past_hi"]))
    new = [_spread(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])] + [1] * case["singles"]
    past = [_spread(rng, case["past_lo"], case["past_hi"]) for _ in new]
    return new, [n + p for n, p in zip(new, past)]


def _bounded(case):
    """Tokens of each sequence whose pages have their bounds already: of a batch with prompts the past, of one that
    only comes back none."""
    new, kv = _lengths(case)
    return [k - n for n, k in zip(new, kv)] if case["new_hi"] > 1 or case["singles"] else [0] * len(new)


def _fresh(case):
    """(from, to) page numbers of each sequence that get bounds."""
    return [(b // case["page"], k // case["page"]) for b, k in zip(_bounded(case), _lengths(case)[1])]


def _tokens(case):
    """Tokens copied of each pair's page."""
    rng = random.Random("tokens %d %d" % (case["lengths"], case["pairs"]))
    return [case["page"] if case["whole"] else rng.randint(1, case["page"]) for _ in range(case["pairs"])]


def _token_bytes(case):
    """Of one token's keys (or values) of one kv head."""
    return case["dim"] * 2 if case["cache"] == "bf16" else case["dim"] + 1


def work(case):
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    held, bound = _token_bytes(case), 2 * d + 1
    if case["op"] == "copy":
        tokens = _tokens(case)
        moved = 2 * held * sum(tokens) + (bound * sum(n == page for n in tokens) if case["bounded"] else 0)
        return {"bytes": 2 * case["layers"] * hk * moved, "flops": 0}
    new, kv = _lengths(case)
    rows = sum(new)
    if case["op"] == "norm":
        size = 4 if case["source"] == "f32" else 2
        moved = rows * ((hq + 2 * hk) * d * size + hq * d * 2 + 2 * hk * held + case["rotary"] * 4)
        return {"bytes": moved, "flops": rows * (hq + hk) * (4 * d + 3 * case["rotary"])}
    if case["op"] == "bounds":
        pages = sum(b - a for a, b in _fresh(case))
        return {"bytes": pages * hk * (page * held + bound), "flops": 2 * pages * hk * page * d}
    total = {"bytes": rows * (hq * d * 2 + hk * case["select"] * 4), "flops": 0}
    for n, k in zip(new, kv):
        scored, seen = 0, 0
        for p in range(k - n, k):
            pages = p // page + 1
            if pages > case["select"]:
                scored += pages
            seen += (min(pages, case["select"]) - 1) * page + p % page + 1
        total["bytes"] += ((k - 1) // page if scored else 0) * hk * bound
        total["flops"] += 4 * d * hq * scored
        if case["op"] == "sparse":
            total["bytes"] += min(seen, k) * hk * 2 * held + n * hq * d * 2
            total["flops"] += 4 * d * hq * seen
    return total


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": case, "g": g}
    if case["op"] == "copy":
        _prepare_copy(s, seed, dev)
        return s
    new, kv = _lengths(case)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    rows = sum(new)
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 7  # a few of another user's
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.zeros(len(kv), max(need), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    s.update(new=new, kv=kv, scale=1 / math.sqrt(d))
    _make_cache(s, (pages, hk, page, d), dev)
    if case["op"] == "norm":
        kind = torch.float32 if case["source"] == "f32" else torch.bfloat16
        # the outputs of one projection of q, k and v: columns of one matrix
        s["qkv"] = _normal(s, rows, (hq + 2 * hk) * d, dtype=kind)
        s["q_out"] = torch.zeros(rows, hq * d, dtype=torch.bfloat16, device=dev)
        for name, heads in (("q", hq), ("k", hk)):
            s[name + "_norm"] = 1 + 0.2 * _normal(s, *((heads, d) if case["per_head"] else (d,)), dtype=torch.float32)
        half = case["rotary"] // 2
        if half:
            turn = torch.arange(max(kv), device=dev, dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
            s["rope"] = torch.cat([turn.cos(), turn.sin()], 1).float().contiguous()
        else:
            s["rope"] = None
    else:
        s["bounds"] = torch.zeros(pages, hk, 2, d, dtype=torch.int8, device=dev)
        s["bound_exp"] = torch.full((pages, hk), 127, dtype=torch.uint8, device=dev)
    if case["op"] in ("select", "sparse"):
        # every complete page's bounds, as the steps before have left them
        full = torch.cat([table[i, :n // page] for i, n in enumerate(kv)]).long().to(dev)
        s["bounds"][full], s["bound_exp"][full] = _bounds_of(_values(s["k"], s["k_exp"], (full,)))
        s["q"] = _normal(s, rows, hq * d)
        s["chosen"] = torch.zeros(rows, hk, case["select"], dtype=torch.int32, device=dev)
        s["out"] = torch.zeros(rows, hq * d, dtype=torch.bfloat16, device=dev)
    if own:
        s["calls"] = _calls(s, table)
    else:
        _indexes(s, table, dev)
    return s


def _normal(s, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=s["g"], device=s["g"].device, dtype=torch.float32).to(dtype)


def _make_cache(s, held, dev):
    """k and v [..., pages, heads, tokens, dim]; the keys of a page lie about a middle of their own."""
    for name in ("k", "v"):
        x = _normal(s, *held)
        if name == "k" and s["case"]["op"] in ("select", "sparse"):
            x += 0.6 * _normal(s, *held[:-2], 1, held[-1])
        if s["case"]["cache"] == "bf16":
            s[name], s[name + "_exp"] = x, None
        else:
            s[name] = (x * 128).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s[name + "_exp"] = torch.randint(119, 122, held[:-1], generator=s["g"], device=dev, dtype=torch.uint8)


def _prepare_copy(s, seed, dev):
    c = s["case"]
    pages = 2 * c["pairs"] + c["spare"]
    _make_cache(s, (c["layers"], pages, c["kv_heads"], c["page"], c["dim"]), dev)
    if c["bounded"]:
        s["bounds"] = torch.randint(-127, 128, (c["layers"], pages, c["kv_heads"], 2, c["dim"]), generator=s["g"],
                                    device=dev, dtype=torch.int8)
        s["bound_exp"] = torch.randint(110, 130, (c["layers"], pages, c["kv_heads"]), generator=s["g"], device=dev,
                                       dtype=torch.uint8)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    src, dst, tokens = order[:c["pairs"]], order[c["pairs"]:2 * c["pairs"]], torch.tensor(_tokens(c))
    s.update(src=src, dst=dst, tokens=tokens)
    if own:
        s["calls"] = _copy_calls(s)
    else:
        pair = torch.repeat_interleave(torch.arange(c["pairs"]), tokens)
        slot = torch.arange(int(tokens.sum())) - torch.repeat_interleave(tokens.cumsum(0) - tokens, tokens)
        s["from"] = (slice(None), src[pair].to(dev), slice(None), slot.to(dev))
        s["to"] = (slice(None), dst[pair].to(dev), slice(None), slot.to(dev))
        full = tokens == c["page"]
        s["full"] = (src[full].to(dev), dst[full].to(dev))


def _copy_calls(s):
    from heterogeneous_adapter_batching_amd.attention import KvCache
    from heterogeneous_adapter_batching_amd.pages import KvCopy
    from heterogeneous_adapter_batching_amd.sparse import KvBounds

    layers = range(s["case"]["layers"])
    exps = [(None, None) if s["k_exp"] is None else (s["k_exp"][i], s["v_exp"][i]) for i in layers]
    caches = [KvCache(s["k"][i], s["v"][i], *exps[i]) for i in layers]
    bounds = [KvBounds(cache, s["bounds"][i], s["bound_exp"][i]) for i, cache in enumerate(caches)] \
        if s["case"]["bounded"] else None
    return [KvCopy(caches, bounds).prepare_copy(s["src"].numpy(), s["dst"].numpy(), s["tokens"].numpy())]


def _calls(s, table):
    from heterogeneous_adapter_batching_amd.attention import AttnBatch, KvCache
    from heterogeneous_adapter_batching_amd.sparse import KvBounds, SparseBatch

    c = s["case"]
    cache = KvCache(s["k"], s["v"], s["k_exp"], s["v_exp"])
    if c["op"] == "norm":
        batch = AttnBatch(cache, c["heads"])
        batch.refresh(s["new"], s["kv"], table.numpy())
        q, k, v = _split(s)
        return [batch.prepare_write(k, v, q, s["q_out"], s["rope"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                                    centred=c["centred"])]
    bounds = KvBounds(cache, s["bounds"], s["bound_exp"])
    batch = SparseBatch(cache, c["heads"], c["select"] or c["first"] + c["last"], c["first"], c["last"])
    batch.refresh(s["new"], s["kv"], table.numpy(), bounded=_bounded(c) if c["op"] == "bounds" else None)
    if c["op"] == "bounds":
        return [batch.prepare_bounds(bounds)]
    calls = [batch.prepare_select(s["q"], bounds, s["chosen"])]
    if c["op"] == "sparse":
        calls.append(batch.prepare_sparse(s["q"], s["out"], s["scale"], s["chosen"]))
    return calls


def _indexes(s, table, dev):
    """Where each row and each page is, for the plain forms."""
    new, kv = torch.tensor(s["new"]), torch.tensor(s["kv"])
    s["table"] = table.to(dev).long()
    seq = torch.repeat_interleave(torch.arange(len(new)), new)
    nth = torch.arange(int(new.sum())) - torch.repeat_interleave(new.cumsum(0) - new, new)
    pos = nth + (kv - new)[seq]
    page = s["case"]["page"]
    s["row_seq"], s["row_nth"], s["row_pos"] = seq.to(dev), nth.to(dev), pos.to(dev)
    s["row_page"], s["row_slot"] = table.long()[seq, pos // page].to(dev), (pos % page).to(dev)
    first = (new.cumsum(0) - new)[:, None]
    step = torch.arange(int(new.max()))[None, :]
    s["q_rows"] = (first + step.clamp(max=(new - 1)[:, None])).to(dev)
    if s["case"]["op"] == "bounds":
        s["fresh"] = torch.cat([table[i, a:b] for i, (a, b) in enumerate(_fresh(s["case"]))]).long().to(dev)


def _split(s):
    c = s["case"]
    q, k = c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
    return s["qkv"][:, :q], s["qkv"][:, q:q + k], s["qkv"][:, q + k:]


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        for call in s["calls"]:
            call()
    elif op == "norm":
        _plain_norm(s)
    elif op == "copy":
        _plain_copy(s)
    elif op == "bounds":
        s["bounds"][s["fresh"]], s["bound_exp"][s["fresh"]] = _bounds_of(_values(s["k"], s["k_exp"], (s["fresh"],)))
    else:
        at = _plain_select(s)
        if op == "sparse":
            _plain_attn(s, at)
    if op in ("select", "sparse"):
        return {"chosen": s["chosen"], "out": s["out"]} if op == "sparse" else {"chosen": s["chosen"]}
    out = {}
    if op != "bounds":
        out = {"k": s["k"], "v": s["v"]}
        if s["k_exp"] is not None:  # the powers of two, as the type that holds them
            out["k_scale"], out["v_scale"] = s["k_exp"].view(torch.float8_e8m0fnu), s["v_exp"].view(torch.float8_e8m0fnu)
    if op == "norm":
        out["q"] = s["q_out"]
    if "bounds" in s:  # whole numbers, and their exponents
        out["bounds"], out["bound_exp"] = s["bounds"], s["bound_exp"]
    return out


def _rotate(x, turn):
    """Elements i and i + half of each head of x [rows, heads, dim] turned by the angle i of the row's position."""
    half = turn.shape[1] // 2
    cos, sin = turn[:, None, :half], turn[:, None, half:]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., 2 * half:]], -1)


def _quantise(x):
    """e4m3 codes of x [..., dim], and the exponent e, biased by 127, of the least power of two with |x| <= 448 * 2^e."""
    top = torch.where(x.isfinite(), x.abs(), 0).amax(-1)
    mantissa, exponent = torch.frexp(top)  # top = mantissa * 2^exponent, mantissa in [0.5, 1)
    e = torch.where(mantissa > 0.875, exponent - 8, exponent - 9)
    e = torch.where(top > 0, e, EXP_LO).clamp(EXP_LO, EXP_HI)
    y = torch.ldexp(x, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return torch.where(x.isfinite(), y, float("nan")).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_norm(s):
    c = s["case"]
    q, k, v = (x.float().unflatten(1, (-1, c["dim"])) for x in _split(s))

    def norm(x, weight):
        if c["centred"]:
            x = x - x.mean(-1, keepdim=True)
        return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight
    q, k = norm(q, s["q_norm"]), norm(k, s["k_norm"])
    if s["rope"] is not None:
        turn = s["rope"][s["row_pos"]]
        q, k = _rotate(q, turn), _rotate(k, turn)
    s["q_out"].copy_(q.flatten(1))
    at = (s["row_page"], slice(None), s["row_slot"])
    if c["cache"] == "bf16":
        s["k"][at], s["v"][at] = k.bfloat16(), v.bfloat16()
        return
    (kc, ke), (vc, ve) = _quantise(k), _quantise(v)
    s["k"].view(torch.uint8)[at], s["v"].view(torch.uint8)[at] = kc.view(torch.uint8), vc.view(torch.uint8)
    s["k_exp"][at], s["v_exp"][at] = ke, ve


def _plain_copy(s):
    k, v = (s[n] if s["k_exp"] is None else s[n].view(torch.uint8) for n in ("k", "v"))
    k[s["to"]], v[s["to"]] = k[s["from"]], v[s["from"]]
    if s["k_exp"] is not None:
        s["k_exp"][s["to"]], s["v_exp"][s["to"]] = s["k_exp"][s["from"]], s["v_exp"][s["from"]]
    if "bounds" in s:
        src, dst = s["full"]
        s["bounds"][:, dst], s["bound_exp"][:, dst] = s["bounds"][:, src], s["bound_exp"][:, src]


def _values(codes, exps, at):
    """The cached values at an index, in 32 bits."""
    if exps is None:
        return codes[at].float()
    return torch.ldexp(codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float(), exps[at].int()[..., None] - 127)


def _exponent(top):
    """The least e with top <= 127 * 2^e, within its limits."""
    mantissa, exponent = torch.frexp(top)  # top = mantissa * 2^exponent, mantissa in [0.5, 1)
    e = torch.where(mantissa > BOUND_MAX / 128, exponent - 6, exponent - 7)
    return torch.where(top > 0, e, -BOUND_EXP).clamp(-BOUND_EXP, BOUND_EXP)


def _codes(x, e):
    return torch.ldexp(x, -e).round().clamp(-BOUND_MAX, BOUND_MAX)


def _bounds_of(x):
    """Codes [pages, heads, 2, dim] of the largest and smallest of x [pages, heads, tokens, dim] over its tokens,
    and exponents biased by 127; NaN is passed over."""
    hi = torch.where(x.isnan(), float("-inf"), x).amax(-2)
    lo = torch.where(x.isnan(), float("inf"), x).amin(-2)
    none = hi < lo
    hi, lo = torch.where(none, 0, hi), torch.where(none, 0, lo)
    e = _exponent(torch.where(x.isfinite(), x.abs(), 0).amax((-2, -1)))
    codes = _codes(torch.stack([hi, lo], -2), e[..., None, None])
    return codes.to(torch.int8), (e + 127).to(torch.uint8)


def _plain_select(s):
    """Chooses pages for every row and kv head; their numbers in the sequence [rows, kv heads, select], -1 behind."""
    c = s["case"]
    hk, group, select = c["kv_heads"], c["heads"] // c["kv_heads"], c["select"]
    q = s["q"].float().unflatten(1, (hk, group, c["dim"]))
    f = _exponent(torch.where(q.isfinite(), q.abs(), 0).amax((-2, -1)))
    q = _codes(torch.nan_to_num(q, nan=0.0, posinf=math.inf, neginf=-math.inf), f[..., None, None])
    # [seq, kv head, rows and heads, dim], every sequence padded to the one with the most rows
    q = q[s["q_rows"]].permute(0, 2, 1, 3, 4).flatten(2, 3)
    hi, lo = s["bounds"][s["table"]].float().permute(3, 0, 2, 4, 1)  # each [seq, kv head, dim, page]
    x = q.clamp(min=0) @ hi + q.clamp(max=0) @ lo  # whole numbers under 2^21: exact
    x = torch.ldexp(x.unflatten(2, (-1, group)).amax(3), s["bound_exp"][s["table"]].int().transpose(1, 2)[:, :, None] - 127)
    x = x[s["row_seq"], :, s["row_nth"]]
    own_page = (s["row_pos"] // c["page"])[:, None, None]
    i = torch.arange(x.shape[2], device=x.device)
    x = torch.where((i < c["first"]) | (i > own_page - c["last"]), float("inf"), x)
    x = torch.where(i > own_page, float("-inf"), x)
    order = x.sort(dim=-1, descending=True, stable=True).indices[..., :select]
    rank = torch.arange(order.shape[2], device=x.device)
    order = torch.where(rank < (own_page + 1).clamp(max=select), order, x.shape[2]).sort(-1).values
    at = torch.full(s["chosen"].shape, -1, dtype=torch.int64, device=x.device)
    at[..., :order.shape[2]] = torch.where(order < x.shape[2], order, -1)
    s["chosen"].copy_(torch.where(at < 0, -1, s["table"][s["row_seq"][:, None, None], at.clamp(min=0)]))
    return at


def _plain_attn(s, at):
    c = s["case"]
    hk, d, page = c["kv_heads"], c["dim"], c["page"]
    where = (s["chosen"].clamp(min=0).long(), torch.arange(hk, device=at.device)[:, None])
    # [row, kv head, chosen token, dim]
    k, v = (_values(s[n], s[n + "_exp"], where).flatten(2, 3) for n in ("k", "v"))
    token = (at[..., None] * page + torch.arange(page, device=at.device)).flatten(2)
    seen = (token >= 0) & (token <= s["row_pos"][:, None, None])
    k, v = torch.where(seen[..., None], k, 0), torch.where(seen[..., None], v, 0)
    p = s["q"].float().unflatten(1, (hk, -1, d)) @ k.transpose(2, 3)
    p *= s["scale"]
    p.masked_fill_(~seen[:, :, None], float("-inf"))
    p -= p.amax(-1, keepdim=True)
    p.exp_()
    s["out"].copy_(((p @ v) / p.sum(-1, keepdim=True)).flatten(1))


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return {"norm": _exact_norm, "copy": _exact_copy, "bounds": _exact_bounds, "select": _exact_sparse,
            "sparse": _exact_sparse}[case["op"]](s, case)


def _exact_norm(s, case):
    d, hk = case["dim"], case["kv_heads"]
    q, k, v = (x.double() for x in _split(s))
    half = case["rotary"] // 2
    for x, weight in ((q, s["q_norm"]), (k, s["k_norm"])):
        y = x.reshape(x.shape[0], -1, d)
        var, mean = torch.var_mean(y, -1, correction=0, keepdim=True)
        if not case["centred"]:
            var, mean = var + mean ** 2, 0
        y = (y - mean) / torch.sqrt(var + EPS) * weight.double()
        if half:
            turn = s["rope"][s["row_pos"]].double()
            unit = torch.complex(turn[:, :half], turn[:, half:])[:, None]
            z = torch.complex(y[..., :half].contiguous(), y[..., half:2 * half].contiguous()) * unit
            y[..., :half], y[..., half:2 * half] = z.real, z.imag
        x.copy_(y.reshape(x.shape))
    out = {"q": q}
    for name, x in (("k", k), ("v", v)):
        x = x.reshape(-1, hk, d)
        at = (s["row_page"], slice(None), s["row_slot"])
        whole = s[name].double()
        if case["cache"] == "e4m3":  # what the code would be with no rounding
            unit = 2.0 ** torch.ceil(torch.log2(x.abs().amax(-1) / E4M3_MAX)).clamp(EXP_LO, EXP_HI)
            scale = torch.exp2(s[name + "_exp"].double() - 127)
            scale[at] = unit
            out[name + "_scale"] = scale
            x = x / unit[..., None]
        whole[at] = x
        out[name] = whole
    return out


def _exact_copy(s, case):
    names = [n for n in ("k", "v", "k_exp", "v_exp", "bounds", "bound_exp") if s.get(n) is not None]
    for src, dst, n in zip(s["src"].tolist(), s["dst"].tolist(), s["tokens"].tolist()):
        for name in names:
            x = s[name]
            if not name.startswith("bound"):
                x.view(torch.uint8 if x.element_size() == 1 else x.dtype)[:, dst, :, :n] = \
                    x.view(torch.uint8 if x.element_size() == 1 else x.dtype)[:, src, :, :n]
            elif n == case["page"]:
                x[:, dst] = x[:, src]
    out = {"k": s["k"].double(), "v": s["v"].double()}
    if s["k_exp"] is not None:
        out["k_scale"], out["v_scale"] = (torch.exp2(s[n].double() - 127) for n in ("k_exp", "v_exp"))
    if case["bounded"]:
        out["bounds"], out["bound_exp"] = s["bounds"], s["bound_exp"]
    return out


def _exact_bounds(s, case):
    for pages in s["fresh"].split(256):
        k = s["k"][pages].double()
        if s["k_exp"] is not None:
            k = k * torch.exp2(s["k_exp"][pages].double() - 127)[..., None]
        top = k.abs().amax((2, 3))
        e = torch.ceil(torch.log2(top / BOUND_MAX)).clamp(-BOUND_EXP, BOUND_EXP)  # no top is this near to a border
        unit = torch.exp2(e)[..., None]
        s["bounds"][pages, :, 0] = (k.amax(2) / unit).round().to(torch.int8)
        s["bounds"][pages, :, 1] = (k.amin(2) / unit).round().to(torch.int8)
        s["bound_exp"][pages] = (e + 127).to(torch.uint8)
    return {"bounds": s["bounds"], "bound_exp": s["bound_exp"]}


def _exact_sparse(s, case):
    d, hk, page, select = case["dim"], case["kv_heads"], case["page"], case["select"]
    chosen = torch.full_like(s["chosen"], -1)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=chosen.device).reshape(-1, hk, case["heads"] // hk, d)
    row = 0
    for i, (n, kv) in enumerate(zip(s["new"], s["kv"])):
        ids = s["table"][i, :-(-kv // page)]
        hi, lo = (s["bounds"][ids][:, :, x].double().movedim(1, 0)[:, None] for x in (0, 1))  # [head, 1, page, dim]
        unit = torch.exp2(s["bound_exp"][ids].double() - 127).T
        for p in range(kv - n, kv):
            q = s["q"][row].double().reshape(hk, -1, d)
            top = q.abs().amax((1, 2), keepdim=True)
            step = torch.exp2(torch.ceil(torch.log2(top / BOUND_MAX)).clamp(-BOUND_EXP, BOUND_EXP))
            code = (q / step).round()[:, :, None]
            last = p // page
            take = torch.ones(hk, last + 1, dtype=torch.bool, device=chosen.device)
            if last + 1 > select:
                between = slice(case["first"], last + 1 - case["last"])
                x = torch.maximum(code * hi[:, :, between], code * lo[:, :, between]).sum(-1).amax(1) * unit[:, between]
                places = torch.arange(x.shape[1], device=x.device)
                before = (x[:, None] > x[:, :, None]) | ((x[:, None] == x[:, :, None]) & (places < places[:, None]))
                take[:, between] = before.sum(-1) < select - case["first"] - case["last"]
            for h in range(hk):
                at = take[h].nonzero()[:, 0]
                chosen[row, h, :len(at)] = ids[at].int()
                if case["op"] == "select":
                    continue
                seen = (at[:, None] * page + torch.arange(page, device=at.device)).flatten() <= p
                k, v = (_exact_values(s, name, ids[at], h)[seen] for name in ("k", "v"))
                out[row, h] = torch.softmax(q[h] @ k.T * s["scale"], -1) @ v
            row += 1
    return {"chosen": chosen} if case["op"] == "select" else {"chosen": chosen, "out": out.reshape(row, -1)}


def _exact_values(s, name, pages, head):
    x = s[name][pages, head].double()
    if s[name + "_exp"] is not None:
        x = x * torch.exp2(s[name + "_exp"][pages, head].double() - 127)[..., None]
    return x.flatten(0, 1)
