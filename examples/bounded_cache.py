"""Decoding with a cache of bounded length, by the library's cache operators.

A prompt fills a paged cache, attention over it accumulates every slot's
weight, cache_evict cuts it back to a budget, and from then on each new token
takes the place of the slot that has drawn the least weight (the first tokens
and the latest ones are protected).  Rows are made from the token's position,
so that what the cache holds can be checked.

    python examples/bounded_cache.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import top_selection_two_amd as ltk  # noqa: E402

SINKS, RECENT, PAGE = 4, 16, 16


def rows_of(positions, dim, salt):
    """A row of `dim` values for each position (stands for a projection)."""
    d = torch.arange(dim, device=positions.device, dtype=torch.float32)
    x = positions.float().unsqueeze(-1) * (0.37 + 0.11 * salt) + d * 0.9
    return torch.sin(x).to(torch.bfloat16)


def decode(batch, heads, group, dim, prompt, budget, tokens):
    dev = torch.device("cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    width = -(-(prompt + 1) // PAGE)
    pages = batch * width
    table = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = table.view(batch, width)
    k = torch.zeros(pages, heads, PAGE, dim, dtype=torch.bfloat16, device=dev)
    v = torch.zeros_like(k)
    # the prompt's rows, slot by slot
    pos = torch.arange(width * PAGE, device=dev, dtype=torch.int32)
    for cache, salt in ((k, 0), (v, 1)):
        rows = rows_of(pos, dim, salt).view(1, width, 1, PAGE, dim)
        cache[table.long()] = rows.expand(batch, width, heads, PAGE, dim)
    positions = pos.expand(batch, heads, -1).contiguous()
    weights = torch.zeros(batch, heads, width * PAGE, device=dev)
    lens = torch.full((batch,), prompt, dtype=torch.int32, device=dev)
    seen = lens.clone()

    def query():
        return torch.randn(batch, heads * group, dim, generator=g,
                           device=dev).to(torch.bfloat16)

    # the last prompt tokens' attention, a call each, says which slots matter
    for _ in range(4):
        ltk.cache_attend(query(), k, v, table, lens, weights=weights)
    weights, positions, lens = ltk.cache_evict(
        k, v, table, lens, seen, weights, positions, budget, sinks=SINKS,
        recent=RECENT)
    outs = []
    for _ in range(tokens):
        k_new = rows_of(seen.view(-1, 1).expand(batch, heads), dim, 0)
        v_new = rows_of(seen.view(-1, 1).expand(batch, heads), dim, 1)
        lens, _ = ltk.cache_append(k_new, v_new, k, v, table, lens, budget,
                                   seen, weights, positions, sinks=SINKS,
                                   recent=RECENT)
        seen = seen + 1
        out, _ = ltk.cache_attend(query(), k, v, table, lens, weights=weights)
        outs.append(out)
    return {"k": k, "v": v, "table": table, "positions": positions,
            "weights": weights, "lens": lens, "out": torch.stack(outs)}


def rows_match(r):
    """Does every slot hold the rows of its position?"""
    batch, heads, n = r["positions"].shape
    slot = torch.arange(n, device=r["k"].device)
    page = r["table"].long()[:, slot // PAGE]
    ok = True
    for name, salt in (("k", 0), ("v", 1)):
        have = r[name][page, :, slot % PAGE].transpose(1, 2)
        ok &= torch.equal(have, rows_of(r["positions"], r[name].shape[3],
                                        salt))
    return bool(ok)


if __name__ == "__main__":
    r = decode(batch=4, heads=8, group=4, dim=128, prompt=5000, budget=1024,
               tokens=100)
    torch.cuda.synchronize()
    print("100 tokens through a cache of 1024 slots a head; rows match their "
          "positions: %s; oldest token kept beyond the first %d: %d"
          % (rows_match(r), SINKS,
             int(r["positions"][r["positions"] >= SINKS].min())))
