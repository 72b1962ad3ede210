"""The paged-cache operators in numpy, float64, from their definitions.

A cache is a dict of k, v [pages, H, page, D] (any float array; copied where
it is changed), table [B, width] and lens [B].  Slot t of sequence b lies in
page table[b, t // page] at place t % page; an entry outside [0, pages) names
no page.  Slots are walked one by one; nothing is shared with the GPU path.
"""
from __future__ import annotations

import numpy as np

SAFE = 2 ** 31 - 1


def slots_of(lens, b, cap):
    return int(min(max(int(lens[b]), 0), cap))


def where(cache, b, t):
    """(page, place) of a slot, or None."""
    page = cache["k"].shape[2]
    p = int(cache["table"][b, t // page])
    if not 0 <= p < cache["k"].shape[0]:
        return None
    return p, t % page


def capacity(cache, slots=None):
    cap = cache["table"].shape[1] * cache["k"].shape[2]
    return cap if slots is None else min(cap, slots)


def attend(q, cache, scale, k_scale=None, v_scale=None, slots=None):
    """out [B, Hq, D], lse [B, Hq], added weights [B, H, cap], and
    spread [B, Hq, D] = sum p |v| and size [B, Hq] = max sum |q k| scale,
    which error bounds are made of."""
    q = np.asarray(q, np.float64)
    batch, hq, dim = q.shape
    heads = cache["k"].shape[1]
    group = hq // heads
    cap = capacity(cache, slots)
    out = np.zeros((batch, hq, dim))
    lse = np.full((batch, hq), -np.inf)
    added = np.zeros((batch, heads, cap))
    spread = np.zeros((batch, hq, dim))
    size = np.zeros((batch, hq))
    for b in range(batch):
        at = [(t, where(cache, b, t))
              for t in range(slots_of(cache["lens"], b, cap))]
        at = [(t, w) for t, w in at if w is not None]
        if not at:
            continue
        ts = np.array([t for t, _ in at])
        pages = np.array([w[0] for _, w in at])
        places = np.array([w[1] for _, w in at])
        for h in range(heads):
            k = cache["k"][pages, h, places].astype(np.float64)
            v = cache["v"][pages, h, places].astype(np.float64)
            if k_scale is not None:
                k = k * float(k_scale[h])
            if v_scale is not None:
                v = v * float(v_scale[h])
            for j in range(h * group, (h + 1) * group):
                x = (k @ q[b, j]) * scale
                size[b, j] = (np.abs(k) @ np.abs(q[b, j])).max() * abs(scale)
                top = x.max()
                if top == -np.inf:
                    continue
                e = np.exp(x - top)
                p = e / e.sum()
                lse[b, j] = top + np.log(e.sum())
                out[b, j] = p @ v
                spread[b, j] = p @ np.abs(v)
                added[b, h, ts] += p
    return out, lse, added, spread, size


def order(weights, positions, seen, sinks, recent):
    """Slots of one row from the first retained to the last."""
    keys = []
    for t in range(len(weights)):
        bits = int(np.float32(weights[t]).view(np.int32))
        key = bits if bits >= 0 else bits ^ 0x7fffffff
        pos = int(positions[t])
        if pos < sinks or pos >= int(seen) - recent:
            key = SAFE
        keys.append((-key, t))
    return [t for _, t in sorted(keys)]


def append(k_new, v_new, cache, limit, seen, weights, positions, sinks,
           recent):
    """(k, v, weights, positions, slots, lens) after the call."""
    k, v = cache["k"].copy(), cache["v"].copy()
    w, pos = weights.copy(), positions.copy()
    batch, heads, n = w.shape
    cap = capacity(cache, n)
    slots = np.zeros((batch, heads), np.int32)
    lens = np.zeros(batch, np.int32)
    for b in range(batch):
        length = slots_of(cache["lens"], b, cap)
        lens[b] = length
        for h in range(heads):
            if length < limit:
                t = length if length < cap else -1
                lens[b] = length + (t >= 0)
            else:
                t = order(w[b, h, :length], pos[b, h, :length], seen[b],
                          sinks, recent)[-1]
            slots[b, h] = t
            if t < 0:
                continue
            w[b, h, t] = 0.0
            pos[b, h, t] = seen[b]
            at = where(cache, b, t)
            if at is not None:
                k[at[0], h, at[1]] = k_new[b, h]
                v[at[0], h, at[1]] = v_new[b, h]
    return k, v, w, pos, slots, lens


def evict(cache, seen, weights, positions, keep, sinks, recent):
    """(k, v, weights, positions, lens) after the call."""
    k, v = cache["k"].copy(), cache["v"].copy()
    batch, heads, n = weights.shape
    cap = capacity(cache, n)
    w = np.zeros((batch, heads, keep), np.float32)
    pos = np.full((batch, heads, keep), -1, np.int32)
    lens = np.zeros(batch, np.int32)
    for b in range(batch):
        length = slots_of(cache["lens"], b, cap)
        lens[b] = min(length, keep)
        for h in range(heads):
            kept = set(order(weights[b, h, :length], positions[b, h, :length],
                             seen[b], sinks, recent)[:keep])
            source = {t: t for t in kept if t < keep}
            holes = [t for t in range(min(length, keep)) if t not in kept]
            movers = sorted(t for t in kept if t >= keep)
            for to, origin in zip(holes, movers):
                source[to] = origin
                a, z = where(cache, b, origin), where(cache, b, to)
                if a is not None and z is not None:
                    k[z[0], h, z[1]] = cache["k"][a[0], h, a[1]]
                    v[z[0], h, z[1]] = cache["v"][a[0], h, a[1]]
            for to, origin in source.items():
                w[b, h, to] = weights[b, h, origin]
                pos[b, h, to] = positions[b, h, origin]
    return k, v, w, pos, lens
