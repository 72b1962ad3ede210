"""The rest of a decoding step in numpy, float64, from the definitions: rows
of 4 bits, the extension of a paged cache by new tokens, and sampling.

Everything is walked one by one (a row, a token, a candidate at a time);
nothing is shared with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.cache import capacity, slots_of, where

NUMBERS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def code_of(y):
    """The 4-bit code of y: the nearest number, of two the even code; numbers
    beyond 6 as 6."""
    a = min(abs(y), 6.0)
    best = min(range(8), key=lambda i: (abs(NUMBERS[i] - a), i % 2))
    return best + (8 if math.copysign(1.0, y) < 0 else 0)


def block_byte(xs):
    """The scale byte of a block: the least s = 2^(byte - 127) with
    max |x| < 7 s."""
    top = max(abs(float(x)) for x in xs)
    if any(x != x for x in xs) or top == math.inf:
        return 255
    for byte in range(255):
        if top < 7 * 2.0 ** (byte - 127):
            return byte
    return 254


def pack(row):
    """(codes [D / 2], bytes [D / 32]), uint8, of a row."""
    codes, blocks = [], []
    for i in range(0, len(row), 32):
        xs = [float(x) for x in row[i:i + 32]]
        byte = block_byte(xs)
        blocks.append(byte)
        c = [0 if byte == 255 else code_of(x / 2.0 ** (byte - 127))
             for x in xs]
        codes += [c[j] | c[j + 1] << 4 for j in range(0, 32, 2)]
    return np.array(codes, np.uint8), np.array(blocks, np.uint8)


def unpack(codes, blocks):
    """Values [..., D] of codes [..., D / 2] and bytes [..., D / 32]."""
    n = np.array(NUMBERS + [-x for x in NUMBERS])
    x = np.stack([n[codes & 15], n[codes >> 4]], -1)
    x = x.reshape(codes.shape[:-1] + (-1, 32))
    s = np.exp2(blocks.astype(np.float64) - 127.0)
    s = np.where(blocks == 255, np.nan, s)
    return (x * s[..., None]).reshape(codes.shape[:-1] + (-1,))


def head_row(x, norm, eps, freqs, position, interleaved):
    """A head's row, normed and rotated."""
    y = [float(a) for a in x]
    if norm is not None:
        ms = math.fsum(a * a for a in y) / len(y)
        y = [a / math.sqrt(ms + eps) * float(g) for a, g in zip(y, norm)]
    half = 0 if freqs is None else len(freqs)
    for j in range(half):
        a = position * float(freqs[j])
        c, d = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        y[c], y[d] = (y[c] * math.cos(a) - y[d] * math.sin(a),
                      y[d] * math.cos(a) + y[c] * math.sin(a))
    return y


def extend(q, k, v, cache, starts, seen=None, q_norm=None, k_norm=None,
           eps=0.0, freqs=None, interleaved=False, k_scale=None, v_scale=None,
           slots=None):
    """(queries [N, Hq, D] (NaN where no sequence has the token), writes,
    lens): writes is a list of (page, head, place, row of k, row of v, b,
    slot, position); page None where the table names none, and only the
    position counts."""
    heads = cache["k"].shape[1]
    cap = capacity(cache, slots)
    lens = np.zeros(len(cache["lens"]), np.int32)
    out = None if q is None else np.full(q.shape, np.nan)
    writes = []
    for b in range(len(lens)):
        length = slots_of(cache["lens"], b, cap)
        first = int(length if seen is None else seen[b])
        n = int(starts[b + 1]) - int(starts[b])
        lens[b] = min(length + n, cap)
        for i in range(n):
            token, slot, pos = int(starts[b]) + i, length + i, first + i
            if q is not None:
                for h in range(q.shape[1]):
                    out[token, h] = head_row(q[token, h], q_norm, eps, freqs,
                                             pos, interleaved)
            if slot >= cap:
                continue
            at = where(cache, b, slot)
            for h in range(heads):
                x = np.array(head_row(k[token, h], k_norm, eps, freqs, pos,
                                      interleaved))
                z = np.array(v[token, h], np.float64)
                if k_scale is not None:
                    x = x / float(k_scale[h])
                if v_scale is not None:
                    z = z / float(v_scale[h])
                writes.append((None if at is None else at[0], h,
                               None if at is None else at[1], x, z, b, slot,
                               pos))
    return out, writes, lens


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability) of one row of numbers, in 64 bits; settings as
    float32 holds them."""
    t, p, m = (float(np.float32(x)) for x in (temperature, top_p, min_p))
    top_k = int(top_k)
    x = [-math.inf if a != a else float(a) for a in logits]
    top = max(x)
    if top == -math.inf:
        return -1, -math.inf
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))
    if not t > 0:
        return order[0], 0.0

    def weight(i):
        if x[i] == top:
            return 1.0
        if top == math.inf or x[i] == -math.inf:
            return 0.0
        return math.exp((x[i] - top) / t)

    if top_k > 0:
        order = order[:top_k]
    w = [weight(i) for i in order]
    if p < 1:
        need, part = p * math.fsum(w), 0.0
        for n, a in enumerate(w):
            part += a
            if part >= need:
                break
        order, w = order[:n + 1], w[:n + 1]
    if m > 0:
        order = [i for i, a in zip(order, w) if a >= min(m, 1.0)]
    order.sort()
    w = [weight(i) for i in order]
    total = math.fsum(w)
    u = float(u)
    goal = min(max(u, 0.0) if u == u else 0.0, 1.0) * total
    part, last = 0.0, None
    for i, a in zip(order, w):
        if a > 0:
            last = i
        part += a
        if part > goal:
            break
    return last, math.log(weight(last) / total)
