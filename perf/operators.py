"""The paged key-value cache operators of decoding, as they are measured.

Three operators work on one cache of K and V rows in pages (slot t of a
sequence lies in page table[b, t // page], place t % page):

  attend  attention of one new token over each sequence's slots, which also
          adds every slot's attention weight to an accumulated weight
  append  writes the new token's rows; in a full cache, in the place of the
          unprotected slot with the lowest accumulated weight
  evict   keeps the `keep` slots of the largest accumulated weight and moves
          the kept rows that lie beyond the new length into the holes below

With `own` false run() computes them from elementary torch operations in 32
bits; with `own` true it makes the calls that a user of
top_selection_two_amd makes.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16,
          "e4m3": torch.float8_e4m3fn}
GOLDEN = 0.6180339887498949
# The most that a drawn case may cost: bytes of cache rows in one pass.
DRAW_BYTES = 4e8


# ------------------------------------------------------------------- cases
def _attend(name, batch, lo, hi, heads, group, dim, page, dtype="bf16",
            cache=None, weights=True, slots_first=False):
    c = {"op": "attend", "batch": batch, "lo": lo, "hi": hi, "heads": heads,
         "group": group, "dim": dim, "page": page, "dtype": dtype,
         "cache": cache or dtype, "weights": weights,
         "slots_first": slots_first}
    return dict(c, name=name) if name else c


def _append(name, batch, lo, hi, heads, dim, page, limit, sinks, recent,
            dtype="bf16", slots_first=False):
    c = {"op": "append", "batch": batch, "lo": lo, "hi": hi, "heads": heads,
         "dim": dim, "page": page, "limit": limit, "sinks": sinks,
         "recent": recent, "dtype": dtype, "cache": dtype,
         "slots_first": slots_first}
    return dict(c, name=name) if name else c


def _evict(name, batch, lo, hi, heads, dim, page, keep, sinks, recent,
           dtype="bf16", slots_first=False):
    c = {"op": "evict", "batch": batch, "lo": lo, "hi": hi, "heads": heads,
         "dim": dim, "page": page, "keep": keep, "sinks": sinks,
         "recent": recent, "dtype": dtype, "cache": dtype,
         "slots_first": slots_first}
    return dict(c, name=name) if name else c


def listed():
    return [
        # One user's short chat: everything fits a fraction of the chip and
        # the call's latency is what the user waits for, once a layer.
        _attend("attend chat", 1, 211, 211, 8, 4, 128, 16),
        # A busy server's batch: sequences of every length side by side.
        _attend("attend batch", 48, 100, 8000, 8, 4, 128, 16,
                slots_first=True),
        # One long document: few rows, so the length has to be split.
        _attend("attend document", 1, 131072, 131072, 4, 8, 128, 256,
                weights=False),
        # The same kind of service with the cache held in 8 bits.
        _attend("attend 8-bit", 24, 2000, 15999, 8, 8, 128, 64,
                cache="e4m3"),
        # Every head with its own keys, small rows, pages that are no power
        # of two, sequences that have just begun (one has nothing yet).
        _attend("attend own heads", 7, 0, 1777, 12, 1, 64, 24, dtype="f16"),
        # One key head for all sixteen query heads, wide rows.
        _attend("attend one key head", 16, 2500, 5001, 1, 16, 256, 32),
        # A decoding step of one user whose cache is full.
        _append("append chat", 1, 1024, 1024, 8, 128, 16, 1024, 4, 64),
        # A large batch, most caches full, some still filling up.
        _append("append batch", 256, 3500, 4500, 8, 128, 16, 4096, 4, 256,
                slots_first=True),
        # A prompt somewhat over the budget, cut back to it.
        _evict("evict chat", 1, 1501, 1501, 8, 128, 16, 1024, 4, 64),
        # Several prompts cut to a quarter; one or two are short already.
        _evict("evict batch", 16, 1500, 8192, 8, 128, 16, 2048, 4, 256,
               slots_first=True),
        # A long document cut to an eighth.
        _evict("evict document", 1, 131072, 131072, 8, 128, 256, 16384, 4,
               1024),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    while True:
        op = rng.choice(("attend", "attend", "append", "evict"))
        dtype = rng.choice(("bf16", "bf16", "f16"))
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, 65536)
        lo = rng.randint(0, hi)
        heads = rng.choice((1, 2, 4, 8, 12))
        dim = rng.choice((64, 80, 96, 128, 128, 192, 256))
        page = rng.choice((8, 16, 16, 20, 32, 64, 100, 128, 256))
        slots_first = rng.random() < 0.4
        if batch * hi * heads * dim * 4 > DRAW_BYTES:
            continue
        if op == "attend":
            cache = dtype
            if dim % 16 == 0 and rng.random() < 0.3:
                cache = "e4m3"
            return _attend(None, batch, lo, hi, heads,
                           rng.choice((1, 2, 3, 4, 6, 7, 8, 12, 16, 20)),
                           dim, page, dtype, cache, rng.random() < 0.6,
                           slots_first)
        recent = rng.choice((0, 16, 64, 333))
        sinks = rng.choice((0, 4))
        if op == "append":
            limit = rng.randint(max(1, hi // 2), hi + 1)
            return _append(None, batch, lo, hi, heads, dim, page, limit,
                           sinks, recent, dtype, slots_first)
        keep = rng.randint(1, hi)
        return _evict(None, batch, lo, hi, heads, dim, page, keep, sinks,
                      recent, dtype, slots_first)


def _lens(case):
    """Slots in use of each sequence: spread over [lo, hi], both there."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    v = [lo + int((hi - lo) * ((i * GOLDEN) % 1.0)) for i in range(n)]
    v[-1] = hi
    return v


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    b, h, d, page = case["batch"], case["heads"], case["dim"], case["page"]
    lens = _lens(case)
    # append may add a slot to a sequence that is not full
    width = -(-(case["hi"] + (case["op"] == "append")) // page)
    width = max(width, 1)
    dtype, cdtype = DTYPES[case["dtype"]], DTYPES[case["cache"]]

    def rows():
        shape = (b * width, page, h, d) if case["slots_first"] else \
            (b * width, h, page, d)
        t = torch.empty(shape, dtype=dtype, device="cuda")
        t.normal_(generator=g)
        t = t.to(cdtype)
        return t.transpose(1, 2) if case["slots_first"] else t

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # the allocator hands out pages in any order
    table = torch.randperm(b * width, generator=g, device="cuda")
    s = {"case": case, "k": rows(), "v": rows(),
         "table": table.to(torch.int32).view(b, width),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "n": width * page}
    if case["cache"] == "e4m3":
        s["k_scale"] = 0.5 + torch.rand(h, generator=g, device="cuda")
        s["v_scale"] = 0.5 + torch.rand(h, generator=g, device="cuda")
    if case["op"] == "attend":
        s["q"] = (normal(b, h * case["group"], d) * 1.5).to(dtype)
        s["scale"] = d ** -0.5
        if case["weights"]:
            s["weights"] = torch.exp(1.5 * normal(b, h, s["n"]))
        return s
    # Weights accumulated so far: a few slots have drawn most of them.
    s["weights"] = torch.exp(1.5 * normal(b, h, s["n"]))
    if case["op"] == "evict":
        # a prompt's slots lie in order
        p = torch.arange(s["n"], dtype=torch.int32, device="cuda")
        s["positions"] = p.expand(b, h, -1).contiguous()
        s["seen"] = s["lens"].clone()
    else:
        # after many replacements a cache's slots are in no order, and each
        # head has kept others
        p = torch.rand(b, h, s["n"], generator=g, device="cuda").argsort(2)
        s["positions"] = (3 * p).to(torch.int32)
        s["seen"] = torch.full((b,), 3 * s["n"], dtype=torch.int32,
                               device="cuda")
        s["k_new"] = normal(b, h, d).to(dtype)
        s["v_new"] = normal(b, h, d).to(dtype)
    return s


# --------------------------------------------------------------- plain form
def _gather(cache, table, scale):
    """The rows of every slot of the table, float32 [B, H, slots, D]."""
    b, w = table.shape
    _, h, page, d = cache.shape
    if cache.dtype == torch.float8_e4m3fn:
        r = cache.view(torch.uint8)[table.long()].view(torch.float8_e4m3fn)
    else:
        r = cache[table.long()]
    r = r.transpose(1, 2).reshape(b, h, w * page, d).float()
    return r if scale is None else r * scale.view(1, h, 1, 1)


def _plain_attend(s):
    q = s["q"].float()
    b, hq, d = q.shape
    k = _gather(s["k"], s["table"], s.get("k_scale"))
    v = _gather(s["v"], s["table"], s.get("v_scale"))
    h, n = k.shape[1], k.shape[2]
    q = q.view(b, h, hq // h, d).transpose(2, 3).contiguous()
    used = (torch.arange(n, device=q.device) < s["lens"][:, None])
    used = used.view(b, 1, n, 1)
    x = (torch.matmul(k, q) * s["scale"]).masked_fill(~used, -torch.inf)
    top = x.amax(2, keepdim=True)
    e = torch.exp(x - top.masked_fill(top == -torch.inf, 0.0))
    total = e.sum(2, keepdim=True)
    p = e / total.masked_fill(total == 0, 1.0)
    out = torch.matmul(p.transpose(2, 3).contiguous(),
                       v.masked_fill(~used, 0.0))
    r = {"out": out.reshape(b, hq, d).to(s["q"].dtype),
         "lse": (top + torch.log(total)).reshape(b, hq)}
    if "weights" in s:
        s["weights"] += p.sum(3)
        r["weights"] = s["weights"]
    return r


def _ranks(s):
    """One int64 a slot, larger for what is kept before: protected slots
    (all alike), then by weight; the earlier slot where these are equal."""
    c = s["case"]
    bits = s["weights"].view(torch.int32)
    key = bits ^ ((bits >> 31) & 0x7fffffff)
    pos, seen = s["positions"], s["seen"].view(-1, 1, 1)
    safe = (pos < c["sinks"]) | (pos >= seen - c["recent"])
    key = key.masked_fill(safe, 0x7fffffff).long()
    slot = torch.arange(s["n"], device=key.device)
    rank = key * 2 ** 31 + (2 ** 31 - 1 - slot)
    return rank, slot < s["lens"].view(-1, 1, 1)


def _place(s, slot):
    """Page, head and place in the page of slots [B, H, m]."""
    page = s["case"]["page"]
    b, h, m = slot.shape
    pages = s["table"].long().gather(1, (slot // page).view(b, h * m))
    heads = torch.arange(h, device=slot.device).view(1, h, 1)
    return pages.view(b, h, m), heads.expand(b, h, m), slot % page


def _plain_append(s):
    c = s["case"]
    rank, used = _ranks(s)
    lowest = rank.masked_fill(~used, 2 ** 63 - 1).argmin(2)
    lens = s["lens"].long().view(-1, 1)
    slot = torch.where(lens < c["limit"], lens, lowest)
    at = _place(s, slot[:, :, None])
    s["k"][at] = s["k_new"][:, :, None]
    s["v"][at] = s["v_new"][:, :, None]
    s["weights"].scatter_(2, slot[:, :, None], 0.0)
    s["positions"].scatter_(2, slot[:, :, None],
                            s["seen"].view(-1, 1, 1).expand(slot.shape
                                                            + (1,)))
    return {"k": s["k"], "v": s["v"], "weights": s["weights"],
            "positions": s["positions"], "slots": slot.int(),
            "lens": (s["lens"] + (s["lens"] < c["limit"])).int()}


def _plain_evict(s):
    keep, n = s["case"]["keep"], s["n"]
    rank, used = _ranks(s)
    b, h, _ = rank.shape
    lens = s["lens"].long().view(-1, 1, 1)
    rank = rank.masked_fill(~used, -2 ** 63)
    best = rank.topk(min(keep, n), dim=2).indices
    kept = torch.zeros_like(used.expand(b, h, n)).scatter_(2, best, True)
    kept &= used
    slot = torch.arange(n, device=rank.device).expand(b, h, n)
    m = min(keep, max(n - keep, 0))
    holes = slot.masked_fill(kept | ~used | (slot >= keep), n)
    holes = holes.sort(2).values[:, :, :m]
    movers = slot.masked_fill(~kept | (slot < keep), n).sort(2)
    movers = movers.values[:, :, :m]
    # Pairs past a row's last move put the row's last slot onto itself: no
    # move writes there (it lies at or beyond keep, or nothing moves).
    none = movers == n
    last = (lens - 1).clamp(min=0).expand(b, h, m)
    src = torch.where(none, last, movers)
    dst = torch.where(none, last, holes)
    a, z = _place(s, src), _place(s, dst)
    s["k"][z] = s["k"][a]
    s["v"][z] = s["v"][a]
    w = s["weights"].clone()
    w.scatter_(2, dst, s["weights"].gather(2, src))
    p = s["positions"].clone()
    p.scatter_(2, dst, s["positions"].gather(2, src))
    cut = min(keep, n)
    left = slot[:, :, :cut] >= lens
    w = w[:, :, :cut].masked_fill(left, 0.0)
    p = p[:, :, :cut].masked_fill(left, -1)
    if keep > n:
        w = torch.nn.functional.pad(w, (0, keep - n))
        p = torch.nn.functional.pad(p, (0, keep - n), value=-1)
    return {"k": s["k"], "v": s["v"], "weights": w, "positions": p,
            "lens": s["lens"].clamp(max=keep)}


# ------------------------------------------------------- the framework's own
def _own_attend(s):
    import top_selection_two_amd as ltk
    out, lse = ltk.cache_attend(
        s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"],
        weights=s.get("weights"), k_scale=s.get("k_scale"),
        v_scale=s.get("v_scale"))
    r = {"out": out, "lse": lse}
    if "weights" in s:
        r["weights"] = s["weights"]
    return r


def _own_append(s):
    import top_selection_two_amd as ltk
    c = s["case"]
    lens, slots = ltk.cache_append(
        s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"],
        limit=c["limit"], seen=s["seen"], weights=s["weights"],
        positions=s["positions"], sinks=c["sinks"], recent=c["recent"])
    return {"k": s["k"], "v": s["v"], "weights": s["weights"],
            "positions": s["positions"], "slots": slots, "lens": lens}


def _own_evict(s):
    import top_selection_two_amd as ltk
    c = s["case"]
    weights, positions, lens = ltk.cache_evict(
        s["k"], s["v"], s["table"], s["lens"], s["seen"], s["weights"],
        s["positions"], c["keep"], sinks=c["sinks"], recent=c["recent"])
    return {"k": s["k"], "v": s["v"], "weights": weights,
            "positions": positions, "lens": lens}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append,
                "evict": _own_evict}[op](state)
    return {"attend": _plain_attend, "append": _plain_append,
            "evict": _plain_evict}[op](state)


# ---------------------------------------------------------------- the floor
def work(case):
    lens, h, d = _lens(case), case["heads"], case["dim"]
    size = 1 if case["cache"] == "e4m3" else 2
    n, b = sum(lens), case["batch"]
    table = sum(-(-x // case["page"]) for x in lens) * 4
    if case["op"] == "attend":
        hq = h * case["group"]
        return {"bytes": 2 * n * h * d * size + 2 * b * hq * d * 2
                + 4 * b * hq + table + 4 * b
                + (8 * n * h if case["weights"] else 0),
                "flops": 4 * n * hq * d}
    if case["op"] == "append":
        full = sum(x for x in lens if x >= case["limit"])
        # weights and positions of full sequences; two rows in and out
        return {"bytes": 8 * full * h + b * h * (4 * d * size + 16) + 16 * b,
                "flops": full * h}
    keep = case["keep"]
    # A slot of a longer sequence is kept with probability keep / n, so
    # about keep * (n - keep) / n rows move, twice, in and out.
    moved = sum(keep * (x - keep) / x for x in lens if x > keep)
    stay = sum(min(x, keep) for x in lens)
    return {"bytes": h * (8 * n + 8 * stay + moved * 4 * d * size) + table
            + 12 * b, "flops": n * h}


# ------------------------------------------------- 64 bits, written apart
def _slot_rows(cache, table_row, n):
    """Rows [n, H, D] of one sequence, float64, slot by slot."""
    page = cache.shape[2]
    t = torch.arange(n, device=cache.device)
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn \
        else cache
    r = raw[table_row.long()[t // page], :, t % page]
    return r.view(cache.dtype).double()


def _exact_attend(s):
    outs, lses = [], []
    w = s["weights"].double() if "weights" in s else None
    h = s["k"].shape[1]
    b, hq, d = s["q"].shape
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            outs.append(torch.zeros(hq, d, dtype=torch.float64,
                                    device="cuda"))
            lses.append(torch.full((hq,), -torch.inf, dtype=torch.float64,
                                   device="cuda"))
            continue
        k = _slot_rows(s["k"], s["table"][i], n)
        v = _slot_rows(s["v"], s["table"][i], n)
        if "k_scale" in s:
            k *= s["k_scale"].double()[None, :, None]
            v *= s["v_scale"].double()[None, :, None]
        o = torch.empty(hq, d, dtype=torch.float64, device="cuda")
        z = torch.empty(hq, dtype=torch.float64, device="cuda")
        for j in range(hq):
            head = j // (hq // h)
            x = (k[:, head] @ s["q"][i, j].double()) * s["scale"]
            z[j] = torch.logsumexp(x, 0)
            p = torch.exp(x - z[j])
            o[j] = p @ v[:, head]
            if w is not None:
                w[i, head, :n] += p
        outs.append(o)
        lses.append(z)
    r = {"out": torch.stack(outs), "lse": torch.stack(lses)}
    if w is not None:
        r["weights"] = w
    return r


def _order(c, weights, positions, seen):
    """Slots of one head from the first kept to the last, numpy."""
    safe = (positions < c["sinks"]) | (positions >= seen - c["recent"])
    rank = np.where(safe, np.inf, weights.astype(np.float64))
    return np.lexsort((np.arange(len(rank)), -rank))


def _host(s, name):
    return s[name].cpu().numpy()


def _exact_append(s):
    c, page = s["case"], s["case"]["page"]
    w, pos = _host(s, "weights").copy(), _host(s, "positions").copy()
    lens, seen, table = _host(s, "lens"), _host(s, "seen"), _host(s, "table")
    b, h, _ = w.shape
    slots = np.zeros((b, h), np.int32)
    places = []
    for i in range(b):
        for j in range(h):
            n = int(lens[i])
            t = n if n < c["limit"] else \
                int(_order(c, w[i, j, :n], pos[i, j, :n], seen[i])[-1])
            slots[i, j] = t
            w[i, j, t] = 0.0
            pos[i, j, t] = seen[i]
            places.append((table[i, t // page], j, t % page))
    at = torch.tensor(places, dtype=torch.int64, device="cuda")
    for name in ("k", "v"):
        s[name][at[:, 0], at[:, 1], at[:, 2]] = s[name + "_new"].reshape(
            b * h, -1)
    return {"k": s["k"], "v": s["v"], "weights": w, "positions": pos,
            "slots": slots,
            "lens": np.where(lens < c["limit"], lens + 1, lens)}


def _exact_evict(s):
    c, page = s["case"], s["case"]["page"]
    keep = c["keep"]
    w, pos = _host(s, "weights"), _host(s, "positions")
    lens, seen, table = _host(s, "lens"), _host(s, "seen"), _host(s, "table")
    b, h, _ = w.shape
    new_w = np.zeros((b, h, keep), np.float32)
    new_p = np.full((b, h, keep), -1, np.int32)
    moves = []
    for i in range(b):
        for j in range(h):
            n = int(lens[i])
            kept = _order(c, w[i, j, :n], pos[i, j, :n], seen[i])[:keep]
            low = np.zeros(min(n, keep), bool)
            low[kept[kept < keep]] = True
            holes = np.nonzero(~low)[0]
            movers = np.sort(kept[kept >= keep])
            source = np.arange(min(n, keep))
            source[holes] = movers
            new_w[i, j, :len(source)] = w[i, j, source]
            new_p[i, j, :len(source)] = pos[i, j, source]
            moves.append(np.stack([
                table[i, movers // page], np.full(len(movers), j),
                movers % page, table[i, holes // page],
                np.full(len(movers), j), holes % page], 1))
    at = torch.from_numpy(np.concatenate(moves)).long().cuda()
    for name in ("k", "v"):
        x = s[name]
        x[at[:, 3], at[:, 4], at[:, 5]] = x[at[:, 0], at[:, 1], at[:, 2]]
    return {"k": s["k"], "v": s["v"], "weights": new_w, "positions": new_p,
            "lens": np.minimum(lens, keep)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append,
            "evict": _exact_evict}[case["op"]](s)
