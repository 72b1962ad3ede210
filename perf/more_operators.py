"""The rest of a decoding step, as it is measured.

  extend  new tokens' heads enter a paged cache: queries and keys normed and
          rotated by position, keys and values rounded to the cache's type
          (16 bits, e4m3, or 4 bits with a scale for each 32 elements)
  attend  attention of one new token over a cache held in 4 bits
  sample  a token for each row of logits by temperature, top-k, top-p and
          min-p from given random numbers

With `own` false run() computes them from elementary torch operations, with
`own` true it makes the calls that a user of top_selection_two_amd makes.
Rotations, roundings to few bits and cumulated probabilities are computed in
64 bits in the plain form: results lie next to borders there.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e2m1": torch.float4_e2m1fn_x2}
GOLDEN = 0.6180339887498949
EPS = 1e-6
# The most that a drawn case may cost.
DRAW_BYTES = 1.2e8


# ------------------------------------------------------------------- cases
def _extend(name, batch, lo, hi, held, q_heads, heads, dim, page,
            dtype="bf16", cache="bf16", rot=None, interleaved=False,
            norm=True, slots_first=False):
    c = {"op": "extend", "batch": batch, "lo": lo, "hi": hi, "held": held,
         "q_heads": q_heads, "heads": heads, "dim": dim, "page": page,
         "dtype": dtype, "cache": cache, "rot": dim if rot is None else rot,
         "interleaved": interleaved, "norm": norm,
         "slots_first": slots_first}
    return dict(c, name=name) if name else c


def _attend(name, batch, lo, hi, heads, group, dim, page, dtype="bf16",
            weights=True, slots_first=False):
    c = {"op": "attend", "batch": batch, "lo": lo, "hi": hi, "heads": heads,
         "group": group, "dim": dim, "page": page, "dtype": dtype,
         "weights": weights, "slots_first": slots_first}
    return dict(c, name=name) if name else c


def _sample(name, rows, cols, dtype, temperature, top_k=0, top_p=1.0,
            min_p=0.0, mixed=False, pad=0):
    c = {"op": "sample", "rows": rows, "cols": cols, "dtype": dtype,
         "temperature": temperature, "top_k": top_k, "top_p": top_p,
         "min_p": min_p, "mixed": mixed, "pad": pad}
    return dict(c, name=name) if name else c


def listed():
    return [
        # One token of each of a busy server's sequences, once a layer: the
        # heads are slices of one projection's output.
        _extend("extend step", 64, 1, 1, 4000, 32, 8, 128, 16),
        # A batch of prompts and parts of prompts.
        _extend("extend prompts", 12, 100, 4001, 500, 32, 8, 128, 16,
                slots_first=True),
        # Small own heads, some of their elements rotated, pairs side by
        # side, pages that are no power of two, some sequences without a
        # token, a cache held in 8 bits.
        _extend("extend 8-bit", 9, 0, 777, 100, 12, 12, 64, 24, "f16", "e4m3",
                rot=32, interleaved=True, norm=False),
        # Prompts into a cache held in 4 bits.
        _extend("extend 4-bit", 6, 700, 2048, 0, 16, 4, 128, 64,
                cache="e2m1"),
        # One user's short chat over 4-bit rows.
        _attend("attend chat", 1, 211, 211, 8, 4, 128, 16),
        # A busy server's batch: sequences of every length side by side.
        _attend("attend batch", 48, 100, 8000, 8, 4, 128, 16,
                slots_first=True),
        # One long document: few rows, so the length has to be split.
        _attend("attend document", 1, 131072, 131072, 4, 8, 128, 256,
                weights=False),
        # float16 queries over own heads of 64 elements in odd pages; one
        # sequence has nothing yet.
        _attend("attend own heads", 7, 0, 1777, 12, 1, 64, 24, dtype="f16"),
        # One user's next token.
        _sample("sample one", 1, 32000, "f32", 0.7, 50, 0.9),
        # A server's batch: each request with settings of its own.
        _sample("sample batch", 256, 131072, "bf16", 0.8, mixed=True),
        # Sampling without truncation, as for training on own samples: rows
        # of an odd length, padded.
        _sample("sample all", 64, 100003, "f32", 1.0, pad=5),
        # Creative settings: the nucleus is most of the vocabulary.
        _sample("sample wide", 32, 200000, "f16", 1.5, top_p=0.98),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    while True:
        op = rng.choice(("extend", "attend", "sample"))
        if op == "sample":
            dtype = rng.choice(("f32", "bf16", "f16"))
            rows, cols = _log(rng, 1, 512), _log(rng, 2, 262144)
            if rows * cols * 4 > DRAW_BYTES:
                continue
            return _sample(None, rows, cols, dtype,
                           round(rng.uniform(0.3, 1.6), 3),
                           rng.choice((0, 0, 1, 20, 50, 333, 2000)),
                           rng.choice((1.0, 1.0, 0.5, 0.9, 0.95, 0.99)),
                           rng.choice((0.0, 0.0, 0.02, 0.1)),
                           rng.random() < 0.4, rng.choice((0, 0, 1, 3, 8)))
        dtype = rng.choice(("bf16", "bf16", "f16"))
        heads = rng.choice((1, 2, 4, 8, 12))
        page = rng.choice((8, 16, 16, 20, 32, 64, 100, 128, 256))
        slots_first = rng.random() < 0.4
        batch = _log(rng, 1, 64)
        if op == "attend":
            dim = rng.choice((64, 96, 128, 128, 192, 256))
            hi = _log(rng, 1, 65536)
            if batch * hi * heads * dim * 4 > DRAW_BYTES * 4:
                continue
            return _attend(None, batch, rng.randint(0, hi), hi, heads,
                           rng.choice((1, 2, 3, 4, 6, 7, 8, 12, 16, 20)),
                           dim, page, dtype, rng.random() < 0.6, slots_first)
        cache = rng.choice((dtype, dtype, "e4m3", "e2m1"))
        dim = rng.choice((64, 96, 128, 128, 192, 256) if cache == "e2m1" else
                         (64, 80, 96, 128, 128, 192, 256))
        hi, held = _log(rng, 1, 8192), _log(rng, 1, 8192)
        q_heads = heads * rng.choice((1, 2, 4, 8))
        if (batch * hi * (q_heads + 2 * heads) * dim * 2 > DRAW_BYTES
                or batch * (hi + held) * heads * dim * 4 > DRAW_BYTES * 2):
            continue
        return _extend(None, batch, rng.randint(0, hi), hi, held, q_heads,
                       heads, dim, page, dtype, cache,
                       rng.choice((dim, dim, dim // 32 * 16, 0)),
                       rng.random() < 0.3, rng.random() < 0.5, slots_first)


def _lens(case):
    """Slots in use, or new tokens, of each sequence: spread over [lo, hi],
    both there."""
    lo, hi, n = case["lo"], case["hi"], case["batch"]
    v = [lo + int((hi - lo) * ((i * GOLDEN) % 1.0)) for i in range(n)]
    v[-1] = hi
    return v


def _held(case):
    """Slots in use before the new tokens."""
    n, held = case["batch"], case["held"]
    return [held - int(held / 2 * ((i * GOLDEN) % 1.0)) for i in range(n)]


# ---------------------------------------------------------------- 4-bit rows
def _pack(x):
    """Rows [..., D] as 4-bit codes, the even element in the low half of a
    byte, and a byte for each 32 elements: s = 2^(byte - 127), the least with
    amax < 7 s."""
    x = x.double()
    blocks = x.unflatten(-1, (-1, 32))
    top = blocks.abs().amax(-1)
    m, e = torch.frexp(top)
    e = (e - 2 - (m < 0.875).to(e.dtype)).clamp(-127, 127)
    e = e.masked_fill(top == 0, -127)
    y = blocks / torch.exp2(e.double()).unsqueeze(-1)
    a = y.abs()
    step = 0.5 + 0.5 * (a >= 2) + 1.0 * (a >= 4)
    a = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code, (e + 127).to(torch.uint8)


def _code_pairs():
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.bfloat16)
    v = torch.cat([v, -v])
    i = torch.arange(256)
    return torch.stack([v[i % 16], v[i // 16]], 1).cuda()


def _values(s, name):
    """The values that a 4-bit array stands for, in bfloat16 (exact)."""
    codes = s[name].view(torch.uint8)
    x = torch.nn.functional.embedding(codes.int(), s["pairs"])
    x = x.flatten(-2).unflatten(-1, (-1, 32))
    return (x * s[name + "_blocks"].to(torch.bfloat16).unsqueeze(-1)
            ).flatten(-2)


# ------------------------------------------------------------------ inputs
def _prepare_sample(case, g):
    rows, cols = case["rows"], case["cols"]
    dtype = DTYPES[case["dtype"]]
    # A vocabulary's logits fall with the logarithm of a token's rank, each
    # row in an order of its own, some rows steeper than others.
    x = torch.rand(rows, cols, generator=g, device="cuda")
    steep = 1.0 + torch.rand(rows, 1, generator=g, device="cuda")
    x = -steep * torch.log(x * cols + 1.0)
    x += 0.3 * torch.randn(rows, cols, generator=g, device="cuda") + 12.0
    logits = torch.full((rows, cols + case["pad"]), 99.0, dtype=dtype,
                        device="cuda")
    logits[:, :cols] = x
    s = {"case": case, "logits": logits[:, :cols],
         "u": torch.rand(rows, generator=g, device="cuda")}
    t, k, p, m = (case[n] for n in ("temperature", "top_k", "top_p", "min_p"))
    if case["mixed"]:
        i = torch.arange(rows, device="cuda")
        t = torch.full((rows,), t, device="cuda") * (0.7 + 0.1 * (i % 7))
        t = t.masked_fill(i % 11 == 10, 0.0)  # greedy
        k = torch.where(i % 4 == 1, 40, torch.where(i % 4 == 3, 500, 0))
        k = k.to(torch.int32)
        p = torch.where(i % 3 == 0, 0.9, torch.where(i % 3 == 1, 0.97, 1.0))
        p = p.float()
        m = torch.where(i % 5 == 2, 0.05, 0.0).float()
    s.update(temperature=t, top_k=k, top_p=p, min_p=m)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] == "sample":
        return _prepare_sample(case, g)
    b, h, d, page = case["batch"], case["heads"], case["dim"], case["page"]
    dtype = DTYPES[case["dtype"]]
    extend = case["op"] == "extend"
    new = _lens(case) if extend else None
    lens = _held(case) if extend else _lens(case)
    most = max(n + m for n, m in zip(lens, new)) if extend else case["hi"]
    width = max(-(-most // page), 1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    table = torch.randperm(b * width, generator=g, device="cuda")
    s = {"case": case, "table": table.to(torch.int32).view(b, width),
         "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "n": width * page}
    kind = case["cache"] if extend else "e2m1"

    def arrange(t):
        return t.transpose(1, 2) if case["slots_first"] else t

    shape = (b * width, page, h) if case["slots_first"] else \
        (b * width, h, page)
    for name in ("k", "v"):
        x = torch.empty(*shape, d, dtype=torch.bfloat16, device="cuda")
        x.normal_(generator=g)
        if kind == "e2m1":
            parts = [_pack(r) for r in x.split(4096)]
            codes = torch.cat([r[0] for r in parts])
            blocks = torch.cat([r[1] for r in parts])
            s[name] = arrange(codes).view(torch.float4_e2m1fn_x2)
            s[name + "_blocks"] = arrange(blocks).view(torch.float8_e8m0fnu)
        else:
            s[name] = arrange(x.to(DTYPES[kind]))
    if kind == "e2m1":
        s["pairs"] = _code_pairs()
    if not extend:
        s["q"] = (normal(b, h * case["group"], d) * 1.5).to(dtype)
        s["scale"] = d ** -0.5
        if case["weights"]:
            s["weights"] = torch.exp(1.5 * normal(b, h, s["n"]))
        return s
    starts = np.concatenate([[0], np.cumsum(new)])
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    # a cache that has been cut back holds fewer slots than tokens were seen
    s["seen"] = s["lens"] * 3
    n, hq = int(starts[-1]), case["q_heads"]
    s["qkv"] = normal(n, (hq + 2 * h) * d).to(dtype)
    s["freqs"] = None
    if case["rot"]:
        j = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
        s["freqs"] = (10000.0 ** (-2 * j / case["rot"])).float()
    s["q_norm"] = s["k_norm"] = s["k_scale"] = s["v_scale"] = None
    if case["norm"]:
        s["q_norm"] = (1 + 0.1 * normal(d)).to(dtype)
        s["k_norm"] = (1 + 0.1 * normal(d)).to(dtype)
    if kind == "e4m3":
        s["k_scale"] = 0.01 + 0.01 * torch.rand(h, generator=g, device="cuda")
        s["v_scale"] = 0.01 + 0.01 * torch.rand(h, generator=g, device="cuda")
    return s


def _heads(s):
    """Queries, keys and values of the new tokens, slices of one array."""
    c = s["case"]
    hq, h, d = c["q_heads"], c["heads"], c["dim"]
    x = s["qkv"].unflatten(1, (hq + 2 * h, d))
    return x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]


# --------------------------------------------------------------- plain form
def _normed(x, g):
    if g is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * g.double()


def _rotated(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([y.flatten(-2), x[..., r:]], -1)
    a, b = x[..., :r // 2], x[..., r // 2:r]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)


def _plain_extend(s):
    c = s["case"]
    q, k, v = (t.double() for t in _heads(s))
    starts, lens = s["starts"].long(), s["lens"].long()
    i = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(starts, i, right=True) - 1
    slot = lens[b] + i - starts[b]
    q, k = _normed(q, s["q_norm"]), _normed(k, s["k_norm"])
    if s["freqs"] is not None:
        pos = s["seen"].long()[b] + i - starts[b]
        a = pos.double()[:, None] * s["freqs"].double()
        cos, sin = a.cos()[:, None], a.sin()[:, None]
        q = _rotated(q, cos, sin, c["interleaved"])
        k = _rotated(k, cos, sin, c["interleaved"])
    page = s["table"].long()[b, slot // c["page"]]
    place = slot % c["page"]
    for name, x in (("k", k), ("v", v)):
        if c["cache"] == "e2m1":
            codes, blocks = _pack(x)
            s[name].view(torch.uint8)[page, :, place] = codes
            s[name + "_blocks"].view(torch.uint8)[page, :, place] = blocks
        elif c["cache"] == "e4m3":
            x = x / s[name + "_scale"].double()[:, None]
            x = x.clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn)
            s[name].view(torch.uint8)[page, :, place] = x.view(torch.uint8)
        else:
            s[name][page, :, place] = x.to(s[name].dtype)
    return _extended(s, q.to(DTYPES[c["dtype"]]),
                     (lens + starts[1:] - starts[:-1]).int())


def _extended(s, q, lens):
    r = {"q": q, "lens": lens, "k": s["k"], "v": s["v"]}
    if s["case"]["cache"] == "e2m1":
        r["k"], r["v"] = _values(s, "k"), _values(s, "v")
    return r


def _rows(s, name):
    """The values of every slot of the table, float32 [B, H, slots, D]."""
    b, w = s["table"].shape
    page = s["table"].long()
    codes = s[name].view(torch.uint8)[page].int()
    x = torch.nn.functional.embedding(codes, s["pairs"].float())
    x = x.flatten(-2).unflatten(-1, (-1, 32))
    scale = s[name + "_blocks"].view(torch.uint8)[page].float() - 127.0
    x = (x * torch.exp2(scale).unsqueeze(-1)).flatten(-2)
    h, d = x.shape[2], x.shape[4]
    return x.transpose(1, 2).reshape(b, h, s["n"], d)


def _plain_attend(s):
    q = s["q"].float()
    b, hq, d = q.shape
    k, v = _rows(s, "k"), _rows(s, "v")
    h, n = k.shape[1], k.shape[2]
    q = q.view(b, h, hq // h, d).transpose(2, 3).contiguous()
    used = (torch.arange(n, device=q.device) < s["lens"][:, None])
    used = used.view(b, 1, n, 1)
    x = (torch.matmul(k, q) * s["scale"]).masked_fill(~used, -torch.inf)
    top = x.amax(2, keepdim=True)
    e = torch.exp(x - top.masked_fill(top == -torch.inf, 0.0))
    total = e.sum(2, keepdim=True)
    p = e / total.masked_fill(total == 0, 1.0)
    out = torch.matmul(p.transpose(2, 3).contiguous(), v)
    r = {"out": out.reshape(b, hq, d).to(s["q"].dtype),
         "lse": (top + torch.log(total)).reshape(b, hq)}
    if "weights" in s:
        s["weights"] += p.sum(3)
        r["weights"] = s["weights"]
    return r


def _settings(s, name):
    """A setting as float64 [rows, 1] (it is given in float32)."""
    x, rows = s[name], s["case"]["rows"]
    if not torch.is_tensor(x):
        x = torch.full((rows,), x, dtype=torch.float32, device="cuda")
    return x.double().view(rows, 1)


def _plain_sample(s):
    t, top_k = _settings(s, "temperature"), _settings(s, "top_k")
    top_p, min_p = _settings(s, "top_p"), _settings(s, "min_p")
    x, order = s["logits"].double().sort(dim=1, descending=True,
                                           stable=True)
    greedy = t <= 0
    w = torch.exp((x - x[:, :1]) / t.masked_fill(greedy, 1.0))
    rank = torch.arange(x.shape[1], device=x.device)
    w = w * ((top_k <= 0) | (rank < top_k))
    before = w.cumsum(1)
    total = before[:, -1:]
    before = before - w
    keep = (before < top_p * total) & (w >= min_p.clamp(max=1.0))
    keep = keep.masked_fill(greedy, False)
    keep[:, 0] = True
    z = torch.zeros_like(w).scatter_(1, order, w * keep)
    c = z.cumsum(1)
    total = c[:, -1:]
    token = (c <= s["u"].double().view(-1, 1) * total).sum(1, keepdim=True)
    p = z.gather(1, token) / total
    return {"tokens": token.view(-1), "logprobs": p.log().float().view(-1)}


# ------------------------------------------------------- the framework's own
def _own_extend(s):
    import top_selection_two_amd as ltk
    q, k, v = _heads(s)
    lens, q = ltk.cache_extend(
        k, v, s["k"], s["v"], s["table"], s["lens"], s["starts"],
        seen=s["seen"], q=q, freqs=s["freqs"],
        interleaved=s["case"]["interleaved"], q_norm=s["q_norm"],
        k_norm=s["k_norm"], eps=EPS, k_scale=s["k_scale"],
        v_scale=s["v_scale"], k_blocks=s.get("k_blocks"),
        v_blocks=s.get("v_blocks"))
    return _extended(s, q, lens)


def _own_attend(s):
    import top_selection_two_amd as ltk
    out, lse = ltk.cache_attend(
        s["q"], s["k"], s["v"], s["table"], s["lens"], scale=s["scale"],
        weights=s.get("weights"), k_blocks=s["k_blocks"],
        v_blocks=s["v_blocks"])
    r = {"out": out, "lse": lse}
    if "weights" in s:
        r["weights"] = s["weights"]
    return r


def _own_sample(s):
    import top_selection_two_amd as ltk
    tokens, logprobs = ltk.sample(
        s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
        top_p=s["top_p"], min_p=s["min_p"])
    return {"tokens": tokens, "logprobs": logprobs}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"extend": _own_extend, "attend": _own_attend,
                "sample": _own_sample}[op](state)
    return {"extend": _plain_extend, "attend": _plain_attend,
            "sample": _plain_sample}[op](state)


# ---------------------------------------------------------------- the floor
def _row_bytes(kind, dim):
    return {"bf16": 2 * dim, "f16": 2 * dim, "e4m3": dim,
            "e2m1": dim // 2 + dim // 32}[kind]


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["cols"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * size + case["rows"] * 16, "flops": 4 * n}
    b, h, d = case["batch"], case["heads"], case["dim"]
    lens = _lens(case)
    n = sum(lens)
    if case["op"] == "attend":
        hq = h * case["group"]
        table = sum(-(-x // case["page"]) for x in lens) * 4
        return {"bytes": 2 * n * h * _row_bytes("e2m1", d) + 4 * b * hq * d
                + 4 * b * hq + table + 4 * b
                + (8 * n * h if case["weights"] else 0),
                "flops": 4 * n * hq * d}
    hq = case["q_heads"]
    moved = 2 * hq * 2 * d + 2 * h * (2 * d + _row_bytes(case["cache"], d))
    if case["cache"] == "e2m1":
        # the values are read back out of the whole 4-bit cache
        slots = b * max(-(-max(x + y for x, y in zip(lens, _held(case)))
                          // case["page"]), 1) * case["page"]
        moved_out = 2 * slots * h * (_row_bytes("e2m1", d) + 2 * d)
    else:
        moved_out = 0
    return {"bytes": n * moved + 16 * b + moved_out,
            "flops": n * (hq + h) * 8 * d}


# ------------------------------------------------- 64 bits, written apart
CODES = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
CODES = np.concatenate([CODES, -CODES])


def _read4(codes, blocks):
    """Values of 4-bit rows on the host: codes [..., D / 2], [..., D / 32]."""
    x = np.stack([CODES[codes & 15], CODES[codes >> 4]], -1)
    x = x.reshape(codes.shape[:-1] + (-1, 32))
    x = x * np.exp2(blocks.astype(np.float64) - 127.0)[..., None]
    return x.reshape(codes.shape[:-1] + (-1,))


def _write4(x):
    """The values that rows become: the nearest representable ones, found in
    a list of all that a block's scale allows."""
    blocks = x.reshape(x.shape[:-1] + (-1, 32))
    top = np.abs(blocks).max(-1, keepdims=True)
    s = np.exp2(np.ceil(np.log2(np.maximum(top, 1e-300) / 7.0)))
    s = np.where(top < 3.5 * s, s / 2, np.where(top >= 7 * s, 2 * s, s))
    y = np.abs(blocks) / s
    grid = CODES[:8]
    i = np.searchsorted((grid[1:] + grid[:-1]) / 2, y, side="left")
    middle = np.append((grid[1:] + grid[:-1]) / 2, np.inf)
    # halfway: to the code that is even
    i = np.where((y == middle[i]) & (i % 2 == 1), i + 1, i)
    return (np.copysign(grid[i], blocks) * s).reshape(x.shape)


def _exact_extend(s):
    c = s["case"]
    host = {n: s[n].cpu().numpy() for n in ("starts", "lens", "seen",
                                            "table")}
    q, k, v = (t.cpu().double().numpy() for t in _heads(s))
    for name in ("q", "k"):
        g = s[name + "_norm"]
        if g is not None:
            g = g.cpu().double().numpy()
            for x in (q,) if name == "q" else (k,):
                x /= np.sqrt((x ** 2).sum(-1, keepdims=True) / c["dim"] + EPS)
                x *= g
    if c["rot"]:
        f = s["freqs"].cpu().double().numpy()
        for b in range(c["batch"]):
            lo, hi = host["starts"][b], host["starts"][b + 1]
            turn = np.exp(1j * (host["seen"][b] + np.arange(hi - lo))[:, None]
                          * f)[:, None]
            for x in (q, k):
                z = x[lo:hi, :, :c["rot"]]
                if c["interleaved"]:
                    z = (z[..., 0::2] + 1j * z[..., 1::2]) * turn
                    x[lo:hi, :, 0:c["rot"]:2] = z.real
                    x[lo:hi, :, 1:c["rot"]:2] = z.imag
                else:
                    half = c["rot"] // 2
                    z = (z[..., :half] + 1j * z[..., half:]) * turn
                    x[lo:hi, :, :half] = z.real
                    x[lo:hi, :, half:c["rot"]] = z.imag
    r = {"q": q, "lens": host["lens"] + np.diff(host["starts"])}
    for name, x in (("k", k), ("v", v)):
        if c["cache"] == "e2m1":
            all_rows = _read4(s[name].view(torch.uint8).cpu().numpy(),
                              s[name + "_blocks"].view(torch.uint8).cpu()
                              .numpy())
            x = _write4(x)
        else:
            all_rows = s[name].cpu().double().numpy()
            if c["cache"] == "e4m3":
                x = x / s[name + "_scale"].cpu().double().numpy()[:, None]
        for b in range(c["batch"]):
            lo, hi = host["starts"][b], host["starts"][b + 1]
            t = host["lens"][b] + np.arange(hi - lo)
            all_rows[host["table"][b][t // c["page"]], :,
                     t % c["page"]] = x[lo:hi]
        r[name] = all_rows
    return r


def _slot_rows(s, name, i, n):
    """Rows [n, H, D] of one sequence, float64, slot by slot."""
    c = s["case"]
    t = torch.arange(n, device="cuda")
    at = s["table"][i].long()[t // c["page"]], t % c["page"]
    codes = s[name].view(torch.uint8)[at[0], :, at[1]].long()
    blocks = s[name + "_blocks"].view(torch.uint8)[at[0], :, at[1]].double()
    grid = torch.from_numpy(CODES).cuda()
    x = torch.stack([grid[codes % 16], grid[codes // 16]], 3)
    x = x.reshape(n, c["heads"], -1, 32) * 2.0 ** (blocks - 127)[..., None]
    return x.reshape(n, c["heads"], c["dim"])


def _exact_attend(s):
    outs, lses = [], []
    w = s["weights"].double() if "weights" in s else None
    h = s["case"]["heads"]
    b, hq, d = s["q"].shape
    for i, n in enumerate(s["lens"].tolist()):
        o = torch.zeros(hq, d, dtype=torch.float64, device="cuda")
        z = torch.full((hq,), -torch.inf, dtype=torch.float64, device="cuda")
        if n:
            k, v = _slot_rows(s, "k", i, n), _slot_rows(s, "v", i, n)
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


def _exact_sample(s):
    rows = s["case"]["rows"]
    logits = s["logits"].float().cpu().numpy()
    u = s["u"].cpu().numpy()

    def setting(name, i):
        x = s[name]
        return float(x[i]) if torch.is_tensor(x) else float(np.float32(x))

    cpu = {n: s[n].cpu() if torch.is_tensor(s[n]) else s[n]
           for n in ("temperature", "top_k", "top_p", "min_p")}
    s = dict(s, **cpu)
    tokens, logprobs = [], []
    for i in range(rows):
        x = logits[i].astype(np.float64)
        t = setting("temperature", i)
        if t <= 0:
            tokens.append(int(x.argmax()))
            logprobs.append(0.0)
            continue
        order = np.argsort(-x, kind="stable")
        k = int(setting("top_k", i))
        if 0 < k < len(order):
            order = order[:k]
        w = np.exp((x[order] - x[order[0]]) / t)
        p = setting("top_p", i)
        if p < 1:
            need = np.searchsorted(np.cumsum(w), p * math.fsum(w)) + 1
            order, w = order[:need], w[:need]
        fine = w >= setting("min_p", i)
        order, w = order[fine], w[fine]
        by_index = np.argsort(order)
        order, w = order[by_index], w[by_index]
        c = np.cumsum(w)
        j = int(np.searchsorted(c, float(u[i]) * c[-1], side="right"))
        tokens.append(int(order[j]))
        logprobs.append(math.log(w[j] / c[-1]))
    return {"tokens": np.array(tokens), "logprobs": np.array(logprobs)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"extend": _exact_extend, "attend": _exact_attend,
            "sample": _exact_sample}[case["op"]](s)
