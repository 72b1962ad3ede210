"""The paged-cache operators on the GPU against the float64 oracle.

Every row that no sequence uses is filled with NaN (0x7f.. in 8 bits), so
that a read beyond a length or through a bad table entry shows, and whole
arrays are compared afterwards, so that a stray write shows.

Bounds of cache_attend, with u = 2^-24 and x the scores: a score's error is
dx <= (dim + 4) u max sum |q k| scale, plus 4 u max |x| for the base-2
argument; a probability's is 2 dx + (n + 8) u relative (sums of n terms, the
exponential, the division); the products with V add at most (n + 8) u and,
where a probability enters as two numbers of the cache's 16-bit type,
2^-16 (bfloat16: 8 bits each) relative.  out is rounded once to q's type:
eps / 2 of it, and half its smallest step.
"""
import numpy as np
import pytest
import torch

import oracle.cache as oc
import top_selection_two_amd as ltk

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16,
         "e4m3": torch.float8_e4m3fn}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}


def _table(rng, lens, page, width, spare=3):
    """Pages of the sequences in any order; entries past a length are
    garbage that names no page."""
    need = [-(-max(n, 0) // page) for n in lens]
    ids = rng.permutation(sum(need) + spare).astype(np.int32)
    t = rng.choice(np.array([-1, -7, 2 ** 30, 2 ** 31 - 1], np.int32),
                   (len(lens), width))
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, sum(need) + spare


def _rows(rng, lens, heads, dim, page, table, pages, dtype, slots_first):
    """A cache tensor on the GPU, unused slots NaN, and its float64 values."""
    x = torch.full((pages, heads, page, dim), float("nan"))
    for b, n in enumerate(lens):
        for p in range(-(-max(n, 0) // page)):
            m = min(page, n - p * page)
            x[int(table[b, p]), :, :m] = torch.from_numpy(
                rng.standard_normal((heads, m, dim)).astype(np.float32))
    x = x.to(TYPES[dtype])
    d = x.transpose(1, 2).contiguous().cuda().transpose(1, 2) \
        if slots_first else x.cuda()
    return d, x.double().numpy()


def _case(seed, lens, heads, dim, page, dtype, slots_first=False, extra=1):
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-max(n, 0) // page) for n in lens)) + extra
    table, pages = _table(rng, lens, page, width)
    k, k64 = _rows(rng, lens, heads, dim, page, table, pages, dtype,
                   slots_first)
    v, v64 = _rows(rng, lens, heads, dim, page, table, pages, dtype,
                   slots_first)
    dev = {"k": k, "v": v, "table": torch.from_numpy(table).cuda(),
           "lens": torch.tensor(lens, dtype=torch.int32).cuda()}
    ref = {"k": k64, "v": v64, "table": table,
           "lens": np.asarray(lens, np.int64)}
    return rng, dev, ref


def _check_attend(got, want, n, dim, qtype, ctype, w0=None, w1=None):
    out, lse = (x.double().cpu().numpy() for x in got)
    o, z, added, spread, size = want
    dx = (dim + 4) * U * size + 4 * U * np.abs(np.where(np.isinf(z), 0, z)) \
        + 8 * U * size
    dp = 2 * dx + (n + 8) * U
    pair = 2.0 ** -16 if "bf16" in (qtype, ctype) or ctype == "e4m3" else \
        2.0 ** -20
    eps = torch.finfo(TYPES[qtype]).eps / 2
    tol = eps * np.abs(o) + TINY[qtype] + \
        (1 + eps) * (dp[:, :, None] + (n + 8) * U + pair) * spread
    bad = np.abs(out - o) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], o[bad][:5],
                           tol[bad][:5])
    empty = np.isinf(z)
    assert np.array_equal(lse == -np.inf, empty)
    ok = ~empty
    ztol = dx + (n + 8) * U + 4 * U * np.abs(np.where(empty, 0, z))
    assert (np.abs(lse[ok] - z[ok]) <= ztol[ok]).all()
    if w0 is None:
        return
    w0 = w0.astype(np.float64)
    group = out.shape[1] // added.shape[1]
    d = dp.reshape(dp.shape[0], -1, group).max(2)[:, :, None]
    cap = added.shape[2]
    want_w = w0.copy()
    want_w[:, :, :cap] += added
    wtol = (d + (group + 4) * U) * added + 2 * U * np.abs(want_w[:, :, :cap])
    assert (np.abs(w1 - want_w)[:, :, :cap] <= wtol).all()
    touched = np.zeros(w0.shape, bool)
    touched[:, :, :cap] = added > 0
    assert np.array_equal(w1[~touched], w0[~touched])


def _attend(dev, q, ref, qtype, ctype, weights=True, slots=None, scale=None,
            k_scale=None, v_scale=None, rng=None):
    b, hq, dim = q.shape
    heads, page = ref["k"].shape[1], ref["k"].shape[2]
    cap = dev["table"].shape[1] * page if slots is None else slots
    w0 = rng.random((b, heads, cap)).astype(np.float32) if weights else None
    w = torch.from_numpy(w0.copy()).cuda() if weights else None
    ks = None if k_scale is None else torch.from_numpy(k_scale).cuda()
    vs = None if v_scale is None else torch.from_numpy(v_scale).cuda()
    got = ltk.cache_attend(q, dev["k"], dev["v"], dev["table"], dev["lens"],
                           scale=scale, weights=w, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    want = oc.attend(q.double().cpu().numpy(), ref,
                     dim ** -0.5 if scale is None else scale, k_scale,
                     v_scale, slots)
    _check_attend(got, want, max(int(max(ref["lens"])), 1), dim, qtype,
                  ctype, w0, None if w is None else w.cpu().numpy())
    return got


def _q(rng, b, hq, dim, qtype, gain=1.5):
    q = torch.from_numpy(rng.standard_normal((b, hq, dim)).astype(np.float32))
    return (q * gain).to(TYPES[qtype]).cuda()


EDGE = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256,
        257, 511, 512, 513, 700]


@pytest.mark.parametrize("qtype,ctype", [("bf16", "bf16"), ("f16", "f16"),
                                         ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_lengths(qtype, ctype, dim):
    rng, dev, ref = _case(dim, EDGE, 2, dim, 16, ctype)
    print("attend lengths", qtype, ctype, dim, flush=True)
    ks = vs = None
    if ctype == "e4m3":
        ks = rng.random(2).astype(np.float32) + 0.5
        vs = rng.random(2).astype(np.float32) + 0.5
    _attend(dev, _q(rng, len(EDGE), 8, dim, qtype), ref, qtype, ctype,
            rng=rng, k_scale=ks, v_scale=vs)


@pytest.mark.parametrize("dim", [8, 16, 40, 80, 96, 120, 136, 192, 200, 248])
@pytest.mark.parametrize("ctype", ["bf16", "e4m3"])
def test_attend_odd_rows(dim, ctype):
    if ctype == "e4m3" and dim % 16:
        dim += 8
        if dim > 256 or dim % 16:
            pytest.skip("no whole 16-byte units")
    rng, dev, ref = _case(dim, [300, 0, 77], 3, dim, 20, ctype,
                          slots_first=True)
    print("attend rows", dim, ctype, flush=True)
    _attend(dev, _q(rng, 3, 6, dim, "bf16"), ref, "bf16", ctype, rng=rng)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 15, 16, 17, 20, 33])
@pytest.mark.parametrize("weights", [False, True])
def test_attend_groups(group, weights):
    rng, dev, ref = _case(group, [513, 40], 2, 128, 32, "bf16")
    print("attend group", group, weights, flush=True)
    _attend(dev, _q(rng, 2, 2 * group, 128, "bf16"), ref, "bf16", "bf16",
            weights, rng=rng)


@pytest.mark.parametrize("page", [1, 3, 8, 24, 100, 128, 1000])
def test_attend_pages(page):
    rng, dev, ref = _case(page, [777, 5, 100], 2, 64, page, "f16",
                          slots_first=page % 2 == 0)
    print("attend page", page, flush=True)
    _attend(dev, _q(rng, 3, 4, 64, "f16"), ref, "f16", "f16", rng=rng)


@pytest.mark.parametrize("n,batch,heads,weights", [
    (9000, 1, 1, True), (9000, 1, 2, False), (5003, 3, 2, True),
    (40000, 1, 1, True)])
def test_attend_long(n, batch, heads, weights):
    lens = [n - 1234 * i for i in range(batch)]
    rng, dev, ref = _case(n, lens, heads, 64, 64, "bf16")
    print("attend long", n, batch, heads, flush=True)
    _attend(dev, _q(rng, batch, 4 * heads, 64, "bf16"), ref, "bf16", "bf16",
            weights, rng=rng)


# Enough slots for every workgroup to take several shares of rows, whole rows
# and split ones, and more scores than one holds: by queries a head, and with
# a table that allows for rows too long to be finished in one launch.
@pytest.mark.parametrize("group,heads,batch,lo,hi,extra", [
    (1, 4, 40, 300, 3000, 1), (4, 4, 40, 300, 3000, 1),
    (4, 4, 40, 300, 3000, 1400), (16, 2, 40, 300, 3000, 1),
    (16, 2, 40, 300, 3000, 1400), (20, 2, 24, 300, 3000, 1),
    (12, 1, 3, 20000, 70000, 1)])
def test_attend_full_device(group, heads, batch, lo, hi, extra):
    lens = [int(x) for x in
            np.random.default_rng(group).integers(lo, hi, size=batch)]
    lens[1], lens[-1] = 0, hi
    rng, dev, ref = _case(group, lens, heads, 16, 16, "bf16", extra=extra)
    print("attend full device", group, heads, batch, extra, flush=True)
    _attend(dev, _q(rng, batch, group * heads, 16, "bf16"), ref, "bf16",
            "bf16", rng=rng)


# The same with slots outside heads, where a workgroup takes four heads.
@pytest.mark.parametrize("group,heads,dim,page,dtype,extra", [
    (1, 4, 16, 16, "bf16", 1), (4, 4, 16, 20, "f16", 1),
    (3, 8, 80, 16, "bf16", 1), (20, 4, 16, 16, "bf16", 1),
    (16, 4, 16, 16, "e4m3", 600), (2, 4, 256, 16, "bf16", 1),
    (2, 4, 136, 3, "bf16", 1), (6, 12, 16, 16, "bf16", 1)])
def test_attend_full_device_slots_first(group, heads, dim, page, dtype,
                                        extra):
    lens = [int(x) for x in
            np.random.default_rng(group).integers(100, 3000, size=40)]
    lens[1], lens[-1] = 0, 3000
    rng, dev, ref = _case(group, lens, heads, dim, page, dtype, True, extra)
    q = "f16" if dtype == "f16" else "bf16"
    print("attend slots first", group, heads, dim, page, dtype, flush=True)
    _attend(dev, _q(rng, 40, group * heads, dim, q), ref, q, dtype, rng=rng)
    _attend(dev, _q(rng, 40, group * heads, dim, q), ref, q, dtype,
            weights=False, rng=rng)


def test_attend_many_sequences():
    lens = [int(x) for x in
            np.random.default_rng(5).integers(0, 90, size=700)]
    rng, dev, ref = _case(6, lens, 1, 16, 8, "bf16")
    print("attend 700 sequences", flush=True)
    _attend(dev, _q(rng, 700, 2, 16, "bf16"), ref, "bf16", "bf16", rng=rng)


def test_attend_without_any_slot():
    rng, dev, ref = _case(1, [0, 0, 0], 2, 64, 16, "bf16")
    got = _attend(dev, _q(rng, 3, 4, 64, "bf16"), ref, "bf16", "bf16",
                  rng=rng)
    assert not got[0].any() and (got[1] == -float("inf")).all()


def test_attend_lengths_outside_the_table():
    rng, dev, ref = _case(2, [96, 64], 1, 64, 16, "bf16", extra=0)
    dev["lens"] = torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32).cuda()
    ref["lens"] = np.array([2 ** 31 - 1, -5])
    _attend(dev, _q(rng, 2, 2, 64, "bf16"), {**ref, "lens": np.array([96, -5])},
            "bf16", "bf16", rng=rng)
    # a ledger shorter than the table bounds the lengths too
    _attend(dev, _q(rng, 2, 2, 64, "bf16"), {**ref, "lens": np.array([96, -5])},
            "bf16", "bf16", rng=rng, slots=50)


def test_attend_pages_that_are_not_there():
    rng, dev, ref = _case(3, [400, 90, 33, 64], 2, 64, 16, "bf16")
    bad = ref["table"].copy()
    pages = ref["k"].shape[0]
    bad[0, 3], bad[0, 7], bad[0, 24] = -1, pages, 2 ** 31 - 1
    bad[1, 0] = -2 ** 31
    bad[2, :] = -1        # nothing left of the third sequence
    bad[3, :] = pages
    ref["table"] = bad
    dev["table"] = torch.from_numpy(bad).cuda()
    print("attend bad pages", flush=True)
    got = _attend(dev, _q(rng, 4, 4, 64, "bf16"), ref, "bf16", "bf16",
                  rng=rng)
    assert not got[0][2:].any() and (got[1][2:] == -float("inf")).all()


def test_attend_peaked_and_flat_scores():
    # one slot far above the others, growing maxima, and equal scores
    for gain in (0.0, 30.0, 200.0):
        rng, dev, ref = _case(11, [600, 31], 2, 64, 16, "bf16")
        _attend(dev, _q(rng, 2, 8, 64, "bf16", gain), ref, "bf16", "bf16",
                rng=rng)
    rng, dev, ref = _case(12, [500], 1, 64, 16, "bf16")
    ramp = np.linspace(-60, 60, 500)  # every tile raises the maximum
    for t in range(500):
        p, z = int(ref["table"][0, t // 16]), t % 16
        ref["k"][p, 0, z] = 0
        ref["k"][p, 0, z, 0] = ramp[t]
    k = torch.from_numpy(ref["k"]).to(torch.bfloat16)
    ref["k"], dev["k"] = k.double().numpy(), k.cuda()
    q = torch.zeros(1, 2, 64)
    q[0, 0, 0], q[0, 1, 0] = 1.0, -1.0
    _attend(dev, q.to(torch.bfloat16).cuda(), ref, "bf16", "bf16", rng=rng,
            scale=1.0)


def test_attend_infinite_and_nan_rows():
    rng, dev, ref = _case(13, [100, 100, 100], 1, 64, 16, "bf16")
    k = dev["k"].cpu()
    t = ref["table"]
    k[int(t[0, 2]), 0, 5, 3] = float("nan")
    k[int(t[1, 2]), 0, 5] = 0
    k[int(t[1, 2]), 0, 5, 3] = float("inf")
    dev["k"] = k.cuda()
    q = torch.ones(3, 1, 64).to(torch.bfloat16).cuda()
    out, lse = ltk.cache_attend(q, dev["k"], dev["v"], dev["table"],
                                dev["lens"])
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1].isnan().all()
    assert out[2].isfinite().all() and lse[2].isfinite().all()
    # a score of -infinity has weight 0 and takes nothing with it
    k[int(t[1, 2]), 0, 5, 3] = -float("inf")
    dev["k"] = k.cuda()
    w = torch.zeros(3, 1, 112).cuda()
    out, lse = ltk.cache_attend(q, dev["k"], dev["v"], dev["table"],
                                dev["lens"], weights=w)
    assert out[1].isfinite().all() and lse[1].isfinite().all()
    assert w[1, 0, 37] == 0 and abs(float(w[1].sum()) - 1) < 1e-5
    # every score -infinity: as no slot
    kk = torch.zeros_like(k)
    kk[:, :, :, 3] = -float("inf")
    w.zero_()
    out, lse = ltk.cache_attend(q, kk.cuda(), dev["v"], dev["table"],
                                dev["lens"], weights=w)
    assert not out.any() and (lse == -float("inf")).all() and not w.any()


def test_attend_strided_inputs():
    rng, dev, ref = _case(14, [260, 31], 2, 64, 16, "bf16")
    wide = torch.full((2, 3, 4, 96), float("nan"), dtype=torch.bfloat16)
    q = wide.cuda()[:, 1, :, 16:80]
    q.copy_(_q(rng, 2, 4, 64, "bf16"))
    # K and V interleaved in one array with padding
    kv = torch.full((dev["k"].shape[0], 2, 2, 16, 72), float("nan"),
                    dtype=torch.bfloat16).cuda()
    kv[:, 0, :, :, :64] = dev["k"]
    kv[:, 1, :, :, :64] = dev["v"]
    table = torch.full((2, 40), -1, dtype=torch.int32).cuda()
    w = dev["table"].shape[1]
    table[:, :w] = dev["table"]
    d = {**dev, "k": kv[:, 0, :, :, :64], "v": kv[:, 1, :, :, :64],
         "table": table[:, :w]}
    a = _attend(d, q, ref, "bf16", "bf16", rng=rng)
    b = _attend(dev, q.contiguous(), ref, "bf16", "bf16", rng=rng)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # weights: heads outside sequences, rows padded
    base = torch.zeros(2, 2, 500).cuda()
    wt = base.transpose(0, 1)[:, :, :w * 16]
    ltk.cache_attend(q, d["k"], d["v"], d["table"], d["lens"], weights=wt)
    plain = torch.zeros(2, 2, w * 16).cuda()
    ltk.cache_attend(q, dev["k"], dev["v"], dev["table"], dev["lens"],
                     weights=plain)
    assert torch.equal(wt, plain) and not base[:, :, w * 16:].any()


def test_attend_is_reproducible_on_any_stream():
    rng, dev, ref = _case(15, [3000, 100, 0, 900], 2, 128, 16, "bf16")
    q = _q(rng, 4, 8, 128, "bf16")

    def call():
        w = torch.zeros(4, 2, dev["table"].shape[1] * 16, device="cuda")
        o, z = ltk.cache_attend(q, dev["k"], dev["v"], dev["table"],
                                dev["lens"], weights=w)
        return o, z, w

    want = call()
    for i in range(4):
        ltk.cache_debug_scramble(i + 1)
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_step_replays():
    """attend and append in one graph, replayed between eager work."""
    rng, dev, ref = _case(16, [64, 40], 2, 64, 16, "bf16", extra=2)
    n = dev["table"].shape[1] * 16
    table = torch.arange(2 * dev["table"].shape[1], dtype=torch.int32).cuda()
    table = table.view(2, -1)
    pages = table.numel()
    g = torch.Generator().manual_seed(3)

    def state():
        g.manual_seed(3)
        k = torch.randn(pages, 2, 16, 64, generator=g).to(torch.bfloat16)
        v = torch.randn(pages, 2, 16, 64, generator=g).to(torch.bfloat16)
        q = torch.randn(2, 8, 64, generator=g).to(torch.bfloat16)
        pos = torch.arange(n, dtype=torch.int32).expand(2, 2, n)
        return {"k": k.cuda(), "v": v.cuda(), "q": q.cuda(),
                "w": torch.rand(2, 2, n, generator=g).cuda(),
                "pos": pos.contiguous().cuda(), "lens": dev["lens"].clone(),
                "seen": dev["lens"].clone()}

    def step(s):
        new = (s["q"][:, ::4] * 0.5).contiguous()
        lens, slots = ltk.cache_append(new, new, s["k"], s["v"], table,
                                       s["lens"], 66, s["seen"], s["w"],
                                       s["pos"], 2, 4)
        s["lens"].copy_(lens)
        o, z = ltk.cache_attend(s["q"], s["k"], s["v"], table, s["lens"],
                                weights=s["w"])
        s["q"].copy_(o.to(torch.bfloat16))
        s["seen"].add_(1)
        return o, z, slots

    eager = state()
    want = []
    for _ in range(6):
        want.append([x.clone() for x in step(eager)] +
                    [eager["w"].clone(), eager["lens"].clone()])
    s = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = state()
        step(warm)          # the stream's workspace
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(s)
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        for a, b in zip(list(out) + [s["w"], s["lens"]], want[i]):
            assert torch.equal(a, b), i
        ltk.cache_attend(warm["q"], warm["k"], warm["v"], table,
                         warm["lens"], weights=warm["w"])
        torch.cuda.synchronize()
    assert torch.equal(s["k"], eager["k"]) and torch.equal(s["v"], eager["v"])


def test_capture_refuses_to_grow_the_workspace():
    rng, dev, ref = _case(17, [100], 1, 64, 16, "bf16")
    q = _q(rng, 1, 2, 64, "bf16")
    side = torch.cuda.Stream()
    w = torch.zeros(1, 1, dev["table"].shape[1] * 16, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    ltk.release()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            x = q * 2
            with pytest.raises(ltk.LibtopkError) as e:
                ltk.cache_attend(q, dev["k"], dev["v"], dev["table"],
                                 dev["lens"], weights=w)
    assert e.value.status == ltk.ERR_NOMEM
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, q * 2) and not w.any()


def test_failing_allocation(monkeypatch):
    rng, dev, ref = _case(18, [100], 1, 64, 16, "bf16")
    q = _q(rng, 1, 2, 64, "bf16")
    w = torch.zeros(1, 1, dev["table"].shape[1] * 16, device="cuda")
    torch.cuda.synchronize()
    ltk.release()
    monkeypatch.setenv("LIBTOPK_TEST_FAIL_ALLOC", "1")
    with pytest.raises(ltk.LibtopkError) as e:
        ltk.cache_attend(q, dev["k"], dev["v"], dev["table"], dev["lens"],
                         weights=w)
    assert e.value.status == ltk.ERR_NOMEM
    monkeypatch.delenv("LIBTOPK_TEST_FAIL_ALLOC")
    _attend(dev, q, ref, "bf16", "bf16", rng=rng)


# ------------------------------------------------------- append and evict
def _ledger(rng, b, heads, n, kind):
    if kind == "equal":
        w = np.full((b, heads, n), 0.5, np.float32)
    elif kind == "few":
        w = rng.integers(0, 3, (b, heads, n)).astype(np.float32)
    elif kind == "special":
        w = rng.choice(np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0,
                                 1e-42, -2.0], np.float32), (b, heads, n))
    else:
        w = np.exp(1.5 * rng.standard_normal((b, heads, n))).astype(
            np.float32)
    pos = np.stack([[rng.permutation(n) for _ in range(heads)]
                    for _ in range(b)]).astype(np.int32)
    return w, pos


def _same(a, b):
    """Equal bits (NaN rows among them)."""
    a, b = a.contiguous(), b.contiguous()
    if a.element_size() == 1:
        return torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    kind = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.view(kind), b.view(kind))


def _as(ref, like):
    """The oracle's float64 rows in the cache's type."""
    return torch.from_numpy(ref).to(like.dtype)


def _nan_equal(x, y):
    x, y = x.float().cpu().numpy(), y.float().cpu().numpy()
    return np.array_equal(x, y, equal_nan=True)


def _check_append(lens, heads, dim, page, limit, sinks, recent, kind="plain",
                  dtype="bf16", slots_first=False, slots=None, extra=1,
                  bad=(), seed=0):
    rng, dev, ref = _case(seed, lens, heads, dim, page, dtype, slots_first,
                          extra)
    b = len(lens)
    for i, j, x in bad:
        ref["table"][i, j] = x
    dev["table"] = torch.from_numpy(ref["table"]).cuda()
    n = dev["table"].shape[1] * page if slots is None else slots
    w, pos = _ledger(rng, b, heads, n, kind)
    seen = np.full(b, n + 7, np.int32)
    kn = torch.from_numpy(rng.standard_normal((b, heads, dim)).astype(
        np.float32)).to(TYPES[dtype])
    vn = torch.from_numpy(rng.standard_normal((b, heads, dim)).astype(
        np.float32)).to(TYPES[dtype])
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    got = ltk.cache_append(kn.cuda(), vn.cuda(), dev["k"], dev["v"],
                           dev["table"], dev["lens"], limit,
                           torch.from_numpy(seen).cuda(), dw, dp, sinks,
                           recent)
    torch.cuda.synchronize()
    k, v, w2, p2, s2, l2 = oc.append(kn.double().numpy(), vn.double().numpy(),
                                     ref, limit, seen, w, pos, sinks, recent)
    assert np.array_equal(got[0].cpu().numpy(), l2)
    assert np.array_equal(got[1].cpu().numpy(), s2)
    assert np.array_equal(dw.cpu().numpy().view(np.int32), w2.view(np.int32))
    assert np.array_equal(dp.cpu().numpy(), p2)
    assert _nan_equal(dev["k"], _as(k, kn)) and _nan_equal(dev["v"],
                                                           _as(v, kn))


@pytest.mark.parametrize("kind", ["plain", "equal", "few", "special"])
@pytest.mark.parametrize("lens,limit", [
    ([0, 1, 63, 64, 65], 64), ([200, 513, 512, 1025, 3], 512), ([9], 1),
    ([5000, 4097], 4096)])
def test_append(kind, lens, limit):
    print("append", kind, lens, limit, flush=True)
    _check_append(lens, 2, 64, 16, limit, 4, 20, kind)


@pytest.mark.parametrize("dim,dtype,page,slots_first", [
    (8, "bf16", 1, False), (80, "f16", 24, True), (256, "bf16", 100, True),
    (128, "e4m3", 16, False), (16, "e4m3", 3, True), (256, "e4m3", 64, True)])
def test_append_rows(dim, dtype, page, slots_first):
    print("append rows", dim, dtype, page, flush=True)
    _check_append([40, 7, 33], 3, dim, page, 33, 0, 0, "plain", dtype,
                  slots_first)


def test_append_protection():
    # everything protected: the latest slot goes; sinks alone; recent alone
    for sinks, recent in ((10 ** 6, 0), (0, 2 ** 31 - 1), (3, 0), (0, 60)):
        _check_append([50, 64], 2, 16, 16, 50, sinks, recent, "few")


def test_append_beyond_the_table_and_bad_pages():
    _check_append([64, 48], 2, 16, 16, 100, 0, 0, extra=0)   # 64 is full
    _check_append([64, 48], 2, 16, 16, 100, 0, 0, slots=50)  # the ledger is
    _check_append([64, 48], 2, 16, 16, 40, 0, 0, slots=41)
    _check_append([64, 48, 20], 2, 16, 16, 30, 0, 0, "equal",
                  bad=[(0, 3, -1), (1, 2, 2 ** 31 - 1), (2, 1, 10 ** 6)])
    _check_append([-3, 10], 1, 16, 16, 8, 0, 0)


def _check_evict(lens, heads, dim, page, keep, sinks, recent, kind="plain",
                 dtype="bf16", slots_first=False, slots=None, bad=(), seed=0,
                 extra=1, seen=None):
    rng, dev, ref = _case(seed, lens, heads, dim, page, dtype, slots_first,
                          extra)
    b = len(lens)
    for i, j, x in bad:
        ref["table"][i, j] = x
    dev["table"] = torch.from_numpy(ref["table"]).cuda()
    n = dev["table"].shape[1] * page if slots is None else slots
    w, pos = _ledger(rng, b, heads, n, kind)
    seen = np.full(b, n if seen is None else seen, np.int32)
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    like = dev["k"].dtype
    got = ltk.cache_evict(dev["k"], dev["v"], dev["table"], dev["lens"],
                          torch.from_numpy(seen).cuda(), dw, dp, keep, sinks,
                          recent)
    torch.cuda.synchronize()
    k, v, w2, p2, l2 = oc.evict(ref, seen, w, pos, keep, sinks, recent)
    assert np.array_equal(got[2].cpu().numpy(), l2)
    assert np.array_equal(got[0].cpu().numpy().view(np.int32),
                          w2.view(np.int32))
    assert np.array_equal(got[1].cpu().numpy(), p2)
    zero = torch.zeros(1, dtype=like)
    assert _nan_equal(dev["k"], _as(k, zero)) and _nan_equal(dev["v"],
                                                             _as(v, zero))
    assert np.array_equal(dw.cpu().numpy().view(np.int32), w.view(np.int32))
    assert np.array_equal(dp.cpu().numpy(), pos)


@pytest.mark.parametrize("kind", ["plain", "equal", "few", "special"])
@pytest.mark.parametrize("lens,keep", [
    ([0, 1, 63, 64, 65, 200], 64), ([700, 513, 512, 90], 100), ([9], 1),
    ([1200, 1030], 1025), ([2000], 3), ([33, 20], 500)])
def test_evict(kind, lens, keep):
    print("evict", kind, lens, keep, flush=True)
    _check_evict(lens, 2, 16, 16, keep, 4, 20, kind)


@pytest.mark.parametrize("kind", ["plain", "few", "special"])
@pytest.mark.parametrize("lens,keep", [
    ([9001, 4096, 8192, 8193], 2000), ([20000], 15000), ([70001], 4000),
    ([40000, 35000], 1)])
def test_evict_long(kind, lens, keep):
    print("evict long", kind, lens, keep, flush=True)
    _check_evict(lens, 1, 8, 256, keep, 4, 333, kind)


@pytest.mark.parametrize("dim,dtype,page,slots_first", [
    (8, "bf16", 1, False), (80, "f16", 24, True), (256, "bf16", 100, True),
    (128, "e4m3", 16, False), (16, "e4m3", 3, True), (256, "e4m3", 64, True)])
def test_evict_rows(dim, dtype, page, slots_first):
    print("evict rows", dim, dtype, page, flush=True)
    _check_evict([140, 7, 133], 3, dim, page, 33, 0, 0, "plain", dtype,
                 slots_first)


def test_evict_protection():
    for sinks, recent in ((10 ** 6, 0), (0, 2 ** 31 - 1), (40, 0), (0, 60),
                          (20, 50)):
        _check_evict([150, 64], 2, 16, 16, 50, sinks, recent, "few")
    _check_evict([150, 64], 2, 16, 16, 50, 0, 2 ** 31 - 1, "few",
                 seen=-2 ** 31)


def test_evict_short_ledger_and_bad_pages():
    _check_evict([64, 48], 2, 16, 16, 20, 0, 0, slots=50)
    _check_evict([64, 48], 2, 16, 16, 50, 0, 0, slots=50)
    _check_evict([64, 48, -9], 2, 16, 16, 20, 0, 0, "equal",
                 bad=[(0, 3, -1), (0, 0, 10 ** 6), (1, 2, 2 ** 31 - 1)])
    _check_evict([300, 148], 2, 16, 16, 20, 0, 0,
                 bad=[(0, 3, -1), (0, 10, 10 ** 6), (1, 1, 2 ** 31 - 1)])


def test_evict_into_given_arrays_and_repeat():
    rng, dev, ref = _case(21, [500, 90], 2, 64, 16, "bf16")
    n = dev["table"].shape[1] * 16
    w, pos = _ledger(rng, 2, 2, n, "few")
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    seen = dev["lens"].clone()
    ow = torch.full((2, 2, 128), 7.0).cuda()
    op = torch.full((2, 2, 128), 7, dtype=torch.int32).cuda()
    r = []
    for i in range(3):
        k, v = dev["k"].clone(), dev["v"].clone()
        ltk.cache_debug_scramble(i)
        a = ltk.cache_evict(k, v, dev["table"], dev["lens"], seen, dw, dp,
                            100, out=(ow[:, :, 20:120], op[:, :, 28:]))
        r.append((a[0].clone(), a[1].clone(), a[2], k, v))
    assert all(_same(x, y) for one in r[1:] for x, y in zip(one, r[0]))
    assert (ow[:, :, :20] == 7).all() and (ow[:, :, 120:] == 7).all()
    assert (op[:, :, :28] == 7).all()
    got = ltk.cache_evict(dev["k"], dev["v"], dev["table"], dev["lens"],
                          seen, dw, dp, 100)
    assert all(_same(x, y) for x, y in zip(got, r[0]))


def test_example_keeps_a_bounded_cache():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(
        os.path.abspath(__file__))), "examples", "bounded_cache.py")
    spec = importlib.util.spec_from_file_location("bounded_cache", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    r = mod.decode(batch=2, heads=2, group=4, dim=64, prompt=300, budget=128,
                   tokens=20)
    # the budget holds, the sinks and the recent tokens are in the cache, and
    # its positions are distinct
    assert r["lens"].tolist() == [128, 128]
    for row in r["positions"].cpu().numpy().reshape(-1, 128):
        have = set(row.tolist())
        assert len(have) == 128 and {0, 1, 2, 3} <= have
        assert set(range(320 - 16, 320)) <= have
    assert r["out"].isfinite().all()
    # what the cache's rows say: every row is its position's
    assert mod.rows_match(r)
