"""cache_extend, and attention and eviction over rows of 4 bits, on the GPU
against the float64 oracle.

Rows that are written are compared as their type holds them.  Values are
computed in 64 bits, with errors of some 2^-45 of a row's largest (sums of up
to 256 terms, angles of positions below 2^31 to 2^-22 turns at most and to
2^-49 of the angle's turns otherwise), and rounded to 16 or 8 bits through
float32: half a step of the type, and 2^-24 of the value for the first
rounding.  A 4-bit element is the number that the oracle's arithmetic gives,
unless its quotient lies within 2^-40 of a border between two.

Attention's bounds are those of test_gpu_cache.py; 4-bit rows are held exactly
by bfloat16, as are float16 queries by two of them.
"""
import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.step as st
import test_gpu_cache as base
import top_selection_two_amd as ltk

pytestmark = pytest.mark.gpu

TYPES = dict(base.TYPES)
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10}


# ------------------------------------------------------------- 4-bit caches
def _four(codes, blocks, slots_first):
    """Device tensors of a 4-bit cache from its bytes."""
    c, b = torch.from_numpy(codes), torch.from_numpy(blocks)
    if slots_first:
        c, b = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
                for x in (c, b))
    else:
        c, b = c.cuda(), b.cuda()
    return c.view(torch.float4_e2m1fn_x2), b.view(torch.float8_e8m0fnu)


def _bytes(x):
    return x.view(torch.uint8).cpu().numpy()


def _case4(seed, lens, heads, dim, page, slots_first=False, extra=1,
           low=118, high=131):
    """A 4-bit cache of random codes and scales; unused slots have the scale
    NaN."""
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-max(n, 0) // page) for n in lens)) + extra
    table, pages = base._table(rng, lens, page, width)
    dev = {"table": torch.from_numpy(table).cuda(),
           "lens": torch.tensor(lens, dtype=torch.int32).cuda()}
    ref = {"table": table, "lens": np.asarray(lens, np.int64)}
    used = np.zeros((pages, page), bool)
    for b, n in enumerate(lens):
        for p in range(-(-max(n, 0) // page)):
            used[table[b, p], :min(page, n - p * page)] = True
    for name in ("k", "v"):
        codes = rng.integers(0, 256, (pages, heads, page, dim // 2))
        codes = codes.astype(np.uint8)
        blocks = rng.integers(low, high, (pages, heads, page, dim // 32))
        blocks = np.where(used[:, None, :, None], blocks, 255)
        blocks = blocks.astype(np.uint8)
        dev[name], dev[name + "_blocks"] = _four(codes, blocks, slots_first)
        ref[name] = st.unpack(codes, blocks)
    return rng, dev, ref


def _attend(rng, dev, ref, group, dim, qtype, weights=True, slots=None,
            gain=0.05, scales=False, scale=None):
    b, heads = len(ref["lens"]), ref["k"].shape[1]
    q = base._q(rng, b, heads * group, dim, qtype, gain)
    cap = dev["table"].shape[1] * ref["k"].shape[2] if slots is None else slots
    w0 = rng.random((b, heads, cap)).astype(np.float32) if weights else None
    w = torch.from_numpy(w0.copy()).cuda() if weights else None
    ks = vs = None
    if scales:
        ks = rng.random(heads).astype(np.float32) + 0.5
        vs = rng.random(heads).astype(np.float32) + 0.5
    got = ltk.cache_attend(
        q, dev["k"], dev["v"], dev["table"], dev["lens"], scale=scale,
        weights=w, k_scale=None if ks is None else torch.from_numpy(ks).cuda(),
        v_scale=None if vs is None else torch.from_numpy(vs).cuda(),
        k_blocks=dev["k_blocks"], v_blocks=dev["v_blocks"])
    torch.cuda.synchronize()
    want = oc.attend(q.double().cpu().numpy(), ref,
                     dim ** -0.5 if scale is None else scale, ks, vs, slots)
    base._check_attend(got, want, max(int(max(ref["lens"])), 1), dim, qtype,
                       "e4m3", w0, None if w is None else w.cpu().numpy())
    return got


@pytest.mark.parametrize("qtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_attend_lengths(qtype, dim):
    print("attend 4-bit", qtype, dim, flush=True)
    rng, dev, ref = _case4(dim, base.EDGE, 2, dim, 16)
    _attend(rng, dev, ref, 4, dim, qtype, scales=dim % 64 == 0)


@pytest.mark.parametrize("page", [1, 3, 8, 24, 100, 128])
@pytest.mark.parametrize("slots_first", [False, True])
def test_attend_pages(page, slots_first):
    print("attend 4-bit page", page, slots_first, flush=True)
    rng, dev, ref = _case4(page, [777, 0, 100], 4, 64, page, slots_first)
    _attend(rng, dev, ref, 2, 64, "bf16")


@pytest.mark.parametrize("group", [1, 3, 8, 16, 17, 33])
@pytest.mark.parametrize("qtype", ["bf16", "f16"])
def test_attend_groups(group, qtype):
    print("attend 4-bit group", group, qtype, flush=True)
    rng, dev, ref = _case4(group, [513, 40], 2, 128, 32)
    _attend(rng, dev, ref, group, 128, qtype, group % 2 == 0)


@pytest.mark.parametrize("group,heads,dim,page,extra,qtype", [
    (4, 4, 32, 16, 1, "bf16"), (4, 4, 32, 16, 1400, "f16"),
    (16, 4, 64, 20, 1, "bf16"), (20, 4, 32, 16, 1, "f16"),
    (2, 4, 256, 16, 1, "bf16"), (2, 8, 192, 3, 1, "f16")])
@pytest.mark.parametrize("slots_first", [False, True])
def test_attend_full_device(group, heads, dim, page, extra, qtype,
                            slots_first):
    """Rows split over workgroups, several rows a workgroup, second launches,
    scores that LDS does not hold."""
    lens = [int(x) for x in
            np.random.default_rng(group).integers(100, 3000, size=40)]
    lens[1], lens[-1] = 0, 3000
    print("attend 4-bit full", group, heads, dim, page, flush=True)
    rng, dev, ref = _case4(group, lens, heads, dim, page, slots_first, extra)
    _attend(rng, dev, ref, group, dim, qtype)
    _attend(rng, dev, ref, group, dim, qtype, weights=False)


@pytest.mark.parametrize("n,heads,weights", [(40000, 1, True),
                                             (9001, 2, False)])
def test_attend_long(n, heads, weights):
    print("attend 4-bit long", n, flush=True)
    rng, dev, ref = _case4(n, [n], heads, 64, 64)
    _attend(rng, dev, ref, 4, 64, "bf16", weights)


def test_attend_reads_every_code_and_scale():
    """Sequences of one slot: out is the row of V.  (Numbers below 2^-126,
    which few operations on this machine keep, may come as 0.)"""
    b, dim = 255, 32
    codes = np.zeros((b, 1, 1, dim // 2), np.uint8)
    # codes 0 .. 15, twice
    codes[:] = np.tile(np.arange(8) * 34 + 16, 2)
    blocks = np.arange(b, dtype=np.uint8).reshape(b, 1, 1, 1)
    v, vb = _four(codes, blocks, False)
    k, kb = _four(codes, np.full_like(blocks, 100), False)
    q = torch.ones(b, 1, dim, dtype=torch.bfloat16).cuda()
    out, lse = ltk.cache_attend(
        q, k, v, torch.arange(b, dtype=torch.int32).view(b, 1).cuda(),
        torch.ones(b, dtype=torch.int32).cuda(), k_blocks=kb, v_blocks=vb)
    want = st.unpack(codes, blocks)[:, 0]
    # bfloat16's largest number is below 1.5 2^128 and 2^129
    over = np.abs(want) >= 2.0 ** 128
    got = out.double().cpu().numpy()
    assert (np.isinf(got) == over).all()
    tiny = np.abs(want) < 2.0 ** -126
    assert (got[~over & ~tiny] == want[~over & ~tiny]).all()
    assert ((got[tiny] == want[tiny]) | (got[tiny] == 0)).all()
    assert lse.isfinite().all()


def test_attend_nan_scales():
    """A block with the scale NaN makes its columns NaN (in V), and its row's
    score (in K); of masked slots it does nothing."""
    rng, dev, ref = _case4(7, [40, 40, 40], 1, 64, 16)
    kb, vb = _bytes(dev["k_blocks"]), _bytes(dev["v_blocks"])
    t = ref["table"]
    vb[t[0, 1], 0, 3, 1] = 255
    kb[t[1, 2], 0, 5, 0] = 255
    dev["k_blocks"] = torch.from_numpy(kb).cuda().view(torch.float8_e8m0fnu)
    dev["v_blocks"] = torch.from_numpy(vb).cuda().view(torch.float8_e8m0fnu)
    q = base._q(rng, 3, 2, 64, "bf16", 0.05)
    out, lse = ltk.cache_attend(q, dev["k"], dev["v"], dev["table"],
                                dev["lens"], k_blocks=dev["k_blocks"],
                                v_blocks=dev["v_blocks"])
    assert out[0, :, 32:].isnan().all() and out[0, :, :32].isfinite().all()
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert out[2].isfinite().all() and lse[[0, 2]].isfinite().all()


def test_attend_strided_blocks():
    """Codes and scales side by side in one array of bytes."""
    rng, dev, ref = _case4(8, [300, 31], 2, 64, 16)
    pages = dev["k"].shape[0]
    both = torch.zeros(pages, 2, 16, 48, dtype=torch.uint8).cuda()
    both[..., :32] = dev["k"].view(torch.uint8)
    both[..., 33:35] = dev["k_blocks"].view(torch.uint8)
    d = dict(dev, k=both[..., :32].view(torch.float4_e2m1fn_x2),
             k_blocks=both[..., 33:35].view(torch.float8_e8m0fnu))
    _attend(rng, d, ref, 2, 64, "bf16")


@pytest.mark.parametrize("slots,keep", [(300, 100), (20000, 3000)])
def test_evict_moves_scales(slots, keep):
    print("evict 4-bit", slots, flush=True)
    page, heads, dim = 16, 2, 96
    rng, dev, ref = _case4(slots, [slots, slots // 2, 5], heads, dim, page,
                           True)
    n = dev["table"].shape[1] * page
    w = rng.random((3, heads, n)).astype(np.float32)
    pos = np.tile(np.arange(n, dtype=np.int32), (3, heads, 1))
    seen = np.array([slots, slots // 2, 5], np.int32)
    k, v, w2, p2, lens2 = oc.evict(ref, seen, w, pos, keep, 4, 16)
    got = ltk.cache_evict(dev["k"], dev["v"], dev["table"], dev["lens"],
                          torch.from_numpy(seen).cuda(),
                          torch.from_numpy(w).cuda(),
                          torch.from_numpy(pos).cuda(), keep, 4, 16,
                          k_blocks=dev["k_blocks"], v_blocks=dev["v_blocks"])
    torch.cuda.synchronize()
    assert np.array_equal(got[0].cpu().numpy(), w2)
    assert np.array_equal(got[1].cpu().numpy(), p2)
    assert np.array_equal(got[2].cpu().numpy(), lens2)
    for name, want in (("k", k), ("v", v)):
        have = st.unpack(_bytes(dev[name]), _bytes(dev[name + "_blocks"]))
        assert np.array_equal(have, want, equal_nan=True)


# ------------------------------------------------------------------- extend
def _new(rng, counts, q_heads, heads, dim, qtype, spare=0, gain=1.0):
    """Slices of one projection's output, spare tokens at its end."""
    n = sum(counts) + spare
    x = rng.standard_normal((n, q_heads + 2 * heads, dim)) * gain
    x = torch.from_numpy(x.astype(np.float32)).to(TYPES[qtype]).cuda()
    return x[:, :q_heads], x[:, q_heads:q_heads + heads], x[:, q_heads + heads:]


def _blank(rng, lens, counts, heads, dim, page, ctype, slots_first=False,
           extra=1):
    """A cache with room for the new tokens, filled with a pattern."""
    most = [min(max(a, 0) + b, 10 ** 9) for a, b in zip(lens, counts)]
    width = max(1, max(-(-n // page) for n in most)) + extra
    table, pages = base._table(rng, most, page, width)
    dev = {"table": torch.from_numpy(table).cuda(),
           "lens": torch.tensor(lens, dtype=torch.int32).cuda()}
    ref = {"table": table, "lens": np.asarray(lens, np.int64)}
    for name in ("k", "v"):
        if ctype == "e2m1":
            codes = rng.integers(0, 256, (pages, heads, page, dim // 2))
            blocks = rng.integers(0, 256, (pages, heads, page, dim // 32))
            dev[name], dev[name + "_blocks"] = _four(
                codes.astype(np.uint8), blocks.astype(np.uint8), slots_first)
        else:
            x = rng.standard_normal((pages, heads, page, dim))
            x = torch.from_numpy(x.astype(np.float32)).to(TYPES[ctype])
            dev[name] = x.transpose(1, 2).contiguous().cuda().transpose(1, 2) \
                if slots_first else x.cuda()
        ref[name] = np.zeros((pages, heads, page, dim))
    return dev, ref


def _raw(x):
    return x.contiguous().view(torch.uint8).cpu().numpy().copy()


def _near(got, want, size, ctype):
    """Half a step of the type, 2^-23 of the value (both sides of the
    rounding to float32) and what 64 bits leave of a row's size."""
    t = torch.finfo(TYPES[ctype])
    tol = (t.eps / 2 + 2.0 ** -23) * np.abs(want) + TINY[ctype] + \
        2.0 ** -40 * size
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


def _same4(row, codes, blocks):
    """Is this the row's 4-bit form (up to elements on a border)?"""
    want, wb = st.pack(row)
    for i in range(len(wb)):
        xs = row[32 * i:32 * i + 32]
        top = np.abs(xs).max()
        if blocks[i] != wb[i]:
            edge = 7 * 2.0 ** (min(int(blocks[i]), int(wb[i])) - 127)
            assert abs(top / edge - 1) < 2.0 ** -40, (top, blocks[i], wb[i])
            continue
        a = codes[16 * i:16 * i + 16]
        b = want[16 * i:16 * i + 16]
        for j in range(32):
            x = (int(a[j // 2]) >> 4 * (j % 2)) & 15
            y = (int(b[j // 2]) >> 4 * (j % 2)) & 15
            if x != y:
                z = abs(xs[j]) / 2.0 ** (int(wb[i]) - 127)
                gap = min(abs(z - m) for m in (.25, .75, 1.25, 1.75, 2.5, 3.5,
                                               5.0))
                assert gap < 2.0 ** -40 or z < 2.0 ** -40, (xs[j], x, y)


def _extend(rng, lens, counts, q_heads, heads, dim, page, qtype, ctype,
            slots_first=False, rot=None, interleaved=False, norm=None,
            seen=None, scales=False, ledger=None, spare=0, extra=1, gain=1.0,
            queries=True, edit=None):
    q, k, v = _new(rng, counts, q_heads, heads, dim, qtype, spare, gain)
    if edit:
        edit(q, k, v)
    dev, ref = _blank(rng, lens, counts, heads, dim, page, ctype, slots_first,
                      extra)
    rot = dim if rot is None else rot
    freqs = None if rot == 0 else \
        (10000.0 ** (-np.arange(rot // 2) / (rot / 2))).astype(np.float32)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    qn = kn = None
    if norm:
        qn = torch.from_numpy(1 + 0.2 * rng.standard_normal(dim)).to(
            torch.float32 if norm == "f32" else TYPES[qtype]).cuda()
        kn = torch.from_numpy(1 + 0.2 * rng.standard_normal(dim)).to(
            qn.dtype).cuda()
    ks = vs = None
    if scales:
        ks = (rng.random(heads) * 0.1 + 0.02).astype(np.float32)
        vs = (rng.random(heads) * 0.1 + 0.02).astype(np.float32)
    w = pos = None
    if ledger:
        w = torch.full((len(lens), heads, ledger), 7.0).cuda()
        pos = torch.full((len(lens), heads, ledger), -9,
                         dtype=torch.int32).cuda()
    names = [n for n in ("k", "v", "k_blocks", "v_blocks") if n in dev]
    before = {n: _raw(dev[n]) for n in names}
    out = torch.full((q.shape[0], q_heads, dim), 5.0, dtype=q.dtype).cuda()

    def cuda(x):
        return None if x is None else torch.from_numpy(x).cuda()

    got_lens, got_q = ltk.cache_extend(
        k, v, dev["k"], dev["v"], dev["table"], dev["lens"], cuda(starts),
        seen=None if seen is None else
        torch.tensor(seen, dtype=torch.int32).cuda(),
        q=q if queries else None, freqs=cuda(freqs), interleaved=interleaved,
        q_norm=qn, k_norm=kn, eps=1e-5, k_scale=cuda(ks), v_scale=cuda(vs),
        weights=w, positions=pos, k_blocks=dev.get("k_blocks"),
        v_blocks=dev.get("v_blocks"), out=out if queries else None)
    torch.cuda.synchronize()

    def host(x):
        return None if x is None else x.double().cpu().numpy()

    eps = float(np.float32(1e-5))
    want_q, writes, want_lens = st.extend(
        host(q), host(k), host(v), ref, starts, seen, host(qn), host(kn), eps,
        freqs, interleaved, ks, vs, ledger)
    assert np.array_equal(got_lens.cpu().numpy(), want_lens)
    if queries:
        assert got_q is out
        have = host(got_q)
        idle = np.isnan(want_q) & ~np.isnan(host(q)).any(-1, keepdims=True)
        assert (have[idle] == 5.0).all()
        fine = ~np.isnan(want_q)
        size = np.abs(want_q).max(-1, keepdims=True) + np.zeros_like(want_q)
        _near(have[fine], want_q[fine], size[fine], qtype)
    else:
        assert got_q is None
    after = {n: _raw(dev[n]) for n in names}
    if ledger:
        want_w, want_p = np.full(w.shape, 7.0), np.full(w.shape, -9)
        for _, h, _, _, _, b, slot, position in writes:
            want_w[b, h, slot], want_p[b, h, slot] = 0.0, position
        assert np.array_equal(w.cpu().numpy(), want_w)
        assert np.array_equal(pos.cpu().numpy(), want_p)
    for page_, h, place, x, z, b, slot, _ in writes:
        if page_ is None:
            continue
        for name, row in (("k", x), ("v", z)):
            if ctype == "e2m1":
                _same4(row, after[name][page_, h, place],
                       after[name + "_blocks"][page_, h, place])
                before[name + "_blocks"][page_, h, place] = \
                    after[name + "_blocks"][page_, h, place]
            else:
                have = torch.from_numpy(after[name][page_, h, place]).view(
                    TYPES[ctype]).double().numpy()
                if ctype == "e4m3":
                    row = np.clip(row, -448, 448)
                _near(have, row, np.abs(row).max(), ctype)
            before[name][page_, h, place] = after[name][page_, h, place]
    for n in names:  # nothing else has changed
        assert np.array_equal(before[n], after[n]), n
    return dev


LENS = [0, 5, 16, 31, 100]
COUNTS = [3, 0, 1, 40, 17]


@pytest.mark.parametrize("qtype,ctype", [
    ("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"),
    ("bf16", "e2m1"), ("f16", "e2m1")])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192, 256])
def test_extend_types(qtype, ctype, dim):
    print("extend", qtype, ctype, dim, flush=True)
    rng = np.random.default_rng(dim)
    _extend(rng, LENS, COUNTS, 4, 2, dim, 16, qtype, ctype, norm="own",
            scales=True)


@pytest.mark.parametrize("dim,rot", [(8, 0), (24, 16), (40, 32), (72, 64),
                                     (80, 80), (136, 16), (200, 192),
                                     (248, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_extend_odd_rows(dim, rot, interleaved):
    print("extend rows", dim, rot, interleaved, flush=True)
    rng = np.random.default_rng(dim)
    _extend(rng, LENS, COUNTS, 3, 3, dim, 20, "bf16", "bf16", True, rot,
            interleaved, norm="f32")


@pytest.mark.parametrize("ctype", ["bf16", "e2m1"])
@pytest.mark.parametrize("counts,q_heads,heads,page", [
    ([1] * 64, 8, 2, 16), ([1], 32, 8, 16), ([1000], 2, 1, 64),
    ([0, 0, 7], 1, 1, 1), ([300, 1, 0, 2, 500], 5, 5, 24),
    ([i % 3 for i in range(700)], 2, 1, 8)])
def test_extend_shapes(ctype, counts, q_heads, heads, page):
    print("extend shapes", ctype, len(counts), sum(counts), flush=True)
    rng = np.random.default_rng(len(counts))
    lens = [int(x) for x in rng.integers(0, 50, len(counts))]
    _extend(rng, lens, counts, q_heads, heads, 32, page, "bf16", ctype,
            seen=[3 * x for x in lens], ledger=1200)


def test_extend_without_queries_norms_or_rotation():
    for ctype in ("bf16", "e4m3", "e2m1"):
        rng = np.random.default_rng(1)
        _extend(rng, LENS, COUNTS, 4, 2, 64, 16, "bf16", ctype, rot=0,
                queries=False)
        _extend(rng, LENS, COUNTS, 4, 2, 64, 16, "bf16", ctype, norm="f32",
                rot=0)


def test_extend_far_positions():
    rng = np.random.default_rng(2)
    _extend(rng, [4, 9], [5, 3], 2, 2, 64, 16, "bf16", "bf16",
            seen=[10 ** 6, 2 ** 24 - 2])
    _extend(rng, [4, 9], [5, 3], 2, 2, 64, 16, "f16", "f16",
            seen=[-10 ** 5, 2 ** 20 + 1], interleaved=True)


def test_extend_stops_at_the_table_and_the_ledger():
    rng = np.random.default_rng(3)
    # no room beyond what is needed: lengths end inside the table
    for ledger in (None, 40):
        _extend(rng, [60, 10, 64, 70, -3], [10, 3, 1, 2, 4], 2, 1, 64, 16,
                "bf16", "e2m1", ledger=ledger, extra=0)


def test_extend_bounds_slots_by_a_narrow_table():
    rng = np.random.default_rng(4)
    q, k, v = _new(rng, [40, 2], 2, 1, 64, "bf16")
    dev, ref = _blank(rng, [20, 0], [40, 2], 1, 64, 16, "bf16", extra=0)
    narrow = dev["table"][:, :2]  # 32 slots
    before = _raw(dev["k"])
    lens, out = ltk.cache_extend(k, v, dev["k"], dev["v"], narrow, dev["lens"],
                                 torch.tensor([0, 40, 42],
                                              dtype=torch.int32).cuda(), q=q)
    assert lens.tolist() == [32, 2] and torch.equal(out, q)
    after = _raw(dev["k"])
    third = int(ref["table"][0, 2])
    assert np.array_equal(before[third], after[third])
    t = [int(x) for x in ref["table"][0, :2]]
    assert np.array_equal(after[t[1], 0, 4:],
                          _raw(k[:12, 0].contiguous()))


def test_extend_pages_that_are_not_there():
    rng = np.random.default_rng(5)
    q, k, v = _new(rng, [40, 2], 2, 1, 64, "bf16")
    dev, ref = _blank(rng, [3, 0], [40, 2], 1, 64, 16, "bf16")
    pages = dev["k"].shape[0]
    table = ref["table"].copy()
    table[0, 1], table[1, 0] = -1, pages
    lost = [int(ref["table"][0, 1]), int(ref["table"][1, 0])]
    before = _raw(dev["v"])
    w = torch.ones(2, 1, 64).cuda()
    p = torch.zeros(2, 1, 64, dtype=torch.int32).cuda()
    lens, _ = ltk.cache_extend(
        k, v, dev["k"], dev["v"], torch.from_numpy(table).cuda(), dev["lens"],
        torch.tensor([0, 40, 42], dtype=torch.int32).cuda(), q=q, weights=w,
        positions=p)
    after = _raw(dev["v"])
    assert lens.tolist() == [43, 2]
    for page in lost:
        assert np.array_equal(before[page], after[page])
    first = int(table[0, 0])
    assert np.array_equal(after[first, 0, 3:], _raw(v[:13, 0].contiguous()))
    assert not w[0, 0, 3:43].any() and w[0, 0, :3].all() and w[0, 0, 43:].all()
    assert p[0, 0, 3:43].tolist() == list(range(3, 43))


def test_extend_leaves_tokens_of_no_sequence_alone():
    rng = np.random.default_rng(6)
    _extend(rng, LENS, COUNTS, 4, 2, 64, 16, "bf16", "e4m3", spare=9)
    # starts that begin late, go past the tokens, or step back write nothing
    # outside the arrays
    q, k, v = _new(rng, [10], 2, 1, 64, "bf16")
    dev, _ = _blank(rng, [0, 0, 0], [10, 10, 10], 1, 64, 16, "bf16")
    for starts, want in (([2, 4, 4, 6], [2, 0, 2]),
                         ([0, 5, 99, 2 ** 31 - 1], [5, 5, 0]),
                         ([-7, 5, 5, 10], [5, 0, 5]),
                         ([4, 2, 8, 1], None)):
        out = torch.zeros_like(q).contiguous()
        lens, _ = ltk.cache_extend(
            k, v, dev["k"], dev["v"], dev["table"], dev["lens"],
            torch.tensor(starts, dtype=torch.int32).cuda(), q=q, out=out)
        torch.cuda.synchronize()
        if want:
            assert lens.tolist() == want
            a, b = max(starts[0], 0), min(starts[-1], 10)
            assert torch.equal(out[a:b], q[a:b])
            assert not out[:a].any() and not out[b:].any()


def test_extend_extreme_numbers():
    """Large, tiny, infinite and NaN values, and blocks at the borders of
    their scales."""
    def edit(q, k, v):
        rows = v[:, 0]
        rows[0] = 0
        rows[1] = 2.0 ** -133
        rows[2] = 3e38
        rows[3, ::2], rows[3, 1::2] = 7.0, -6.96875
        rows[4] = 6.96875
        rows[5, :32] = torch.tensor([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5] * 4)
        rows[5, 32:] = -rows[5, :32]
        rows[6] = 2.0 ** -120
        k[0] = 0
        q[0] = 0
        k[1] = 1e19
        q[1] = 1e19

    for ctype in ("bf16", "e2m1"):
        rng = np.random.default_rng(7)
        _extend(rng, [0], [9], 2, 2, 64, 16, "bf16", ctype, norm="f32",
                edit=edit)
    # e4m3 saturates
    rng = np.random.default_rng(7)
    _extend(rng, [0], [9], 2, 2, 64, 16, "bf16", "e4m3", gain=400.0)
    # infinities and NaN: in 4 bits the block is NaN, in 8 infinities saturate
    x = torch.ones(3, 1, 64, dtype=torch.bfloat16).cuda()
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 5] = float("inf"), float("nan"), \
        -float("inf")
    table = torch.zeros(1, 1, dtype=torch.int32).cuda()
    lens = torch.zeros(1, dtype=torch.int32).cuda()
    starts = torch.tensor([0, 3], dtype=torch.int32).cuda()
    c = torch.zeros(1, 1, 16, 32, dtype=torch.uint8).cuda()
    b = torch.zeros(1, 1, 16, 2, dtype=torch.uint8).cuda()
    ltk.cache_extend(x, x, c.view(torch.float4_e2m1fn_x2),
                     c.clone().view(torch.float4_e2m1fn_x2), table, lens,
                     starts, k_blocks=b.view(torch.float8_e8m0fnu),
                     v_blocks=b.clone().view(torch.float8_e8m0fnu))
    assert b[0, 0, :3].tolist() == [[255, 125], [125, 255], [255, 125]]
    e = torch.zeros(1, 1, 16, 64).cuda().to(torch.float8_e4m3fn)
    ltk.cache_extend(x, x, e, e.clone(), table, lens, starts)
    e = e.float()
    assert e[0, 0, 0, 3] == 448 and e[0, 0, 2, 5] == -448
    assert e[0, 0, 1, 40].isnan() and e[0, 0, 1, 41] == 1


def test_extend_in_place():
    """Queries turned where they are, in the projection's own output."""
    rng = np.random.default_rng(8)
    for n in ([30, 1], [1]):
        q, k, v = _new(rng, n, 4, 2, 64, "bf16")
        dev, _ = _blank(rng, [0] * len(n), n, 2, 64, 16, "bf16")
        f = torch.linspace(1, 0.01, 32).cuda()
        starts = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32)
        args = (k, v, dev["k"], dev["v"], dev["table"], dev["lens"],
                starts.cuda())
        _, want = ltk.cache_extend(*args, q=q, freqs=f, q_norm=f.repeat(2))
        keep = k.clone(), v.clone()
        if len(n) > 1:
            _, got = ltk.cache_extend(*args, q=q, freqs=f,
                                      q_norm=f.repeat(2), out=q)
            assert got is q
        else:
            q = q.contiguous()
            ltk.cache_extend(*args, q=q, freqs=f, q_norm=f.repeat(2), out=q)
        assert torch.equal(q, want)
        assert torch.equal(k, keep[0]) and torch.equal(v, keep[1])


def test_extend_any_stream_and_graph():
    rng = np.random.default_rng(9)
    q, k, v = _new(rng, [30, 1, 2], 4, 2, 128, "bf16")
    dev, _ = _blank(rng, [0, 3, 40], [30, 1, 2], 2, 128, 16, "e2m1")
    f = torch.linspace(1, 0.01, 64).cuda()
    starts = torch.tensor([0, 30, 31, 33], dtype=torch.int32).cuda()
    blank = {n: dev[n].view(torch.uint8).clone() for n in
             ("k", "v", "k_blocks", "v_blocks")}

    def call(d):
        return ltk.cache_extend(
            k, v, d["k"], d["v"], d["table"], d["lens"], starts, q=q, freqs=f,
            k_blocks=d["k_blocks"], v_blocks=d["v_blocks"])

    lens, out = call(dev)
    want = {n: dev[n].view(torch.uint8).clone() for n in blank}
    s = dict(dev)
    for n in blank:
        s[n] = blank[n].clone().view(dev[n].dtype)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            lens2, out2 = call(s)
    for i in range(3):
        for n in blank:
            s[n].view(torch.uint8).copy_(blank[n])
        out2.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert torch.equal(out, out2) and torch.equal(lens, lens2)
        assert all(torch.equal(s[n].view(torch.uint8), want[n])
                   for n in blank)


def test_extend_past_32_bits():
    """A cache whose rows lie more than 2^32 bytes apart."""
    pages, page, dim = 40000, 512, 128
    dev = torch.device("cuda")
    k = torch.zeros(pages, 1, page, dim, dtype=torch.bfloat16, device=dev)
    assert k.numel() * 2 > 2 ** 32
    vv = torch.zeros_like(k)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device=dev)
    x = torch.randn(3, 1, dim, device=dev).to(torch.bfloat16)
    ltk.cache_extend(x, x * 2, k, vv, table,
                     torch.tensor([500], dtype=torch.int32, device=dev),
                     torch.tensor([0, 3], dtype=torch.int32, device=dev))
    assert torch.equal(k[pages - 1, 0, 500:503], x[:, 0])
    assert torch.equal(vv[pages - 1, 0, 500:503], (x * 2)[:, 0])
    assert not k[0].any() and not k[pages - 1, 0, :500].any()


def test_gradients_are_refused():
    rng = np.random.default_rng(10)
    q, k, v = _new(rng, [4], 2, 1, 64, "bf16")
    dev, _ = _blank(rng, [0], [4], 1, 64, 16, "bf16")
    q = q.detach().clone().requires_grad_()
    starts = torch.tensor([0, 4], dtype=torch.int32).cuda()
    version = dev["k"]._version
    _, out = ltk.cache_extend(k, v, dev["k"], dev["v"], dev["table"],
                              dev["lens"], starts, q=q)
    assert dev["k"]._version > version
    with pytest.raises(RuntimeError, match="cache_extend"):
        out.float().sum().backward()
