"""The paged-cache operators on the CPU: where rows lie and how slots are
ordered (the kernels' own integer header, compiled with g++), the oracle on
hand-worked cases, and the refusals of the C interface and of the binding."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle.cache as oc
import top_selection_two_amd as ltk

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "top_selection_two_amd", "csrc")
FAKE = 0x100000  # addresses that are never dereferenced


# ------------------------------------------------------------------ layout
LAYOUT = r"""
#include "cache_layout.hpp"
extern "C" {
int quotient_of(int n, int d) { return ltk::quotient(ltk::make_divisor(d), n); }
int ok(int id, long long pages) { return ltk::page_ok(id, pages); }
int len_of(int len, int cap) { return ltk::clamp_len(len, cap); }
int key(int bits, int pos, int seen, int sinks, int recent) {
  return ltk::rank_key(bits, pos, seen, sinks, recent);
}
unsigned long long word(int key, int slot) { return ltk::rank_word(key, slot); }
long long offset(long long p, long long h, long long s, int id, int head,
                 int place) {
  return ltk::row_offset(ltk::RowStrides{p, h, s}, id, head, place);
}
}
"""


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    d = tmp_path_factory.mktemp("layout")
    src, so = str(d / "layout.cpp"), str(d / "layout.so")
    with open(src, "w") as f:
        f.write(LAYOUT)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
                           "-I", CSRC, src, "-o", so])
    lib = ctypes.CDLL(so)
    lib.word.restype = ctypes.c_uint64
    lib.offset.restype = ctypes.c_int64
    lib.offset.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 3
    lib.ok.argtypes = [ctypes.c_int, ctypes.c_int64]
    return lib


def test_quotient_is_exact(layout):
    top = 2 ** 31 - 1
    for d in list(range(1, 70)) + [100, 127, 128, 255, 256, 257, 999, 65535,
                                   65536, 65537, 2 ** 29 + 1, 2 ** 30 - 1]:
        ns = {0, 1, d - 1, d, d + 1, top, top - 1, 2 ** 30, 2 ** 30 - 1}
        m = top // d
        for q in (2, 3, 1000, m // 2, m - 1, m):
            ns |= {q * d - 1, q * d, q * d + 1}
        for n in ns:
            if 0 <= n <= top:
                assert layout.quotient_of(n, d) == n // d, (n, d)


def test_pages_and_lengths_are_bounded(layout):
    assert [layout.ok(i, 5) for i in (-2 ** 31, -1, 0, 4, 5, 2 ** 31 - 1)] \
        == [0, 0, 1, 1, 0, 0]
    assert layout.ok(0, 0) == 0
    assert [layout.len_of(n, 48) for n in (-2 ** 31, -1, 0, 47, 48, 49,
                                           2 ** 31 - 1)] \
        == [0, 0, 0, 47, 48, 48, 48]


def test_offsets_pass_32_bits(layout):
    assert layout.offset(2 ** 20, 2 ** 12, 256, 2 ** 22, 7, 15) == \
        2 ** 42 + 7 * 2 ** 12 + 15 * 256


def _bits(x):
    return int(np.float32(x).view(np.int32))


def test_keys_follow_the_numbers(layout):
    xs = [-np.inf, -3.5, -1e-40, -0.0, 0.0, 1e-40, 1e-3, 2.0, np.inf]
    keys = [layout.key(_bits(x), 500, 1000, 4, 64) for x in xs]
    assert keys == sorted(keys) and len(set(keys)) == len(keys)
    nan = layout.key(0x7fc00000, 500, 1000, 4, 64)
    assert keys[-1] < nan < 2 ** 31 - 1
    assert layout.key(-1, 500, 1000, 4, 64) == -2 ** 31
    safe = 2 ** 31 - 1
    for pos, want in ((0, True), (3, True), (4, False), (935, False),
                      (936, True), (2000, True), (-1, True)):
        got = layout.key(_bits(1.0), pos, 1000, 4, 64) == safe
        assert got == want, pos
    # the window's lower end passes the least int32
    assert layout.key(_bits(1.0), 5, -2 ** 31, 0, 2 ** 31 - 1) == safe
    assert layout.key(_bits(1.0), 5, 2 ** 31 - 1, 0, 0) != safe


def test_words_order_by_key_then_earlier_slot(layout):
    seq = [(2 ** 31 - 1, 0), (2 ** 31 - 1, 9), (7, 3), (0, 0), (0, 1),
           (0, 2 ** 30), (-1, 0), (-2 ** 31, 5)]
    words = [layout.word(k, t) for k, t in seq]
    assert words == sorted(words, reverse=True)
    assert len(set(words)) == len(words)


# ------------------------------------------------------------------ oracle
def _cache(k, v, table, lens):
    return {"k": np.asarray(k, float), "v": np.asarray(v, float),
            "table": np.asarray(table, np.int32),
            "lens": np.asarray(lens, np.int32)}


def test_oracle_attends_by_hand():
    # two pages of two slots, one head, rows of one element; slot order is
    # page 1 then page 0; three slots in use, scores 0, ln 3, 0
    k = np.array([[[[0.0], [99.0]]], [[[0.0], [math.log(3)]]]])
    v = np.array([[[[5.0], [99.0]]], [[[10.0], [20.0]]]])
    c = _cache(k, v, [[1, 0]], [3])
    out, lse, added, spread, _ = oc.attend([[[1.0], [0.0]]], c, 1.0)
    assert np.allclose(out[0, 0], (10 + 3 * 20 + 5) / 5)
    assert np.allclose(out[0, 1], 35 / 3)
    assert np.allclose(lse, [[math.log(5), math.log(3)]])
    assert np.allclose(added[0, 0], [1 / 5 + 1 / 3, 3 / 5 + 1 / 3,
                                     1 / 5 + 1 / 3, 0])
    c["lens"][0] = 0
    out, lse, added, _, _ = oc.attend([[[1.0], [0.0]]], c, 1.0)
    assert not out.any() and not added.any() and (lse == -np.inf).all()
    # without page 1 only slot 2 is left
    c["lens"][0], c["table"][0, 0] = 3, 2
    out, lse, added, _, _ = oc.attend([[[1.0], [0.0]]], c, 1.0)
    assert np.allclose(out, 5) and np.allclose(added[0, 0], [0, 0, 2, 0])


def test_oracle_appends_and_evicts_by_hand():
    k = np.arange(8.0).reshape(2, 1, 4, 1)
    c = _cache(k, k + 100, [[0, 1]], [6])
    w = np.array([[[5, 1, 1, 7, 3, 9, 0, 0]]], np.float32)
    pos = np.arange(8, dtype=np.int32).reshape(1, 1, 8)
    seen = np.array([6], np.int32)
    new = np.array([[[-1.0]]])
    # full at 6: the lowest weight, the later of the two equal slots
    k2, v2, w2, p2, slots, lens = oc.append(new, new, c, 6, seen, w, pos, 0,
                                            0)
    assert slots[0, 0] == 2 and lens[0] == 6 and k2[0, 0, 2, 0] == -1
    assert w2[0, 0, 2] == 0 and p2[0, 0, 2] == 6
    # not full at 7
    _, v2, _, p2, slots, lens = oc.append(new, new, c, 7, seen, w, pos, 0, 0)
    assert slots[0, 0] == 6 and lens[0] == 7 and v2[1, 0, 2, 0] == -1
    # keep 3: order 5 (9), 3 (7), 0 (5) -> holes 1, 2 from 3, 5
    k2, _, w2, p2, lens = oc.evict(c, seen, w, pos, 3, 0, 0)
    assert lens[0] == 3 and w2[0, 0].tolist() == [5, 7, 9]
    assert p2[0, 0].tolist() == [0, 3, 5]
    assert k2[0, 0, :, 0].tolist() == [0, 3, 5, 3]
    # protected: sink 0..1, last two positions 4, 5
    _, _, _, p2, _ = oc.evict(c, seen, w, pos, 4, 2, 2)
    assert p2[0, 0].tolist() == [0, 1, 4, 5]
    # nothing to do
    _, _, w2, p2, lens = oc.evict(c, seen, w, pos, 8, 0, 0)
    assert lens[0] == 6 and w2[0, 0].tolist() == [5, 1, 1, 7, 3, 9, 0, 0]
    assert p2[0, 0].tolist() == [0, 1, 2, 3, 4, 5, -1, -1]


# ------------------------------------------------- refusals, C interface
def _c(**kw):
    c = dict(k=FAKE, v=FAKE << 12, k_page_stride=4 * 16 * 64,
             k_head_stride=16 * 64, k_slot_stride=64,
             v_page_stride=4 * 16 * 64, v_head_stride=16 * 64,
             v_slot_stride=64, pages=32, table_stride=4, table=FAKE << 13,
             lens=FAKE << 14, batch=2, table_width=4, heads=4, page=16,
             dim=64, dtype=ltk.BF16)
    c.update(kw)
    return ltk.CacheStruct(**c)


def _l(base=FAKE << 15, **kw):
    d = dict(weights=base, positions=base + 0x40000,
             weights_batch_stride=256, weights_head_stride=64,
             positions_batch_stride=256, positions_head_stride=64, slots=64)
    d.update(kw)
    return ltk.LedgerStruct(**d)


def _attend(c=None, q=FAKE << 16, q_dtype=0, q_heads=8, qb=512, qh=64,
            ks=None, vs=None, ledger=None, out=FAKE << 17, lse=FAKE << 18):
    return ltk.lib.cache_attend(c if c is not None else _c(), q, q_dtype,
                                q_heads, qb, qh, 0.125, ks, vs, ledger, out,
                                lse, None)


def _append(c=None, kn=FAKE << 16, vn=(FAKE << 16) + 0x1000, nb=256, nh=64,
            limit=32, seen=FAKE << 17, ledger=None, sinks=4, recent=8,
            lens=FAKE << 18, slots=FAKE << 19):
    return ltk.lib.cache_append(c if c is not None else _c(), kn, vn, nb, nh,
                                limit, seen,
                                ledger if ledger is not None else _l(),
                                sinks, recent, lens, slots, None)


def _evict(c=None, seen=FAKE << 17, ledger=None, keep=32, sinks=4, recent=8,
           after=None, lens=FAKE << 18):
    return ltk.lib.cache_evict(
        c if c is not None else _c(), seen,
        ledger if ledger is not None else _l(), keep, sinks, recent,
        after if after is not None else _l(FAKE << 20), lens, None)


BAD_CACHES = [
    dict(k=0), dict(v=0), dict(k=FAKE + 8), dict(v=(FAKE << 12) + 2),
    dict(table=0), dict(lens=0), dict(table=(FAKE << 13) + 2),
    dict(lens=(FAKE << 14) + 1), dict(batch=-1), dict(pages=-1),
    dict(pages=2 ** 31), dict(heads=0), dict(heads=65536), dict(page=0),
    dict(page=-4), dict(dim=0), dict(dim=60), dict(dim=264),
    dict(dim=56, dtype=ltk.E4M3), dict(dtype=3), dict(dtype=-1),
    dict(table_width=0), dict(table_width=2 ** 26, page=16),
    dict(k_page_stride=-1), dict(v_slot_stride=-64),
    dict(k_slot_stride=68), dict(v_head_stride=1028),
    dict(k_page_stride=2 ** 61), dict(v_page_stride=2 ** 57),
    dict(table_stride=-1), dict(table_stride=2 ** 60),
]


@pytest.mark.parametrize("kw", BAD_CACHES, ids=str)
def test_calls_refuse_bad_caches(kw):
    for call in (_attend, _append, _evict):
        assert call(_c(**kw)) == ltk.ERR_INVALID


def test_null_cache_and_ledgers():
    assert ltk.lib.cache_attend(None, FAKE, 0, 8, 512, 64, 1.0, None, None,
                                None, FAKE << 17, FAKE << 18, None) \
        == ltk.ERR_INVALID
    assert ltk.lib.cache_append(_c(), FAKE << 16, FAKE << 16, 256, 64, 32,
                                FAKE << 17, None, 4, 8, FAKE << 18,
                                FAKE << 19, None) == ltk.ERR_INVALID
    assert ltk.lib.cache_evict(_c(), FAKE << 17, _l(), 32, 4, 8, None,
                               FAKE << 18, None) == ltk.ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=(FAKE << 16) + 8), dict(q_dtype=2), dict(q_dtype=1),
    dict(q_heads=0), dict(q_heads=6), dict(q_heads=-8), dict(qb=516),
    dict(qh=-64), dict(qh=65), dict(qb=2 ** 61), dict(ks=FAKE + 2),
    dict(vs=FAKE + 1), dict(out=None), dict(out=(FAKE << 17) + 4),
    dict(lse=None), dict(lse=(FAKE << 18) + 2),
    dict(out=FAKE << 16), dict(out=FAKE), dict(out=FAKE << 12),
    dict(out=FAKE << 13), dict(lse=FAKE << 14), dict(lse=FAKE << 17),
    dict(vs=(FAKE << 18) + 16),
    dict(ledger=_l(weights=0)), dict(ledger=_l(weights=FAKE + 2)),
    dict(ledger=_l(slots=0)), dict(ledger=_l(weights_batch_stride=-1)),
    dict(ledger=_l(weights_head_stride=32)),      # rows overlap
    dict(ledger=_l(weights_batch_stride=192)),    # sequences overlap
    dict(ledger=_l(weights=FAKE + 64)),           # in k
    dict(ledger=_l(weights=FAKE << 17)),          # on out
], ids=str)
def test_attend_refuses(kw):
    assert _attend(**kw) == ltk.ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(kn=None), dict(vn=None), dict(kn=(FAKE << 16) + 4), dict(nb=260),
    dict(nh=-64), dict(nh=4), dict(limit=0), dict(limit=-1), dict(seen=None),
    dict(seen=(FAKE << 17) + 2), dict(sinks=-1), dict(recent=-1),
    dict(lens=None), dict(slots=None), dict(lens=FAKE << 14),
    dict(lens=FAKE << 19), dict(slots=(FAKE << 19) + 1), dict(kn=FAKE),
    dict(slots=FAKE << 15), dict(ledger=_l(positions=0)),
    dict(ledger=_l(positions=FAKE << 15)),        # on the weights
    dict(ledger=_l(positions_head_stride=8)),
], ids=str)
def test_append_refuses(kw):
    assert _append(**kw) == ltk.ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(seen=None), dict(keep=0), dict(keep=65), dict(sinks=-1),
    dict(recent=-1), dict(lens=None), dict(lens=FAKE << 14),
    dict(after=_l(FAKE << 20, weights=0)), dict(after=_l(FAKE << 15)),
    dict(after=_l(FAKE)), dict(after=_l(FAKE << 20, positions=FAKE << 20)),
    dict(after=_l(FAKE << 20, positions_head_stride=16)),
    dict(ledger=_l(weights=0)), dict(ledger=_l(positions=FAKE + 1)),
], ids=str)
def test_evict_refuses(kw):
    assert _evict(**kw) == ltk.ERR_INVALID


def test_no_sequences_is_a_no_op():
    none = _c(batch=0, table=0, lens=0)
    led = _l(0, positions=0)
    assert _attend(none, q=None, out=None, lse=None) == ltk.OK
    assert _append(none, kn=None, vn=None, seen=None, ledger=led, lens=None,
                   slots=None) == ltk.OK
    assert _evict(none, seen=None, ledger=led, after=led, lens=None) == ltk.OK
    assert _attend(none, q_heads=3) == ltk.ERR_INVALID


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is visible")
def test_valid_calls_without_a_device():
    assert _attend() == ltk.ERR_HIP
    assert _attend(ledger=_l()) == ltk.ERR_HIP
    assert _attend(_c(dtype=ltk.E4M3), q_dtype=1) == ltk.ERR_HIP
    assert _append() == ltk.ERR_HIP
    assert _evict() == ltk.ERR_HIP
    # rows of the two arrays interleaved in one
    both = dict(k_page_stride=8 * 16 * 64, v_page_stride=8 * 16 * 64,
                v=FAKE + 4 * 16 * 64 * 2)
    assert _append(_c(**both)) == ltk.ERR_HIP
    assert _evict(_c(**both)) == ltk.ERR_HIP


# ------------------------------------------------------ refusals, binding
def _t(**kw):
    bf = torch.bfloat16
    d = dict(q=torch.zeros(2, 8, 64, dtype=bf),
             k=torch.zeros(32, 4, 16, 64, dtype=bf),
             v=torch.zeros(32, 4, 16, 64, dtype=bf),
             table=torch.zeros(2, 4, dtype=torch.int32),
             lens=torch.zeros(2, dtype=torch.int32),
             seen=torch.zeros(2, dtype=torch.int32),
             new=torch.zeros(2, 4, 64, dtype=bf),
             weights=torch.zeros(2, 4, 64),
             positions=torch.zeros(2, 4, 64, dtype=torch.int32))
    d.update(kw)
    return d


def _calls(d):
    yield lambda: ltk.cache_attend(d["q"], d["k"], d["v"], d["table"],
                                   d["lens"], weights=d["weights"])
    yield lambda: ltk.cache_append(d["new"], d["new"], d["k"], d["v"],
                                   d["table"], d["lens"], 32, d["seen"],
                                   d["weights"], d["positions"])
    yield lambda: ltk.cache_evict(d["k"], d["v"], d["table"], d["lens"],
                                  d["seen"], d["weights"], d["positions"], 32)


def test_binding_wants_device_tensors():
    for call in _calls(_t()):
        with pytest.raises(ValueError, match="device"):
            call()


@pytest.mark.parametrize("kw,error", [
    (dict(k=np.zeros((32, 4, 16, 64))), TypeError),
    (dict(k=torch.zeros(32, 4, 16, 64)), TypeError),
    (dict(v=torch.zeros(32, 4, 16, 64, dtype=torch.float16)), TypeError),
    (dict(v=torch.zeros(32, 4, 8, 64, dtype=torch.bfloat16)), ValueError),
    (dict(k=torch.zeros(32, 4, 64, dtype=torch.bfloat16)), ValueError),
    (dict(k=torch.zeros(32, 4, 64, 16, dtype=torch.bfloat16)
          .transpose(2, 3)), ValueError),
    (dict(table=torch.zeros(2, 4, dtype=torch.int64)), TypeError),
    (dict(table=torch.zeros(8, dtype=torch.int32)), ValueError),
    (dict(table=torch.zeros(2, 0, dtype=torch.int32)), ValueError),
    (dict(lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(lens=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(lens=torch.zeros(4, dtype=torch.int32)[::2]), ValueError),
    (dict(weights=torch.zeros(2, 3, 64)), ValueError),
    (dict(weights=torch.zeros(2, 4, 64, dtype=torch.float64)), TypeError),
    (dict(weights=torch.zeros(2, 4, 0)), ValueError),
    (dict(weights=torch.zeros(2, 64, 4).transpose(1, 2)), ValueError),
], ids=lambda x: str(x)[:40])
def test_binding_refuses(kw, error):
    for call in _calls(_t(**kw)):
        with pytest.raises(error):
            call()


def test_binding_refuses_rows():
    bad = dict(k=torch.zeros(32, 4, 16, 60, dtype=torch.bfloat16),
               v=torch.zeros(32, 4, 16, 60, dtype=torch.bfloat16))
    big = dict(k=torch.zeros(2, 1, 2, 264, dtype=torch.bfloat16),
               v=torch.zeros(2, 1, 2, 264, dtype=torch.bfloat16))
    for kw in (bad, big):
        for call in _calls(_t(**kw)):
            with pytest.raises(ValueError, match="16 bytes"):
                call()


@pytest.mark.parametrize("kw,error", [
    (dict(q=torch.zeros(2, 6, 64, dtype=torch.bfloat16)), ValueError),
    (dict(q=torch.zeros(2, 0, 64, dtype=torch.bfloat16)), ValueError),
    (dict(q=torch.zeros(2, 8, 32, dtype=torch.bfloat16)), ValueError),
    (dict(q=torch.zeros(2, 8, 64)), TypeError),
    (dict(q=torch.zeros(2, 8, 64, dtype=torch.float16)), TypeError),
    (dict(q=torch.zeros(2, 64, 8, dtype=torch.bfloat16).transpose(1, 2)),
     ValueError),
], ids=lambda x: str(x)[:40])
def test_attend_binding_refuses(kw, error):
    with pytest.raises(error):
        next(_calls(_t(**kw)))()


def test_slots_binding_refuses():
    d = _t()
    for limit in (0, 2 ** 31, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="limit"):
            ltk.cache_append(d["new"], d["new"], d["k"], d["v"], d["table"],
                             d["lens"], limit, d["seen"], d["weights"],
                             d["positions"])
    for keep in (0, -1, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="keep"):
            ltk.cache_evict(d["k"], d["v"], d["table"], d["lens"], d["seen"],
                            d["weights"], d["positions"], keep)
    for name in ("weights", "positions"):
        with pytest.raises(ValueError):
            list(_calls(_t(**{name: None})))[2]()
    with pytest.raises(TypeError):
        list(_calls(_t(new=torch.zeros(2, 4, 64))))[1]()
    with pytest.raises(ValueError, match="out"):
        ltk.cache_evict(d["k"], d["v"], d["table"], d["lens"], d["seen"],
                        d["weights"], d["positions"], 32,
                        out=(torch.zeros(2, 4, 33),
                             torch.zeros(2, 4, 33, dtype=torch.int32)))
