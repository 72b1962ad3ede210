"""The calls around the paged cache in a decoding step, on the CPU: the oracle
on hand-worked cases, what the C entry points refuse and launch, and what the
binding refuses."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle.step as st
import test_cache_host as host
import top_selection_two_amd as ltk

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
FAKE = host.FAKE


# ------------------------------------------------------------------- oracle
def test_four_bits_by_hand():
    assert [st.code_of(x) for x in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)] \
        == [0, 2, 2, 4, 4, 6, 6]            # halves go to the even code
    assert [st.code_of(x) for x in (0.26, -0.24, -0.0, 6.9, -100.0)] \
        == [1, 8, 8, 7, 15]
    assert st.block_byte([0.0] * 32) == 0
    assert st.block_byte([6.0, -6.99]) == 127
    assert st.block_byte([7.0]) == 128      # 7 itself does not fit
    assert st.block_byte([3.5]) == 127 and st.block_byte([3.4]) == 126
    assert st.block_byte([math.inf]) == st.block_byte([math.nan]) == 255
    row = [0.5 * i for i in range(13)] + [0.0] * 19 + [-1.0] * 32
    codes, blocks = st.pack(row)
    assert blocks.tolist() == [127, 125]
    assert codes[:7].tolist() == [0x10, 0x32, 0x44, 0x65, 0x66, 0x76, 0x07]
    assert codes[16] == 0xee                # -1 = -4 * 2^-2
    back = st.unpack(codes[None], blocks[None])[0]
    assert back[:6].tolist() == [0, .5, 1, 1.5, 2, 2] and back[32] == -1
    assert math.isnan(st.unpack(codes, np.array([255, 0], np.uint8))[0])


def test_extension_by_hand():
    cache = {"k": np.zeros((3, 1, 2, 8)), "v": np.zeros((3, 1, 2, 8)),
             "table": np.array([[2, 0], [1, 7]], np.int32),
             "lens": np.array([1, 1], np.int32)}
    k = np.ones((5, 1, 8))
    freqs = [math.pi / 2] * 4
    q, writes, lens = st.extend(k, k, 3 * k, cache, [0, 2, 5], seen=[9, 1],
                                freqs=freqs, k_norm=2 * np.ones(8),
                                k_scale=[4.0], v_scale=[3.0])
    assert lens.tolist() == [3, 4]
    assert [(w[0], w[2], w[5], w[6], w[7]) for w in writes] == \
        [(2, 1, 0, 1, 9), (0, 0, 0, 2, 10), (1, 1, 1, 1, 1),
         (None, None, 1, 2, 2), (None, None, 1, 3, 3)]
    # position 9: 9 quarter turns, (x, y) -> (-y, x); the norm of ones is 2
    assert np.allclose(writes[0][3], [-.5] * 4 + [.5] * 4)
    assert np.allclose(writes[0][4], 1)
    assert np.allclose(q[0, 0], [-1] * 4 + [1] * 4)


def test_sampling_by_hand():
    x = [0.0, math.log(4), math.log(2), math.log(1)]  # weights 1 4 2 1
    for u, token in ((0.0, 0), (0.12, 0), (0.13, 1), (0.62, 1), (0.63, 2),
                     (0.874, 2), (0.876, 3), (0.999, 3)):
        assert st.sample(x, u)[0] == token
    assert st.sample(x, 0.6)[1] == pytest.approx(math.log(0.5))
    # two kept: 1 and 2; their order is the row's
    assert st.sample(x, 0.66, top_k=2) == (1, pytest.approx(math.log(2 / 3)))
    assert st.sample(x, 0.67, top_k=2)[0] == 2
    assert st.sample(x, 0.9, top_p=0.5)[0] == 1     # 4 of 8 are half
    assert st.sample(x, 0.9, top_p=0.51)[0] == 2
    assert st.sample(x, 0.1, min_p=0.5)[0] == 1
    # equal ones: the first three are 1, 2, 0
    assert st.sample(x, 0.0, top_k=3)[0] == 0
    assert st.sample(x, 0.999, top_k=3)[0] == 2
    assert st.sample(x, 0.5, temperature=0.0) == (1, 0.0)
    assert st.sample([-math.inf, math.nan], 0.5) == (-1, -math.inf)


# ------------------------------------------------- refusals, C interface
def _c4(**kw):
    """host._c's cache in 4 bits: strides in bytes."""
    c = dict(k_page_stride=4 * 16 * 32, k_head_stride=16 * 32,
             k_slot_stride=32, v_page_stride=4 * 16 * 32,
             v_head_stride=16 * 32, v_slot_stride=32, dtype=ltk.E2M1,
             k_blocks=FAKE << 21, v_blocks=FAKE << 22,
             k_block_page_stride=128, k_block_head_stride=32,
             k_block_slot_stride=2, v_block_page_stride=128,
             v_block_head_stride=32, v_block_slot_stride=2)
    c.update(kw)
    return host._c(**c)


def _extend(c=None, ledger=None, lens=FAKE << 18, **kw):
    t = dict(q=FAKE << 23, k=FAKE << 24, v=FAKE << 25, q_out=FAKE << 26,
             q_token_stride=512, q_head_stride=64, k_token_stride=256,
             k_head_stride=64, v_token_stride=256, v_head_stride=64,
             q_out_token_stride=512, q_out_head_stride=64,
             starts=FAKE << 27, tokens=5, q_heads=8, dtype=ltk.BF16,
             norm_dtype=ltk.BF16, eps=1e-6)
    t.update(kw)
    return ltk.lib.cache_extend(c if c is not None else _c4(),
                                ltk.TokensStruct(**t), ledger, lens, None)


BAD_BLOCKS = [
    dict(k_blocks=0), dict(v_blocks=0), dict(dim=48), dict(dim=16),
    dict(dim=288), dict(k_block_slot_stride=-1),
    dict(v_block_page_stride=2 ** 61), dict(k_slot_stride=24),
    dict(k=FAKE + 8), dict(v_page_stride=4 * 16 * 32 + 8)]


@pytest.mark.parametrize("kw", BAD_BLOCKS, ids=str)
def test_calls_refuse_bad_4_bit_caches(kw):
    assert host._attend(_c4(**kw)) == ltk.ERR_INVALID
    assert host._evict(_c4(**kw)) == ltk.ERR_INVALID
    assert _extend(_c4(**kw)) == ltk.ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(k_block_slot_stride=1), dict(v_block_slot_stride=0),
    dict(k_block_head_stride=31), dict(v_block_page_stride=127),
    dict(k_slot_stride=16), dict(v_blocks=FAKE << 13)], ids=str)
def test_writers_refuse_scales_that_overlap(kw):
    c = _c4(**kw)
    assert _extend(c) == ltk.ERR_INVALID
    assert host._evict(c) == ltk.ERR_INVALID


def test_4_bit_rows_are_not_appended():
    assert host._append(_c4()) == ltk.ERR_INVALID


def test_outputs_may_not_lie_on_scales():
    c = _c4()
    assert host._attend(c, out=FAKE << 21) == ltk.ERR_INVALID
    assert host._attend(c, lse=FAKE << 22) == ltk.ERR_INVALID
    assert host._attend(c, ledger=host._l(weights=FAKE << 21)) == \
        ltk.ERR_INVALID
    assert host._evict(c, lens=FAKE << 22) == ltk.ERR_INVALID
    assert _extend(c, lens=FAKE << 22) == ltk.ERR_INVALID
    assert _extend(c, q_out=FAKE << 21) == ltk.ERR_INVALID


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(q_out=None), dict(starts=None),
    dict(lens=None), dict(k=(FAKE << 24) + 8), dict(q=(FAKE << 23) + 2),
    dict(q_out=(FAKE << 26) + 4), dict(starts=(FAKE << 27) + 2),
    dict(seen=FAKE + 2), dict(k_norm=FAKE + 1), dict(q_norm=FAKE + 1),
    dict(k_norm=(FAKE << 28) + 2, norm_dtype=ltk.F32),
    dict(k_norm=FAKE << 28, norm_dtype=ltk.F16),
    dict(k_norm=FAKE << 28, eps=-1.0), dict(q_norm=FAKE << 28, eps=math.nan),
    dict(tokens=-1), dict(q_heads=0), dict(q_heads=-4), dict(dtype=ltk.F32),
    dict(dtype=ltk.E4M3), dict(dtype=7), dict(rot=8, freqs=FAKE << 28),
    dict(rot=-16, freqs=FAKE << 28), dict(rot=80, freqs=FAKE << 28),
    dict(rot=16), dict(rot=16, freqs=(FAKE << 28) + 2),
    dict(k_token_stride=-256), dict(q_token_stride=516),
    dict(v_head_stride=60), dict(k_head_stride=2 ** 61),
    dict(q_out_token_stride=256), dict(q_out_head_stride=32),  # rows overlap
    dict(k_scale=FAKE + 2), dict(v_scale=FAKE + 1),
    dict(lens=FAKE << 14), dict(lens=FAKE << 13), dict(lens=FAKE << 27),
    dict(lens=FAKE << 26), dict(lens=FAKE), dict(q_out=FAKE << 24),
    dict(q_out=(FAKE << 23) + 1024), dict(q_out=FAKE << 12),
    dict(q_out=FAKE << 23, q_out_token_stride=1024),
    dict(k=FAKE), dict(v=FAKE << 21), dict(starts=FAKE + 64),
    dict(seen=FAKE << 18), dict(freqs=FAKE << 26, rot=16),
    dict(ledger=host._l(weights=0)), dict(ledger=host._l(positions=0)),
    dict(ledger=host._l(slots=0)),
    dict(ledger=host._l(positions=FAKE << 15)),
    dict(ledger=host._l(weights=FAKE << 21)),
    dict(ledger=host._l(weights_head_stride=32)),
    dict(c=host._c(dtype=ltk.F16)), dict(c=host._c(dtype=ltk.F32)),
    dict(c=host._c(k_slot_stride=32)),
], ids=str)
def test_extend_refuses(kw):
    assert _extend(**kw) == ltk.ERR_INVALID


def test_extend_wants_structs():
    t = ltk.TokensStruct()
    assert ltk.lib.cache_extend(None, t, None, FAKE, None) == ltk.ERR_INVALID
    assert ltk.lib.cache_extend(_c4(), None, None, FAKE, None) == \
        ltk.ERR_INVALID


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is visible")
@pytest.mark.parametrize("kw", [
    dict(), dict(q=None, q_out=None, q_heads=0), dict(tokens=0),
    dict(tokens=0, k=None, v=None, q_out=None), dict(dtype=ltk.F16),
    dict(k_norm=FAKE << 28, q_norm=FAKE << 29, norm_dtype=ltk.F32, eps=0.0),
    dict(rot=64, freqs=FAKE << 28), dict(seen=FAKE << 28),
    dict(ledger=host._l()), dict(k_scale=FAKE << 28, v_scale=FAKE << 28),
    dict(c=host._c()), dict(c=host._c(dtype=ltk.F16), dtype=ltk.F16),
    dict(c=host._c(dtype=ltk.E4M3)), dict(q_out=FAKE << 23),
    # queries turned where they are, between the keys and values of an array
    dict(q_out=FAKE << 23, k=(FAKE << 23) + 1024, v=(FAKE << 23) + 1536,
         q_token_stride=1024, q_out_token_stride=1024, k_token_stride=1024,
         v_token_stride=1024),
    # pages of k's rows and v's, and of their scales
    dict(c=_c4(v=FAKE + 2048, k_page_stride=4096, v_page_stride=4096,
               v_blocks=(FAKE << 21) + 128, k_block_page_stride=256,
               v_block_page_stride=256)),
    # pages of rows and their scales
    dict(c=_c4(k_page_stride=4096, k_blocks=FAKE + 2048,
               k_block_page_stride=4096)),
    # keys that all tokens share
    dict(k_token_stride=0, v_head_stride=0),
], ids=str)
def test_extensions_that_are_taken(kw):
    """(Without a device a valid call ends at the device.)"""
    assert _extend(**kw) == ltk.ERR_HIP


@pytest.mark.parametrize("kw", [
    # the same, but the keys lie across the queries
    dict(k=(FAKE << 23) + 1008), dict(v=(FAKE << 23) + 2032),
    dict(k=(FAKE << 23) + 1024, k_token_stride=1032)], ids=str)
def test_queries_in_place_may_not_meet_keys(kw):
    t = dict(q_out=FAKE << 23, k=(FAKE << 23) + 1024, v=(FAKE << 23) + 1536,
             q_token_stride=1024, q_out_token_stride=1024,
             k_token_stride=1024, v_token_stride=1024)
    t.update(kw)
    assert _extend(**t) == ltk.ERR_INVALID


def test_no_sequences_is_a_no_op():
    none = _c4(batch=0, table=0, lens=0)
    assert host._attend(none, q=None, out=None, lse=None) == ltk.OK
    assert _extend(none, starts=None, lens=None) == ltk.OK
    assert _extend(none, starts=None, lens=None, rot=8) == ltk.ERR_INVALID
    assert _sample(rows=0, logits=None, u=None, tokens=None, logprobs=None) \
        == ltk.OK
    assert _sample(rows=0, cols=0) == ltk.ERR_INVALID


def _sample(logits=FAKE, dtype=ltk.F32, rows=4, cols=1000, ld=1000, how=0,
            u=FAKE << 12, tokens=FAKE << 13, logprobs=FAKE << 14, **kw):
    if how == 0:
        how = ltk.SamplingStruct(**dict(dict(temperature_all=1.0,
                                             top_p_all=1.0), **kw))
    return ltk.lib.sample_logits(logits, dtype, rows, cols, ld, how, u,
                                 tokens, logprobs, None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(u=None), dict(tokens=None), dict(logprobs=None),
    dict(how=None), dict(logits=FAKE + 2), dict(u=(FAKE << 12) + 2),
    dict(dtype=ltk.BF16, logits=FAKE + 1), dict(tokens=(FAKE << 13) + 4),
    dict(logprobs=(FAKE << 14) + 2), dict(dtype=ltk.E4M3),
    dict(dtype=ltk.E2M1), dict(dtype=-1), dict(rows=-1), dict(rows=1 << 22),
    dict(cols=0), dict(cols=-5), dict(cols=(1 << 24) + 1, ld=1 << 25),
    dict(ld=999), dict(ld=1 << 37), dict(temperature=FAKE + 2),
    dict(top_k=FAKE + 1), dict(top_p=FAKE + 3), dict(min_p=FAKE + 2),
    dict(tokens=FAKE), dict(tokens=FAKE + 15992), dict(logprobs=FAKE + 8),
    dict(logprobs=FAKE << 13), dict(logprobs=(FAKE << 13) + 28),
    dict(tokens=FAKE << 12), dict(logprobs=(FAKE << 12) + 12),
    dict(top_k=FAKE << 14), dict(min_p=(FAKE << 13) + 16),
], ids=str)
def test_sample_refuses(kw):
    assert _sample(**kw) == ltk.ERR_INVALID


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is visible")
def test_samplings_that_are_taken():
    for kw in (dict(), dict(dtype=ltk.BF16, logits=FAKE + 2),
               dict(dtype=ltk.F16), dict(ld=5000),
               dict(rows=1, tokens=FAKE + 4000), dict(tokens=FAKE + 16000),
               dict(cols=1 << 24, ld=1 << 24, logits=1 << 50),
               dict(top_k_all=-1, top_p_all=math.nan, min_p_all=-1.0),
               dict(temperature=FAKE << 15, top_k=FAKE << 15)):
        assert _sample(**kw) == ltk.ERR_HIP, kw


# ---------------------------------------------------------- what is launched
@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("stub") / "step_stub")
    pkg = os.path.dirname(ltk.LIBRARY_PATH)
    subprocess.check_call(
        ["g++", "-O1", "-std=c++17", "-pthread", "-rdynamic",
         "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
         "-I", HERE, "-isystem", "/opt/rocm/include",
         os.path.join(HERE, "step_stub.cpp"), ltk.LIBRARY_PATH, "-o", exe,
         "-Wl,-rpath," + pkg, "-Wl,-rpath-link,/opt/rocm/lib"])

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True,
                           text=True, timeout=120)
        assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
        words = r.stdout.split()
        return dict(zip(words[::2], map(int, words[1::2])))

    return run


def test_a_call_s_launches_stay_together(stub):
    r = stub("threads")
    assert r["failed"] == 0 and r["torn"] == 0
    assert r["calls"] == 36 and r["most"] >= 5


def test_launches_of_sampling(stub):
    """Two without settings, five with any; rows beyond a workspace of 64 MB
    (and its doubling, when it grows) go in batches; rows beyond 2^20 logits
    take one."""
    assert stub("sample", 4, 1000, 1)["launches"] == 2
    assert stub("sample", 4, 1000, 0.5)["launches"] == 5
    assert stub("sample", 4, 1 << 20, 0.5)["launches"] == 5
    r = stub("sample", 7, (1 << 20) + 1, 0.5)
    assert (r["launches"], r["groups"], r["bytes"]) == (1, 7, 0)
    for rows, cols in (((1 << 22) - 1, 1), ((1 << 22) - 1, 5000),
                       (70000, 262144), (3, 1 << 20)):
        r = stub("sample", rows, cols, 0.5)
        assert r["rc"] == 0 and r["launches"] % 5 == 0, (rows, cols, r)
        assert r["wide"] == 0 and r["bytes"] <= (1 << 26) + (1 << 17), r
    r = stub("sample", (1 << 22) - 1, 1 << 24, 0.5)
    assert r["rc"] == 0 and r["launches"] == 1 and r["wide"] == 0


def test_launches_of_extension(stub):
    """One: with few tokens a wave a row or so, with many a wave a token; for
    no token too, since the lengths are written."""
    for batch, tokens, q_heads, heads in ((1, 1, 32, 8), (1, 0, 8, 8),
                                          (5000, 0, 1, 1), (64, 64, 32, 8),
                                          (3, 100000, 32, 8)):
        r = stub("extend", batch, tokens, q_heads, heads)
        assert r["rc"] == 0 and r["launches"] == 1, r
        assert r["groups"] * 4 >= tokens and r["groups"] * 256 >= batch
        assert r["groups"] <= max(4096, (tokens + 3) // 4), r
    assert stub("extend", 1, 1 << 27, 1, 1)["rc"] == ltk.ERR_INVALID


def test_structs_match_the_header(tmp_path):
    src, exe = str(tmp_path / "sizes.cpp"), str(tmp_path / "sizes")
    names = {"libtopk_cache_t": ltk.CacheStruct,
             "libtopk_tokens_t": ltk.TokensStruct,
             "libtopk_sampling_t": ltk.SamplingStruct,
             "libtopk_ledger_t": ltk.LedgerStruct}
    lines = []
    for c, py in names.items():
        lines.append('printf("%%zu\\n", sizeof(%s));' % c)
        for f, _ in py._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (c, f))
    with open(src, "w") as f:
        f.write('#include <stddef.h>\n#include <stdio.h>\n#include "libtopk.h"'
                "\nint main() {\n" + "\n".join(lines) + "\n}\n")
    subprocess.check_call(["g++", "-I", os.path.join(ROOT, "include"), src,
                           "-o", exe])
    got = list(map(int, subprocess.check_output([exe]).split()))
    want = []
    for py in names.values():
        want.append(ctypes.sizeof(py))
        want += [getattr(py, f).offset for f, _ in py._fields_]
    assert got == want


# ------------------------------------------------------ refusals, binding
BF, F4, E8 = torch.bfloat16, torch.float4_e2m1fn_x2, torch.float8_e8m0fnu


def _codes(*size):
    return torch.zeros(size, dtype=torch.uint8).view(F4)


def _blocks(*size):
    return torch.zeros(size, dtype=torch.uint8).view(E8)


def _t(**kw):
    d = dict(q=torch.zeros(5, 8, 64, dtype=BF), k_new=torch.zeros(
                 5, 4, 64, dtype=BF), v_new=torch.zeros(5, 4, 64, dtype=BF),
             k=_codes(32, 4, 16, 32), v=_codes(32, 4, 16, 32),
             k_blocks=_blocks(32, 4, 16, 2),
             v_blocks=_blocks(32, 4, 16, 2),
             table=torch.zeros(2, 4, dtype=torch.int32),
             lens=torch.zeros(2, dtype=torch.int32),
             starts=torch.zeros(3, dtype=torch.int32),
             weights=torch.zeros(2, 4, 64),
             positions=torch.zeros(2, 4, 64, dtype=torch.int32))
    d.update(kw)
    return d


def _call(**kw):
    return ltk.cache_extend(**_t(**kw))


def _calls4(d):
    yield lambda: ltk.cache_extend(**d)
    yield lambda: ltk.cache_attend(
        torch.zeros(2, 8, 64, dtype=BF), d["k"], d["v"], d["table"],
        d["lens"], k_blocks=d["k_blocks"], v_blocks=d["v_blocks"])
    yield lambda: ltk.cache_evict(
        d["k"], d["v"], d["table"], d["lens"],
        torch.zeros(2, dtype=torch.int32), d["weights"], d["positions"], 32,
        k_blocks=d["k_blocks"], v_blocks=d["v_blocks"])


def test_binding_wants_device_tensors():
    for call in _calls4(_t()):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(ValueError, match="device"):
        ltk.sample(torch.zeros(2, 9), torch.zeros(2))


@pytest.mark.parametrize("kw,error", [
    (dict(k_blocks=None), ValueError),
    (dict(v_blocks=None), ValueError),
    (dict(k_blocks=torch.zeros(32, 4, 16, 2)), TypeError),
    (dict(v_blocks=_blocks(32, 4, 16, 3)), ValueError),
    (dict(v_blocks=_blocks(32, 16, 4, 2)), ValueError),
    (dict(k_blocks=_blocks(32, 4, 2, 16).transpose(2, 3)), ValueError),
    (dict(k_blocks=torch.zeros(32, 4, 16, 2, dtype=torch.uint8)), TypeError),
    (dict(k=_codes(32, 4, 16, 24), v=_codes(32, 4, 16, 24)), ValueError),
    (dict(k=torch.zeros(32, 4, 16, 64, dtype=BF),
          v=torch.zeros(32, 4, 16, 64, dtype=BF)), ValueError),
    (dict(v=torch.zeros(32, 4, 16, 32, dtype=torch.uint8)), TypeError),
    (dict(k=torch.zeros(32, 4, 16, 32, dtype=torch.uint8)), TypeError),
], ids=lambda x: str(x)[:60])
def test_binding_refuses_4_bit_caches(kw, error):
    for call in _calls4(_t(**kw)):
        with pytest.raises(error):
            call()


def test_append_binding_refuses_4_bit_caches():
    d = _t()
    with pytest.raises((TypeError, ValueError)):
        ltk.cache_append(d["k_new"][:2], d["v_new"][:2], d["k"], d["v"],
                         d["table"], d["lens"], 32,
                         torch.zeros(2, dtype=torch.int32), d["weights"],
                         d["positions"])


@pytest.mark.parametrize("kw,error", [
    (dict(k_new=np.zeros((5, 4, 64))), TypeError),
    (dict(k_new=torch.zeros(5, 4, 64)), TypeError),
    (dict(v_new=torch.zeros(5, 4, 64, dtype=torch.float16)), TypeError),
    (dict(v_new=torch.zeros(4, 4, 64, dtype=BF)), ValueError),
    (dict(k_new=torch.zeros(5, 64, dtype=BF)), ValueError),
    (dict(k_new=torch.zeros(5, 3, 64, dtype=BF)), ValueError),
    (dict(k_new=torch.zeros(5, 64, 4, dtype=BF).transpose(1, 2)), ValueError),
    (dict(q=torch.zeros(5, 8, 32, dtype=BF)), ValueError),
    (dict(q=torch.zeros(5, 0, 64, dtype=BF)), ValueError),
    (dict(q=torch.zeros(5, 512, dtype=BF)), ValueError),
    (dict(q=torch.zeros(5, 8, 64)), TypeError),
    (dict(starts=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(starts=torch.zeros(3, dtype=torch.int64)), TypeError),
    (dict(starts=torch.zeros(6, dtype=torch.int32)[::2]), ValueError),
    (dict(seen=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(freqs=torch.zeros(33)), ValueError),
    (dict(freqs=torch.zeros(40)), ValueError),
    (dict(freqs=torch.zeros(4)), ValueError),
    (dict(freqs=torch.zeros(16, dtype=torch.float64)), TypeError),
    (dict(freqs=torch.zeros(2, 16)), ValueError),
    (dict(k_norm=torch.zeros(32, dtype=BF)), ValueError),
    (dict(q_norm=torch.zeros(64, dtype=torch.float16)), TypeError),
    (dict(k_norm=torch.zeros(64), q_norm=torch.zeros(64, dtype=BF)),
     TypeError),
    (dict(eps=-1.0), ValueError), (dict(eps=math.nan), ValueError),
    (dict(eps="x"), TypeError),
    (dict(k_scale=torch.zeros(3)), ValueError),
    (dict(v_scale=torch.zeros(4, dtype=BF)), TypeError),
    (dict(weights=None), ValueError), (dict(positions=None), ValueError),
    (dict(weights=torch.zeros(2, 3, 64)), ValueError),
    (dict(lens=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(k=torch.zeros(32, 4, 16, 64, dtype=torch.float16),
          v=torch.zeros(32, 4, 16, 64, dtype=torch.float16), k_blocks=None,
          v_blocks=None), TypeError),
], ids=lambda x: str(x)[:60])
def test_extend_binding_refuses(kw, error):
    with pytest.raises(error):
        _call(**kw)


@pytest.mark.parametrize("kw,error", [
    (dict(logits=np.zeros((2, 9))), TypeError),
    (dict(logits=torch.zeros(2, 9, dtype=torch.float64)), TypeError),
    (dict(logits=torch.zeros(9)), ValueError),
    (dict(logits=torch.zeros(2, 0)), ValueError),
    (dict(logits=torch.zeros(9, 2).t()), ValueError),
    (dict(logits=torch.zeros(1, 9).expand(2, 9)), ValueError),
    (dict(u=torch.zeros(3)), ValueError),
    (dict(u=torch.zeros(2, dtype=torch.float64)), TypeError),
    (dict(u=0.5), TypeError),
    (dict(temperature=-1.0), ValueError), (dict(top_p=math.nan), ValueError),
    (dict(min_p=-0.1), ValueError), (dict(top_k=-1), ValueError),
    (dict(top_k=1.5), TypeError), (dict(top_k=2 ** 31), ValueError),
    (dict(temperature="hot"), TypeError),
    (dict(temperature=torch.zeros(3)), ValueError),
    (dict(top_k=torch.zeros(2, dtype=torch.int64)), TypeError),
    (dict(top_p=torch.zeros(2, dtype=BF)), TypeError),
    (dict(min_p=torch.zeros(4)[::2]), ValueError),
    (dict(out=torch.zeros(2)), TypeError),
], ids=lambda x: str(x)[:60])
def test_sample_binding_refuses(kw, error):
    d = dict(logits=torch.zeros(2, 9), u=torch.zeros(2))
    d.update(kw)
    with pytest.raises(error):
        ltk.sample(**d)
