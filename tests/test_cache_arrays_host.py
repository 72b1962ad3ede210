"""The calls that write to a cache refuse arrays of it that share bytes, and
take those that interleave: k, v and the scales of 4-bit rows.  On the CPU,
where a call that is taken ends at the missing device."""
import os

import numpy as np
import pytest

import test_cache_host as base
import test_step_host as step
import top_selection_two_amd as ltk

FAKE = base.FAKE
pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                                reason="a GPU is visible")


def _all(c, four):
    """Statuses of extension, eviction, and append (of 16-bit rows)."""
    r = [step._extend(c), base._evict(c)]
    return r if four else r + [base._append(c)]


ROW, PAGE = 64 * 2, 4 * 16 * 64 * 2  # bytes


@pytest.mark.parametrize("kw", [
    dict(v=FAKE + 16), dict(v=FAKE + ROW), dict(v=FAKE + PAGE),
    dict(v=FAKE + 31 * PAGE), dict(v=FAKE + 32 * PAGE - 16),
    dict(v=FAKE - 16), dict(v=FAKE - PAGE),
    # one page of both, the second an element late
    dict(k_page_stride=PAGE, v_page_stride=PAGE, v=FAKE + PAGE - 16),
    # strides that differ where the extents meet
    dict(k_page_stride=PAGE, v_page_stride=2 * PAGE, v=FAKE + PAGE),
    dict(v=FAKE + ROW, k_slot_stride=256, v_slot_stride=128,
         k_head_stride=16 * 256, v_head_stride=16 * 256,
         k_page_stride=64 * 256, v_page_stride=64 * 256),
    dict(v=FAKE, v_head_stride=64, v_slot_stride=256),
], ids=str)
def test_shared_rows_are_refused(kw):
    c = base._c(**kw)
    assert _all(c, False) == [ltk.ERR_INVALID] * 3


@pytest.mark.parametrize("kw", [
    dict(v=FAKE + 32 * PAGE), dict(v=FAKE - 32 * PAGE),
    # pages, heads, slots of both in turn
    dict(k_page_stride=PAGE, v_page_stride=PAGE, v=FAKE + PAGE),
    dict(k_head_stride=2048, v_head_stride=2048, k_page_stride=8192,
         v_page_stride=8192, v=FAKE + 2048),
    dict(k_slot_stride=128, v_slot_stride=128, k_head_stride=2048,
         v_head_stride=2048, k_page_stride=8192, v_page_stride=8192,
         v=FAKE + ROW),
    dict(k_slot_stride=128, v_slot_stride=128, k_head_stride=2048,
         v_head_stride=2048, k_page_stride=8192, v_page_stride=8192,
         v=FAKE - ROW),
    # v's pages between k's, in the other order within a page
    dict(k_page_stride=PAGE, v_page_stride=PAGE, v=FAKE - PAGE,
         v_head_stride=64, v_slot_stride=256),
    # v two pages on
    dict(k_page_stride=PAGE, v_page_stride=PAGE, v=FAKE + 5 * PAGE),
], ids=str)
def test_interleaved_rows_are_taken(kw):
    c = base._c(**kw)
    assert _all(c, False) == [ltk.ERR_HIP] * 3


@pytest.mark.parametrize("kw", [
    dict(v_blocks=FAKE << 21), dict(v_blocks=(FAKE << 21) + 1),
    dict(v_blocks=(FAKE << 21) + 128), dict(k_blocks=FAKE + 40),
    dict(v_blocks=FAKE + 2048), dict(v=FAKE), dict(v=FAKE + 16),
    dict(k_blocks=(FAKE << 12) + 512), dict(v_blocks=(FAKE << 12) + 2047),
    # rows and scales in one slot, one byte too near
    dict(k_slot_stride=64, k_head_stride=1024, k_page_stride=4096,
         k_blocks=FAKE + 31, k_block_slot_stride=64, k_block_head_stride=1024,
         k_block_page_stride=4096),
    dict(k_slot_stride=64, k_head_stride=1024, k_page_stride=4096,
         k_blocks=FAKE + 63, k_block_slot_stride=64, k_block_head_stride=1024,
         k_block_page_stride=4096),
], ids=str)
def test_shared_scales_are_refused(kw):
    c = step._c4(**kw)
    assert _all(c, True) == [ltk.ERR_INVALID] * 2


@pytest.mark.parametrize("kw", [
    # rows and scales in one slot
    dict(k_slot_stride=64, k_head_stride=1024, k_page_stride=4096,
         k_blocks=FAKE + 32, k_block_slot_stride=64, k_block_head_stride=1024,
         k_block_page_stride=4096),
    dict(k_slot_stride=64, k_head_stride=1024, k_page_stride=4096,
         k_blocks=FAKE + 62, k_block_slot_stride=64, k_block_head_stride=1024,
         k_block_page_stride=4096),
    # all four in one page
    dict(k_page_stride=4352, v_page_stride=4352, k_block_page_stride=4352,
         v_block_page_stride=4352, v=FAKE + 2048, k_blocks=FAKE + 4096,
         v_blocks=FAKE + 4224),
    # both rows' scales in turn
    dict(k_block_slot_stride=4, v_block_slot_stride=4, k_block_head_stride=64,
         v_block_head_stride=64, k_block_page_stride=256,
         v_block_page_stride=256, v_blocks=(FAKE << 21) + 2),
], ids=str)
def test_interleaved_scales_are_taken(kw):
    c = step._c4(**kw)
    assert _all(c, True) == [ltk.ERR_HIP] * 2


def test_one_array_for_keys_and_values():
    """Moved rows are the same in both; new ones if they are one array."""
    c = base._c(v=FAKE)
    assert base._evict(c) == ltk.ERR_HIP
    assert base._append(c) == ltk.ERR_INVALID
    assert base._append(c, vn=FAKE << 16) == ltk.ERR_HIP
    assert step._extend(c) == ltk.ERR_INVALID
    c = step._c4(v=FAKE, v_blocks=FAKE << 21)
    assert base._evict(c) == ltk.ERR_HIP
    assert step._extend(c) == ltk.ERR_INVALID
    assert base._evict(step._c4(v=FAKE)) == ltk.ERR_INVALID
    assert base._evict(base._c(v=FAKE, v_page_stride=PAGE)) == ltk.ERR_INVALID
    assert base._evict(base._c(v=FAKE, v_page_stride=PAGE, pages=1)) == \
        ltk.ERR_HIP


def _bytes_of(n, strides, row, at):
    i = [np.arange(m) * s for m, s in zip(n, strides)]
    x = at + i[0][:, None, None] + i[1][:, None] + i[2]
    return {int(b) + e for b in x.ravel() for e in range(row)}


@pytest.mark.parametrize("seed", range(12))
def test_sharing_by_brute_force(seed):
    """Scales anywhere around rows of 32 bytes: taken exactly where no byte is
    shared, if the strides are the same; never taken where one is."""
    rng = np.random.default_rng(seed)
    met = taken = 0
    for _ in range(150):
        n = [int(rng.integers(1, 5)) for _ in range(3)]
        order = rng.permutation(3)
        s, span = [0, 0, 0], 32
        for axis in order:
            s[axis] = -(-span // 16) * 16 + 16 * int(rng.integers(0, 4))
            span = (n[axis] - 1) * s[axis] + span
        same = rng.random() < 0.7
        t = list(s)
        if not same:
            span_t = 2
            for axis in rng.permutation(3):
                t[axis] = span_t + int(rng.integers(0, 40))
                span_t = (n[axis] - 1) * t[axis] + span_t
        d = int(rng.integers(-span - 8, span + 8))
        at = FAKE << 6
        c = step._c4(k=at, k_page_stride=s[0], k_head_stride=s[1],
                     k_slot_stride=s[2], k_blocks=at + d,
                     k_block_page_stride=t[0], k_block_head_stride=t[1],
                     k_block_slot_stride=t[2], pages=n[0], heads=n[1],
                     page=n[2])
        share = bool(_bytes_of(n, s, 32, 0) & _bytes_of(n, t, 2, d))
        rc = step._extend(c)
        if share:
            assert rc == ltk.ERR_INVALID, (n, s, t, d)
            met += 1
        elif same:
            assert rc == ltk.ERR_HIP, (n, s, t, d)
            taken += 1
    assert met > 10 and taken > 10
