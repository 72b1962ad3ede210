"""What the cache_* entry points do on the host: a program of its own with
HIP's calls answered by a stub (hip_stub.cpp), so that no GPU is needed and
every launch is seen."""
import ctypes
import os
import subprocess

import pytest

import test_cache_host as host
import top_selection_two_amd as ltk

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("stub") / "hip_stub")
    pkg = os.path.dirname(ltk.LIBRARY_PATH)
    subprocess.check_call(
        ["g++", "-O1", "-std=c++17", "-pthread", "-rdynamic",
         "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
         "-isystem", "/opt/rocm/include", os.path.join(HERE, "hip_stub.cpp"),
         ltk.LIBRARY_PATH, "-o", exe, "-Wl,-rpath," + pkg,
         "-Wl,-rpath-link,/opt/rocm/lib"])

    def run(*args):
        r = subprocess.run([exe, *args], capture_output=True, text=True,
                           timeout=120)
        assert r.returncode == 0, (r.returncode, r.stderr[-2000:])
        words = r.stdout.split()
        return dict(zip(words[::2], map(int, words[1::2])))

    return run


def test_a_call_s_launches_stay_together(stub):
    """Calls of several launches on one stream, from several threads: none
    comes between another's, whose workspace it would overwrite."""
    r = stub("threads")
    assert r["failed"] == 0 and r["torn"] == 0
    assert r["calls"] == 36 and r["most"] >= 7


def test_selections_of_several_launches_stay_together(stub):
    """The same for top-k above 128 and of segments, with a histogram, which
    counts in the same words, between them."""
    r = stub("selection_threads")
    assert r["failed"] == 0 and r["torn"] == 0
    assert r["calls"] == 48 and r["most"] >= 6


# 4 heads of 16 slots of 64 elements (k and v have 32 pages)
@pytest.mark.parametrize("strides", [
    (4096, 0, 64), (4096, 1024, 0), (0, 1024, 64), (2048, 1024, 64),
    (4096, 1024, 32), (4096, 512, 64), (4096, 8, 64), (4096 - 64, 1024, 64),
    (64, 64 * 32, 64 * 32)], ids=str)
@pytest.mark.parametrize("name", ["k", "v"])
def test_append_and_evict_refuse_rows_that_overlap(name, strides):
    kw = {name + "_%s_stride" % a: x
          for a, x in zip(("page", "head", "slot"), strides)}
    assert host._append(host._c(**kw)) == ltk.ERR_INVALID
    assert host._evict(host._c(**kw)) == ltk.ERR_INVALID


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is visible")
@pytest.mark.parametrize("kw", [
    # slots outside heads, and with padding
    dict(k_head_stride=64, k_slot_stride=256),
    dict(k_head_stride=72, k_slot_stride=296, k_page_stride=8192),
    # pages inside heads
    dict(k_page_stride=1024, k_head_stride=32 * 1024),
    # an axis of one does not step at all
    dict(heads=1, k_head_stride=0, v_head_stride=0),
    dict(page=1, k_slot_stride=0, v_slot_stride=8),
    dict(pages=1, k_page_stride=0, v_page_stride=0)], ids=str)
def test_rows_that_lie_apart_are_taken(kw):
    """(Without a device a valid call ends at the device.)"""
    assert host._append(host._c(**kw)) == ltk.ERR_HIP
    assert host._evict(host._c(**kw)) == ltk.ERR_HIP


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is visible")
def test_attend_reads_rows_that_overlap():
    assert host._attend(host._c(k_head_stride=0, v_head_stride=0,
                                v_page_stride=0)) == ltk.ERR_HIP


def test_launches_of_too_many_threads_are_refused(stub):
    """2^32 threads or more along an axis cannot be launched: such calls are
    refused before anything is."""
    for batch, heads, width, append, evict in (
            (1 << 12, 1 << 10, 1, 0, 1),          # 2^22 rows
            ((1 << 22) - 1, 1, 1, 0, 0),
            (1 << 14, 1 << 10, 1, 1, 1),          # 2^24 rows
            ((1 << 24) - 1, 1, 1, 0, 1),
            (1 << 19, 1, 2048, 0, 1),             # of 8 chunks each
            ((1 << 19) - 1, 1, 2048, 0, 0)):
        r = stub("rows", str(batch), str(heads), str(width))
        assert (r["append"], r["evict"]) == (append, evict), (batch, r)
        assert r["append_wide"] == r["evict_wide"] == 0, (batch, r)
        for name in ("append", "evict"):
            assert (r[name + "_launches"] == 0) == (r[name] != 0), (batch, r)


@pytest.mark.parametrize("fit", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("dim,cols,waves", [
    (64, 64, 8), (96, 128, 8), (128, 128, 8), (192, 256, 4), (256, 256, 4)])
def test_attention_has_room_for_scores(stub, dim, cols, waves, fit):
    """However many workgroups the device would hold at once, each gets room
    for the waves' results of 16 queries and the scores of a tile at least (of
    32 slots, and of 4 heads where slots lie outside heads): with none the
    kernel would not advance."""
    for slots_first in (0, 1):
        r = stub("lds", str(dim), str(slots_first), str(fit))
        tile = 32 * 16 * 4 * (4 if slots_first else 1)
        assert r["rc"] == 0 and r["threads"] == 64 * waves
        join = waves * 16 * cols * 4
        assert join + tile <= r["lds"] <= 160 * 1024, (slots_first, r)


def test_shares_lie_in_whole_vectors(tmp_path):
    """Results of shares follow one another in units of 16 bytes, in which
    they are read, also those of an odd number of queries."""
    src, so = str(tmp_path / "share.cpp"), str(tmp_path / "share.so")
    with open(src, "w") as f:
        f.write('#include "cache_layout.hpp"\nextern "C" int floats(int rows, '
                'int cols) { return ltk::share_floats(rows, cols); }\n')
    subprocess.check_call(["g++", "-std=c++17", "-shared", "-fPIC", "-I",
                           host.CSRC, src, "-o", so])
    floats = ctypes.CDLL(so).floats
    for cols in (64, 128, 256):
        for rows in range(1, 65):
            need = rows * (cols + 2)
            assert floats(rows, cols) % 4 == 0
            assert need <= floats(rows, cols) < need + 4
