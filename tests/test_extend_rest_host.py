"""cache_extend's queries of tokens that belong to no sequence: what the C
entry point checks, on the CPU."""
import os

import pytest

import test_step_host as host
import top_selection_two_amd as ltk


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="a GPU is visible")
def test_queries_of_no_sequence_are_a_launch_of_their_own():
    """(Without a device a valid call ends at the device, a no-op before.)"""
    none = host._c4(batch=0, table=0, lens=0)
    assert host._extend(none, starts=None, lens=None) == ltk.OK
    assert host._extend(none, starts=None, lens=None, rest=1) == ltk.ERR_HIP
    assert host._extend(none, starts=None, lens=None, rest=1, tokens=0) == \
        ltk.OK
    assert host._extend(none, starts=None, lens=None, rest=1, q=None) == \
        ltk.OK
    assert host._extend(rest=1) == ltk.ERR_HIP


def test_they_are_checked_without_sequences_too():
    none = host._c4(batch=0, table=0, lens=0)
    for kw in (dict(q_out=None), dict(q_out=(host.FAKE << 23) + 64),
               dict(q_out=host.FAKE << 24), dict(k=None)):
        assert host._extend(none, starts=None, lens=None, rest=1, **kw) == \
            ltk.ERR_INVALID, kw
    assert host._extend(rest=1, starts=None) == ltk.ERR_INVALID
    assert host._extend(rest=1, lens=None) == ltk.ERR_INVALID
