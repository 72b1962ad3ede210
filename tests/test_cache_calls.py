"""What the cache_* entry points do on the host: a program of its own with
HIP's calls answered by a stub (hip_stub.cpp), so that no GPU is needed and
every launch is seen."""
import os
import subprocess

import pytest

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
