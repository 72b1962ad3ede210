"""Paths of the paged-cache operators that the sizes of test_gpu_cache.py leave
out, against the same oracle and with its bounds."""
import pytest
import torch

import test_gpu_cache as t
import top_selection_two_amd as ltk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,n,dim", [(1, 40000, 64), (3, 12000, 128),
                                         (5, 9000, 256), (15, 4001, 64)])
def test_attend_long_rows_of_odd_groups(group, n, dim):
    """Joined by the second launch, from shares of an odd number of queries."""
    rng, dev, ref = t._case(group, [n, n // 3], 1, dim, 16, "bf16")
    print("attend odd group", group, n, dim, flush=True)
    t._attend(dev, t._q(rng, 2, group, dim, "bf16"), ref, "bf16", "bf16",
              rng=rng)


@pytest.mark.parametrize("lens,keep,extra", [
    ([2000, 0, 1, 1024], 2000, 80), ([500, 20000, 3000, 4096], 4096, 1),
    ([100, 90], 64, 80)])
@pytest.mark.parametrize("kind", ["plain", "special"])
def test_evict_short_rows_in_a_wide_table(lens, keep, extra, kind):
    """Rows of at most `keep` slots, and short rows that are cut, where the
    table can name more slots than one workgroup selects from."""
    print("evict in a wide table", lens, keep, kind, flush=True)
    t._check_evict(lens, 2, 8, 256, keep, 4, 20, kind, extra=extra)


# ---------------------------------------------------------------- autograd
def _state(seed=31):
    rng, dev, ref = t._case(seed, [100, 40], 2, 64, 16, "bf16")
    n = dev["table"].shape[1] * 16
    w, pos = t._ledger(rng, 2, 2, n, "plain")
    dev["w"] = torch.from_numpy(w).cuda()
    dev["pos"] = torch.from_numpy(pos).cuda()
    dev["q"] = t._q(rng, 2, 4, 64, "bf16")
    dev["seen"] = dev["lens"].clone()
    return dev


@pytest.mark.parametrize("name", ["q", "k", "v", "w"])
def test_attend_says_that_it_has_no_backward(name):
    s = _state()
    want = ltk.cache_attend(s["q"], s["k"], s["v"], s["table"], s["lens"])
    assert not want[0].requires_grad and not want[1].requires_grad
    s[name].requires_grad_(True)
    got = ltk.cache_attend(s["q"], s["k"], s["v"], s["table"], s["lens"],
                           weights=s["w"])
    for a, b in zip(got, want):
        assert torch.equal(a, b) and a.requires_grad
        with pytest.raises(RuntimeError, match="not implemented"):
            a.float().sum().backward()
    assert s[name].grad is None
    with torch.no_grad():
        got = ltk.cache_attend(s["q"], s["k"], s["v"], s["table"], s["lens"])
    assert not got[0].requires_grad and torch.equal(got[0], want[0])


def test_calls_count_as_changes_in_place():
    def versions():
        return [s[n]._version for n in ("q", "k", "v", "w", "pos", "table",
                                        "lens", "seen")]

    def changed(call):
        a = versions()
        call()
        return [x != y for x, y in zip(a, versions())]

    s = _state()
    args = s["k"], s["v"], s["table"], s["lens"]
    assert not any(changed(lambda: ltk.cache_attend(s["q"], *args)))
    assert changed(lambda: ltk.cache_attend(s["q"], *args, weights=s["w"])) \
        == [False] * 3 + [True] + [False] * 4
    new = s["q"][:, :2].contiguous()
    assert changed(lambda: ltk.cache_append(
        new, new, *args, 60, s["seen"], s["w"], s["pos"])) \
        == [False] + [True] * 4 + [False] * 3
    out = torch.empty(2, 2, 30).cuda(), \
        torch.empty(2, 2, 30, dtype=torch.int32).cuda()
    was = [x._version for x in out]
    assert changed(lambda: ltk.cache_evict(
        *args, s["seen"], s["w"], s["pos"], 30, out=out)) \
        == [False] + [True] * 2 + [False] * 5
    assert [x._version > y for x, y in zip(out, was)] == [True, True]
    pair = torch.empty_like(s["q"]), torch.empty(2, 4).cuda()
    was = [x._version for x in pair]
    ltk.cache_attend(s["q"], *args, out=pair)
    assert [x._version > y for x, y in zip(pair, was)] == [True, True]
    # a gradient that needs what a call has overwritten is refused
    x = torch.ones(2, 2, s["w"].shape[2], device="cuda", requires_grad=True)
    y = (x * s["w"]).sum()
    ltk.cache_attend(s["q"], *args, weights=s["w"])
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()


def test_inference_tensors_are_taken_anywhere():
    with torch.inference_mode():
        s = _state()
    args = s["k"], s["v"], s["table"], s["lens"]
    a = ltk.cache_attend(s["q"], *args, weights=s["w"])
    with torch.inference_mode():
        b = ltk.cache_attend(s["q"], *args, weights=s["w"])
    assert torch.equal(a[0], b[0])
