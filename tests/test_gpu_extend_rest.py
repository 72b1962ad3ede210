"""cache_extend's queries of tokens that belong to no sequence, on the GPU: in
a tensor that the call makes they are those given, bit for bit; in one that is
given they are left alone."""
import numpy as np
import pytest
import torch

import test_gpu_extend as ext
import top_selection_two_amd as ltk

pytestmark = pytest.mark.gpu


def _call(q, k, v, dev, starts, **kw):
    return ltk.cache_extend(
        k, v, dev["k"], dev["v"], dev["table"], dev["lens"],
        torch.tensor(starts, dtype=torch.int32).cuda(), q=q,
        k_blocks=dev.get("k_blocks"), v_blocks=dev.get("v_blocks"), **kw)


def _made(shape, dtype):
    """Memory of that size which the allocator hands out next holds NaN."""
    x = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("ctype,dim,rot,interleaved", [
    ("bf16", 64, 64, False), ("bf16", 80, 32, True), ("e4m3", 128, 0, False),
    ("e2m1", 256, 64, False), ("bf16", 24, 16, False)])
@pytest.mark.parametrize("q_heads", [1, 3, 32])
def test_rows_of_no_sequence(ctype, dim, rot, interleaved, q_heads):
    print("rest", ctype, dim, rot, q_heads, flush=True)
    rng = np.random.default_rng(dim)
    for n, starts in ((40, [0, 10, 10, 23]), (9, [4, 5, 5, 9]),
                      (700, [3, 3, 3, 3]), (2, [0, 0, 0, 1]),
                      (5000, [1000, 1500, 1600, 4000])):
        q, k, v = ext._new(rng, [n], q_heads, 2, dim, "bf16")
        q[n - 1, 0, 1] = float("nan")
        lens = [0, 5, 1]
        counts = [b - a for a, b in zip(starts, starts[1:])]
        dev, _ = ext._blank(rng, lens, counts, 2, dim, 16, ctype)
        f = torch.linspace(1, .01, rot // 2).cuda() if rot else None
        how = dict(freqs=f, interleaved=interleaved,
                   q_norm=torch.full((dim,), 1.5).cuda())
        given = torch.full((n, q_heads, dim), 7.0, dtype=q.dtype).cuda()
        _made(q.shape, q.dtype)
        _, made = _call(q, k, v, dev, starts, **how)
        got_lens, given = _call(q, k, v, dev, starts, out=given, **how)
        torch.cuda.synchronize()
        idle = np.ones(n, bool)
        idle[starts[0]:starts[-1]] = False
        idle = torch.from_numpy(idle).cuda()
        assert torch.equal(made[idle].view(torch.int16),
                           q[idle].contiguous().view(torch.int16))
        assert (given[idle] == 7.0).all()
        assert torch.equal(made[~idle].view(torch.int16),
                           given[~idle].view(torch.int16))
        assert got_lens.tolist() == [a + b for a, b in zip(lens, counts)]


def test_no_sequence_at_all():
    rng = np.random.default_rng(1)
    q, k, v = ext._new(rng, [30], 4, 2, 64, "f16")
    dev, _ = ext._blank(rng, [0], [30], 2, 64, 16, "f16")
    dev["table"], dev["lens"] = dev["table"][:0], dev["lens"][:0]
    before = ext._raw(dev["k"])
    _made(q.shape, q.dtype)
    lens, made = _call(q, k, v, dev, [0])
    assert lens.shape == (0,) and torch.equal(made, q)
    assert np.array_equal(ext._raw(dev["k"]), before)
    out = torch.full_like(made, 7.0)
    _call(q, k, v, dev, [0], out=out)
    assert (out == 7.0).all()


def test_one_token_in_place_in_its_projection():
    """A token's queries turned where they lie, between nothing and its keys
    and values, in one array."""
    rng = np.random.default_rng(2)
    for heads in (1, 2, 8):
        q, k, v = ext._new(rng, [1], 4, heads, 64, "bf16")
        assert q.data_ptr() + 4 * 64 * 2 == k.data_ptr()
        dev, _ = ext._blank(rng, [0], [1], heads, 64, 16, "bf16")
        f = torch.linspace(1, 0.01, 32).cuda()
        how = dict(freqs=f, q_norm=f.repeat(2), k_norm=f.repeat(2),
                   seen=torch.tensor([77], dtype=torch.int32).cuda())
        _, want = _call(q, k, v, dev, [0, 1], **how)
        rows, keep = ext._raw(dev["k"]), (k.clone(), v.clone())
        _, got = _call(q, k, v, dev, [0, 1], out=q, **how)
        assert got is q and torch.equal(q, want)
        assert torch.equal(k, keep[0]) and torch.equal(v, keep[1])
        assert np.array_equal(ext._raw(dev["k"]), rows)
