"""sample() on the GPU against the float64 oracle.

Tokens have to be equal: weights are added in units of 2^-38 of the largest or
finer and taken to 2^-46, so that a token can only differ where u times the
sum lies within some 2^-38 of it of a border, which no case here does (the
random numbers are multiples of 2^-24, the borders none).  Where weights are
equal and borders are met exactly, both sides' sums are exact.  A log
probability is computed in 64 bits and rounded to float32: 2^-24 of it, and
2^-36 for the sums.
"""
import numpy as np
import pytest
import torch

import oracle.step as st
import top_selection_two_amd as ltk

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _check(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, got=None):
    """x: a device tensor of logits; settings: numbers or numpy arrays."""
    rows = x.shape[0]
    how = {"temperature": temperature, "top_k": top_k, "top_p": top_p,
           "min_p": min_p}
    u = np.asarray(u, np.float32)
    dev = {n: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v
           for n, v in how.items()}
    if got is None:
        got = ltk.sample(x, torch.from_numpy(u).cuda(), **dev)
        torch.cuda.synchronize()
    tokens, logprobs = got[0].cpu().numpy(), got[1].double().cpu().numpy()
    host = x.double().cpu().numpy()
    for r in range(rows):
        s = {n: v[r] if isinstance(v, np.ndarray) else v
             for n, v in how.items()}
        token, lp = st.sample(host[r].tolist(), u[r], **s)
        assert tokens[r] == token, (r, s, u[r], int(tokens[r]), token)
        if np.isinf(lp):
            assert logprobs[r] == lp
        else:
            tol = 2.0 ** -24 * abs(lp) + 2.0 ** -36
            assert abs(logprobs[r] - lp) <= tol, (r, logprobs[r], lp)
    return got


def _logits(rng, rows, cols, dtype, peak=1.5, pad=0, shift=0):
    """Logits that fall with the logarithm of a random rank."""
    x = -peak * np.log(rng.random((rows, cols)) * cols + 1.0)
    x += 0.3 * rng.standard_normal((rows, cols)) + 8
    full = torch.full((rows, shift + cols + pad), 50.0, dtype=TYPES[dtype])
    full[:, shift:shift + cols] = torch.from_numpy(x)
    return full.cuda()[:, shift:shift + cols]


SETTINGS = [dict(), dict(temperature=0.7), dict(temperature=1.7),
            dict(top_k=1), dict(top_k=5), dict(top_k=50, temperature=0.8),
            dict(top_k=700), dict(top_p=0.9), dict(top_p=0.5, temperature=2.0),
            dict(top_p=0.999), dict(min_p=0.05), dict(min_p=1.0),
            dict(top_k=40, top_p=0.9), dict(top_k=900, top_p=0.97),
            dict(top_p=0.95, min_p=0.02), dict(temperature=0.0),
            dict(top_k=30, top_p=0.8, min_p=0.1, temperature=0.6),
            dict(top_p=0.0), dict(min_p=3.0), dict(temperature=0.05),
            dict(temperature=30.0, top_p=0.9)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("how", SETTINGS, ids=str)
def test_settings(dtype, how):
    print("sample", dtype, how, flush=True)
    rng = np.random.default_rng(1)
    x = _logits(rng, 6, 5003, dtype, pad=2)
    _check(x, rng.random(6), **how)


@pytest.mark.parametrize("cols", [1, 2, 3, 7, 8, 9, 63, 64, 65, 511, 1000,
                                  1023, 1024, 1025, 2049, 8191, 8192, 8193,
                                  16385, 40000])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lengths(cols, dtype):
    print("sample cols", cols, dtype, flush=True)
    rng = np.random.default_rng(cols)
    x = _logits(rng, 5, cols, dtype, pad=cols % 3, shift=cols % 2)
    u = rng.random(5)
    _check(x, u)
    _check(x, u, top_k=17, top_p=0.9)
    _check(x, u, top_p=0.95, temperature=1.3)
    _check(x, u, temperature=0.0)


@pytest.mark.parametrize("rows,cols,dtype", [
    (1, 32000, "f32"), (3, 131072, "bf16"), (2, 200001, "f16"),
    (2, 262144, "f32"), (300, 333, "f32")])
def test_mixed_settings(rows, cols, dtype):
    print("sample mixed", rows, cols, dtype, flush=True)
    rng = np.random.default_rng(cols)
    x = _logits(rng, rows, cols, dtype)
    for i in range(4):
        j = np.arange(rows) + i
        _check(x, rng.random(rows),
               temperature=np.choose(j % 4, [0.6, 1.0, 1.4, 0.0]).astype(
                   np.float32),
               top_k=np.choose(j % 3, [0, 40, 3000]).astype(np.int32),
               top_p=np.choose(j // 2 % 3, [1.0, 0.9, 0.98]).astype(
                   np.float32),
               min_p=np.choose(j // 3 % 2, [0.0, 0.03]).astype(np.float32))


def test_wide_nuclei():
    rng = np.random.default_rng(2)
    for cols, dtype in ((50000, "f32"), (70001, "bf16"), (131072, "f16")):
        print("sample wide", cols, dtype, flush=True)
        x = _logits(rng, 3, cols, dtype, peak=0.7)
        u = rng.random(3)
        _check(x, u, top_p=0.98, temperature=1.5)
        _check(x, u, top_k=cols - 100)
        _check(x, u, top_k=cols // 2, top_p=0.9)
        _check(x, u, min_p=0.001, temperature=1.5)
        _check(x, u, top_k=9000)


def test_ends_of_the_random_numbers():
    rng = np.random.default_rng(3)
    x = _logits(rng, 8, 3001, "f32")
    u = np.array([0.0, 1.0 - 2.0 ** -24, 2.0 ** -149, 0.5, 1.0, 7.0, -3.0,
                  np.nan], np.float32)
    for how in (dict(), dict(top_k=9), dict(top_p=0.9)):
        _check(x, u, **how)
    # the first index without weight is not taken at u = 0
    x[:, 0] = -float("inf")
    x[:, 1] = -1e30
    _check(x, u)
    x[:, -1] = -float("inf")
    _check(x, u)


def test_equal_logits():
    """Ties rank by index; sums meet borders exactly."""
    for dtype in TYPES:
        for cols in (100, 1000, 9000, 70000):
            print("sample equal", dtype, cols, flush=True)
            x = torch.full((4, cols), -2.5, dtype=TYPES[dtype]).cuda()
            u = np.array([0.0, 0.25, 0.5, 0.999], np.float32)
            _check(x, u)
            for how in (dict(top_k=10), dict(top_p=0.5), dict(top_p=0.25),
                        dict(top_k=64, top_p=0.5), dict(min_p=1.0),
                        dict(top_k=cols - 1), dict(temperature=0.0)):
                _check(x, u, **how)
    # few values, each many times; the cut falls among equal ones
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.integers(-3, 4, (6, 20000)).astype(
        np.float32)).cuda()
    for k in (1, 100, 2857, 2900, 10000, 19999):
        _check(x, rng.random(6), top_k=k)
    for p in (0.3, 0.7, 0.95):
        _check(x, rng.random(6), top_p=p)
        _check(x, rng.random(6), top_p=p, top_k=5000)


def test_ordered_rows():
    """The largest logits side by side, at either end or in the middle."""
    for cols in (4000, 100000):
        ramp = torch.linspace(9, -9, cols)
        x = torch.stack([ramp, ramp.flip(0), ramp.roll(cols // 3),
                         torch.cat([ramp[::2], ramp[1::2].flip(0)])]).cuda()
        rng = np.random.default_rng(cols)
        print("sample ordered", cols, flush=True)
        for how in (dict(), dict(top_k=50), dict(top_k=2000),
                    dict(top_p=0.9), dict(top_p=0.9, top_k=300),
                    dict(min_p=0.5), dict(temperature=0.1, top_p=0.9)):
            _check(x, rng.random(4), **how)


def test_masked_and_infinite_logits():
    rng = np.random.default_rng(5)
    inf, nan = float("inf"), float("nan")
    for dtype in TYPES:
        low = torch.finfo(TYPES[dtype]).min
        for cols in (40, 3001, 20000):
            print("sample masked", dtype, cols, flush=True)
            x = _logits(rng, 12, cols, dtype).contiguous()
            x[0] = -inf
            x[1] = nan
            x[2] = low
            x[3, 1:] = -inf
            x[4, :-1] = low
            x[5, ::2] = nan
            x[6, 5], x[6, 9] = inf, inf
            x[7] = inf
            x[8, cols // 2:] = low
            x[9] = -0.0
            x[9, ::3] = 0.0
            x[10, 3:] = -inf
            x[11, 7] = torch.finfo(TYPES[dtype]).max
            u = rng.random(12)
            for how in (dict(), dict(top_k=7), dict(top_p=0.9),
                        dict(min_p=0.1), dict(temperature=0.0),
                        dict(top_k=30, top_p=0.5, temperature=0.01),
                        dict(temperature=float("inf"))):
                _check(x, u, **how)


def test_settings_of_no_meaning_are_read_as_off():
    """NaN, and negative numbers, in the settings' tensors."""
    rng = np.random.default_rng(6)
    x = _logits(rng, 4, 3001, "f32")
    u = rng.random(4).astype(np.float32)
    off = ltk.sample(x, torch.from_numpy(u).cuda())
    nan = torch.full((4,), float("nan")).cuda()
    got = ltk.sample(x, torch.from_numpy(u).cuda(), top_p=nan, min_p=nan,
                     top_k=torch.full((4,), -5, dtype=torch.int32).cuda())
    assert all(torch.equal(a, b) for a, b in zip(got, off))
    for t in (nan, -torch.ones(4).cuda()):
        got = ltk.sample(x, torch.from_numpy(u).cuda(), temperature=t)
        assert torch.equal(got[0], x.argmax(1)) and not got[1].any()


def test_no_rows_and_outputs():
    x = torch.zeros(0, 10).cuda()
    t, p = ltk.sample(x, torch.zeros(0).cuda())
    assert t.shape == (0,) and p.shape == (0,)
    x = torch.randn(3, 100).cuda()
    out = (torch.zeros(3, dtype=torch.int64).cuda(), torch.zeros(3).cuda())
    got = ltk.sample(x, torch.rand(3).cuda(), out=out)
    assert got[0] is out[0] and got[1] is out[1]
    assert out[1].lt(0).all()


def test_frequencies():
    """A row drawn from at even steps of u: each token gets its probability,
    to within one step."""
    n = 4096
    row = torch.randn(37)
    x = row.expand(n, 37).contiguous().cuda()
    u = ((torch.arange(n) + 0.5) / n).cuda()
    t, _ = ltk.sample(x, u, temperature=0.9)
    p = torch.softmax(row.double() / float(np.float32(0.9)), 0)
    got = torch.bincount(t.cpu(), minlength=37) / n
    assert ((got - p).abs() <= 1.0 / n + 1e-9).all()


def test_any_stream_and_graph():
    rng = np.random.default_rng(7)
    x = _logits(rng, 5, 40001, "f32")
    u = torch.from_numpy(rng.random(5).astype(np.float32)).cuda()
    how = dict(temperature=torch.full((5,), 0.9).cuda(),
               top_k=torch.tensor([0, 9, 0, 20000, 0],
                                  dtype=torch.int32).cuda(),
               top_p=torch.tensor([1, .9, .999, .5, .9]).cuda())
    want = ltk.sample(x, u, **how)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = ltk.sample(x, u, **how)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s, su = x.clone(), u.clone()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = ltk.sample(s, su, **how)
    for i in range(4):
        y = _logits(rng, 5, 40001, "f32")
        v = torch.from_numpy(rng.random(5).astype(np.float32)).cuda()
        eager = ltk.sample(y, v, **how)
        s.copy_(y)
        su.copy_(v)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_gradients_are_refused():
    x = torch.randn(2, 50).cuda().requires_grad_()
    _, lp = ltk.sample(x, torch.rand(2).cuda())
    with pytest.raises(RuntimeError, match="sample_logits"):
        lp.sum().backward()


def test_rows_past_32_bits():
    """The last row lies more than 2^32 bytes from the first."""
    rows, ld = 3, 600_000_000
    base = torch.zeros(2 * ld + 1000, dtype=torch.float32, device="cuda")
    x = torch.as_strided(base, (rows, 1000), (ld, 1))
    rng = np.random.default_rng(8)
    x.copy_(_logits(rng, rows, 1000, "f32"))
    _check(x, rng.random(rows), top_p=0.9)
