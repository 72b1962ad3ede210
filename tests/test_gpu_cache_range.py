"""Attention over a paged cache where the range of the numbers counts: slots of
tiny probability that alone decide an output, infinite V rows, and sums that
cancel.

Bounds, with u = 2^-24: as for finite rows in test_gpu_cache.py (a score's
error is dx, a probability's 2 dx + (n + 8) u relative, the sum over V another
(n + 8) u), but with probabilities that enter the sum as float32: out is off by
those times sum p |V|, and by its one rounding.  The bounds are relative to the
probabilities, however small these are.
"""
import numpy as np
import pytest
import torch

import oracle.cache as oc
import top_selection_two_amd as ltk
from test_gpu_cache import TINY, TYPES, U, _case

pytestmark = pytest.mark.gpu

PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")]


def _put(dev, ref, name, b, t, row, head=slice(None)):
    """Row(s) of slot t of a sequence, on both sides, rounded to the type."""
    page = ref["k"].shape[2]
    p, z = int(ref["table"][b, t // page]), t % page
    x = torch.as_tensor(row, dtype=torch.float32).to(dev[name].dtype)
    if x.element_size() == 1:
        dev[name].view(torch.uint8)[p, head, z] = x.view(torch.uint8).cuda()
    else:
        dev[name][p, head, z] = x.cuda()
    ref[name][p, head, z] = x.double().numpy()


def _run(dev, q, ref, scale, weights, seed):
    b, dim = q.shape[0], q.shape[2]
    heads, page = ref["k"].shape[1], ref["k"].shape[2]
    w = torch.zeros(b, heads, dev["table"].shape[1] * page,
                    device="cuda") if weights else None
    out, lse = ltk.cache_attend(q, dev["k"], dev["v"], dev["table"],
                                dev["lens"], scale=scale, weights=w)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        want = oc.attend(q.double().cpu().numpy(), ref, scale)
    return out.double().cpu().numpy(), want


def _bound(want, n, dim, qtype):
    o, z, _, spread, size = want
    dx = (dim + 12) * U * size + 4 * U * np.abs(z)
    dp = 2 * dx + (n + 8) * U
    eps = torch.finfo(TYPES[qtype]).eps / 2
    return eps * np.abs(o) + TINY[qtype] + \
        (1 + eps) * (dp[:, :, None] + (n + 8) * U) * spread


@pytest.mark.parametrize("qtype,ctype", PAIRS)
@pytest.mark.parametrize("gap", [8.0, 12.0, 16.0, 18.0, 26.0])
@pytest.mark.parametrize("heads,slots_first", [(2, False), (4, True)])
def test_attend_outputs_of_tiny_probabilities(qtype, ctype, gap, heads,
                                              slots_first):
    """A slot that takes nearly all weight and whose V row is zero: what is
    left of out comes from slots exp(gap) times less probable."""
    lens = [2, 31, 70, 1000, 9000]
    rng, dev, ref = _case(int(gap), lens, heads, 64, 16, ctype, slots_first)
    print("tiny probabilities", qtype, ctype, gap, heads, flush=True)
    # scores: elements 0 and 1 of K times ones, the others times zero
    for b, n in enumerate(lens):
        for t in range(n):
            at = ref["table"][b, t // 16], slice(None), t % 16
            ref["k"][at][:, 0] = 0.0
            ref["k"][at][:, 1] *= 0.25
            ref["v"][at] = rng.choice([96.0, 288.0, 448.0], (heads, 64))
    for name in ("k", "v"):
        x = torch.from_numpy(ref[name]).to(TYPES[ctype])
        ref[name] = x.double().numpy()
        dev[name] = x.transpose(1, 2).contiguous().cuda().transpose(1, 2) \
            if slots_first else x.cuda()
    for b, t in enumerate((0, 17, 69, 500, 8000)):
        row = np.zeros((heads, 64))
        row[:, 0] = gap
        _put(dev, ref, "k", b, t, row)
        _put(dev, ref, "v", b, t, np.zeros((heads, 64)))
    q = torch.zeros(len(lens), heads * 2, 64)
    q[:, :, :2] = 1.0
    for weights in (True, False):
        out, want = _run(dev, q.to(TYPES[qtype]).cuda(), ref, 1.0, weights, 1)
        tol = _bound(want, max(lens), 64, qtype)
        bad = np.abs(out - want[0]) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5],
                               want[0][bad][:5], tol[bad][:5])


def test_attend_two_slots_far_apart():
    """Scores 0 and -25 ln 2, V 0 and 1000: out is 1000 / (2^25 + 1)."""
    _, dev, ref = _case(1, [2], 1, 64, 16, "f16")
    for t, (x, v) in enumerate(((0.0, 0.0), (-17.328125, 1000.0))):
        k = np.zeros(64)
        k[0] = x
        _put(dev, ref, "k", 0, t, k)
        _put(dev, ref, "v", 0, t, np.full(64, v))
    q = torch.zeros(1, 1, 64)
    q[..., 0] = 1.0
    out, want = _run(dev, q.to(torch.float16).cuda(), ref, 1.0, False, 1)
    assert want[0][0, 0, 0] > 2.9e-5
    assert (np.abs(out - want[0]) <= _bound(want, 2, 64, "f16")).all()


@pytest.mark.parametrize("qtype,ctype", PAIRS)
@pytest.mark.parametrize("weights", [True, False])
def test_attend_sums_that_cancel(qtype, ctype, weights):
    """Pairs of slots with V rows of opposite signs whose scores differ by
    2^-13: out is about 2^-14 of sum p |V| and its rounding at most 2^-22 of
    it, so that probabilities held in fewer bits than float32 show.

    Scores are sums of few exact products: off by the rounding of scale *
    log2 e and of the product with it, 2 u |x|; the exponential by 2 u, sums
    of n terms by n u each, the division by 4 u and the products by u."""
    lens = [3, 5, 7] * 8
    rng, dev, ref = _case(5, lens, 2, 64, 16, ctype)
    print("cancelling", qtype, ctype, weights, flush=True)
    for b, n in enumerate(lens):
        # slot 0: the largest score, 0, and no V
        _put(dev, ref, "k", b, 0, np.zeros((2, 64)))
        _put(dev, ref, "v", b, 0, np.zeros((2, 64)))
        for t in range(1, n, 2):
            v = rng.choice([-1.75, -1.0, 1.0, 1.5], (2, 64))
            base = -rng.integers(1, 9) / 8
            for i in range(2):
                k = np.zeros((2, 64))
                k[:, 0] = base
                k[:, 1] = float(i)
                _put(dev, ref, "k", b, t + i, k)
                _put(dev, ref, "v", b, t + i, v if i else -v)
    q = torch.zeros(len(lens), 6, 64)
    q[:, :, 0] = torch.tensor([0.5, 1.0, 0.625, 0.75, 0.875, 0.25])
    q[:, :, 1] = 2.0 ** -13
    out, want = _run(dev, q.to(TYPES[qtype]).cuda(), ref, 1.0, weights, 2)
    n = np.asarray(lens)[:, None, None]
    eps = torch.finfo(TYPES[qtype]).eps / 2
    tol = eps * np.abs(want[0]) + TINY[qtype] + \
        (2 * 1.0 + 2 + 2 * n + 4 + 1) * U * want[3]
    assert (np.abs(want[0]) < 2.0 ** -12 * want[3].max()).all()
    bad = np.abs(out - want[0]) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5],
                           want[0][bad][:5], tol[bad][:5])


INF = float("inf")


@pytest.mark.parametrize("ctype", ["bf16", "f16"])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("heads,dim,slots_first", [(2, 64, False),
                                                   (4, 136, True)])
def test_attend_infinite_v(ctype, weights, heads, dim, slots_first):
    """Infinities of V, at the largest score, at ordinary ones and at scores
    down to 80 below it, make their columns infinite (NaN where both signs or
    a NaN meet), and no others."""
    lens = [1, 2, 33, 100, 700, 5000]
    rng, dev, ref = _case(7, lens, heads, dim, 16, ctype, slots_first)
    print("infinite v", ctype, weights, heads, dim, flush=True)
    for b, n in enumerate(lens):
        for t in (0, n // 2, n - 1):
            k = np.zeros((heads, dim))
            # 0 the largest, and far below it
            k[:, 0] = 40.0 if t == 0 else -40.0 if t == n - 1 else 0.0
            _put(dev, ref, "k", b, t, k)
            v = rng.standard_normal((heads, dim))
            v[:, 3 + (t == 0)] = INF
            v[:, 6 + (t == n - 1)] = -INF
            v[:, 9] = -INF if t == 0 else 1.0
            v[:, 10] = INF if t == n - 1 else 1.0
            v[:, 11] = INF if t == n // 2 else 1.0
            v[:, 12] = float("nan") if t == n - 1 else 2.0
            v[:, dim - 1] = INF if t == n - 1 else 1.0
            _put(dev, ref, "v", b, t, v)
    q = torch.zeros(len(lens), heads * 3, dim)
    q[:, :, 0] = 1.0
    q[:, 1::3, 1] = 0.5
    out, want = _run(dev, q.to(TYPES[ctype]).cuda(), ref, 1.0, weights, 3)
    o = want[0]
    assert np.isposinf(o).any() and np.isneginf(o).any() and np.isnan(o).any()
    assert np.array_equal(np.isnan(out), np.isnan(o))
    assert np.array_equal(np.isposinf(out), np.isposinf(o))
    assert np.array_equal(np.isneginf(out), np.isneginf(o))
    fin = np.isfinite(o)
    with np.errstate(invalid="ignore"):
        tol = _bound(want, max(lens), dim, ctype)
        bad = fin & (np.abs(out - o) > tol)
    assert not bad.any()


@pytest.mark.parametrize("ctype", ["bf16", "f16"])
def test_attend_infinite_v_under_every_weight(ctype):
    """Weights over the whole range, powers of two and others, each before an
    infinity of its own column."""
    n, dim = 128, 128
    _, dev, ref = _case(8, [n], 1, dim, 16, ctype)
    for t in range(n):
        k = np.zeros((1, dim))
        k[:, 0] = -t * 0.625
        _put(dev, ref, "k", 0, t, k)
        v = np.ones((1, dim))
        v[:, t] = INF if t % 3 else -INF
        _put(dev, ref, "v", 0, t, v)
    q = torch.zeros(1, 4, dim)
    # steps of 0.625 and 0.3 nats, of one and of half a power of two
    q[0, :, 0] = torch.tensor([1.0, 0.5, 1.109375, 0.5546875])
    out, want = _run(dev, q.to(TYPES[ctype]).cuda(), ref, 1.0, False, 3)
    assert np.isinf(want[0]).all()
    assert np.array_equal(out, want[0])


@pytest.mark.parametrize("ctype", ["bf16", "f16"])
def test_attend_infinite_v_in_joined_rows(ctype):
    """Long rows with weights, whose shares the second launch joins."""
    lens, dim = [12000, 7001], 64
    rng, dev, ref = _case(9, lens, 1, dim, 16, ctype)
    print("infinite v, joined", ctype, flush=True)
    for b, n in enumerate(lens):
        for i, t in enumerate((0, 31, n // 2, n - 1)):
            v = rng.standard_normal((1, dim))
            v[:, 5 + i] = -INF if i % 2 else INF
            v[:, 20] = INF
            v[:, 21] = -INF if i == 2 else INF
            _put(dev, ref, "v", b, t, v)
    q = torch.from_numpy(rng.standard_normal((2, 5, dim)).astype(np.float32))
    out, want = _run(dev, q.to(TYPES[ctype]).cuda(), ref, dim ** -0.5, True, 3)
    o = want[0]
    for f in (np.isnan, np.isposinf, np.isneginf):
        assert f(o).any() and np.array_equal(f(out), f(o))
    fin = np.isfinite(o)
    with np.errstate(invalid="ignore"):
        bad = fin & (np.abs(out - o) > _bound(want, max(lens), dim, ctype))
    assert not bad.any()
