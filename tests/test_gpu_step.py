"""A decoding step's calls together on the GPU: prompts enter a 4-bit cache,
attention over it, eviction and sampling, each against the float64 oracle on
what the call before it left; and calls that share a stream's workspace, from
two threads and from captured graphs.

Bounds are those of the calls' own tests."""
import importlib.util
import os
import threading

import numpy as np
import pytest
import torch

import oracle.cache as oc
import oracle.step as st
import test_gpu_cache as base
import test_gpu_extend as ext
import test_gpu_sample as smp
import top_selection_two_amd as ltk

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(
        os.path.abspath(__file__))), "examples", "generate.py")
    spec = importlib.util.spec_from_file_location("generate", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _host(x):
    return x.double().cpu().numpy()


def _ref(cache):
    r = {"table": cache.table.cpu().numpy(),
         "lens": cache.lens.cpu().numpy().astype(np.int64)}
    for name in ("k", "v"):
        r[name] = st.unpack(ext._bytes(getattr(cache, name)),
                            ext._bytes(getattr(cache, name + "_blocks")))
    return r


def _extended(model, cache, tokens, counts):
    """Extends the cache, checked; the queries and the rows they came with."""
    x, q, k, v = model.projected(tokens)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    want_q, writes, lens = st.extend(
        _host(q), _host(k), _host(v), _ref(cache), starts,
        cache.seen.cpu().numpy(), _host(model.q_norm), _host(model.k_norm),
        float(np.float32(1e-6)), _host(model.freqs),
        slots=cache.weights.shape[2])
    k0, v0 = k.clone(), v.clone()
    q = cache.extend(model, q, k, v, torch.from_numpy(starts).cuda())
    torch.cuda.synchronize()
    assert torch.equal(k, k0) and torch.equal(v, v0)
    size = np.abs(want_q).max(-1, keepdims=True) + np.zeros_like(want_q)
    ext._near(_host(q), want_q, size, "bf16")
    assert np.array_equal(cache.lens.cpu().numpy(), lens)
    for page, h, place, kr, vr, b, slot, position in writes:
        for name, row in (("k", kr), ("v", vr)):
            at = page, h, place
            ext._same4(row, ext._bytes(getattr(cache, name))[at],
                       ext._bytes(getattr(cache, name + "_blocks"))[at])
        assert int(cache.positions[b, h, slot]) == position
    return x, q


def _attended(cache, q):
    w0 = cache.weights.cpu().numpy()
    want = oc.attend(_host(q), _ref(cache), q.shape[2] ** -0.5,
                     slots=cache.weights.shape[2])
    got = ltk.cache_attend(q, cache.k, cache.v, cache.table, cache.lens,
                           weights=cache.weights, k_blocks=cache.k_blocks,
                           v_blocks=cache.v_blocks)
    torch.cuda.synchronize()
    base._check_attend(got, want, int(cache.lens.max()), q.shape[2], "bf16",
                       "e4m3", w0, cache.weights.cpu().numpy())
    return got[0]


def test_steps_follow_the_oracle():
    gen = _example()
    rng = np.random.default_rng(7)
    model = gen.Decoder(vocab=3001, heads=2, group=4, dim=64)
    counts = [37, 0, 1, 90]
    cache = gen.Cache(4, 2, 64, 96)
    tokens = torch.from_numpy(rng.integers(0, 3001, sum(counts))).cuda()
    print("prompts", flush=True)
    x, q = _extended(model, cache, tokens, counts)
    last = torch.tensor([36, 0, 37, 127], device="cuda")  # (the second's: any)
    x, q = x[last], q[last]
    for step in range(6):
        print("step", step, flush=True)
        out = _attended(cache, q)
        if step == 2:
            before, ref = cache.weights.cpu().numpy(), _ref(cache)
            positions = cache.positions.cpu().numpy()
            k, v, w, p, lens = oc.evict(ref, cache.seen.cpu().numpy(), before,
                                        positions, 40, gen.SINKS, gen.RECENT)
            cache.evict(40)
            torch.cuda.synchronize()
            assert np.array_equal(cache.weights[..., :40].cpu().numpy(), w)
            assert np.array_equal(cache.positions[..., :40].cpu().numpy(), p)
            now = _ref(cache)
            assert np.array_equal(now["lens"], lens)
            assert np.array_equal(now["k"], k, equal_nan=True)
            assert np.array_equal(now["v"], v, equal_nan=True)
        logits = model.logits(x, out)
        u = rng.random(4).astype(np.float32)
        got = smp._check(logits, u, top_k=np.array([0, 40, 0, 5], np.int32),
                         top_p=np.array([1, .9, .95, 1], np.float32),
                         temperature=np.array([.7, 1, 1.3, 0], np.float32))
        x, q = _extended(model, cache, got[0], [1, 1, 1, 1])


@pytest.mark.parametrize("steps", [0, 1, 60])
def test_example_eager_and_captured(steps):
    gen = _example()
    model = gen.Decoder(vocab=2000, heads=2, group=4, dim=64)
    r = np.random.default_rng(1)
    prompts = [r.integers(0, 2000, n).tolist() for n in (50, 3, 200)]
    results = []
    side = torch.cuda.Stream()
    for graph in (False, True, True):
        print("generate", steps, graph, flush=True)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            results.append(gen.generate(model, prompts, steps, 64,
                                        graph=graph))
        side.synchronize()
    tokens, logprobs, cache = results[0]
    assert tokens.shape == (steps + 1, 3) and (tokens >= 0).all()
    assert logprobs.isfinite().all() and (logprobs <= 0).all()
    for t, p, c in results[1:]:
        assert torch.equal(t, tokens) and torch.equal(p, logprobs)
        assert torch.equal(c.lens, cache.lens)
        assert torch.equal(c.weights, cache.weights)
        for name in ("k", "v", "k_blocks", "v_blocks"):
            assert torch.equal(getattr(c, name).view(torch.uint8),
                               getattr(cache, name).view(torch.uint8))
    assert cache.seen.tolist() == [50 + steps, 3 + steps, 200 + steps]
    for b in range(3):
        n, seen = int(cache.lens[b]), int(cache.seen[b])
        assert n <= 64
        for row in cache.positions[b, :, :n].cpu().numpy():
            have = set(row.tolist())
            assert len(have) == n and set(range(min(4, seen))) <= have
            assert set(range(max(0, seen - 16), seen)) <= have


def test_two_threads_share_a_stream():
    """Calls of several launches that hand results to one another."""
    rng = np.random.default_rng(3)
    x = smp._logits(rng, 5, 30001, "f32")
    y = smp._logits(rng, 70, 131072, "bf16", peak=0.7)
    u = torch.from_numpy(rng.random(70).astype(np.float32)).cuda()
    _, dev, _ = ext._case4(1, [3000, 9000], 2, 64, 16)
    q = base._q(rng, 2, 32, 64, "bf16", 0.05)

    def a():
        return ltk.sample(x, u[:5], top_k=700, top_p=0.9)

    def b():
        return ltk.sample(y, u, top_p=0.98)

    def c():
        w = torch.zeros(2, 2, dev["table"].shape[1] * 16, device="cuda")
        got = ltk.cache_attend(q, dev["k"], dev["v"], dev["table"],
                               dev["lens"], weights=w,
                               k_blocks=dev["k_blocks"],
                               v_blocks=dev["v_blocks"])
        return (*got, w)

    want = [f() for f in (a, b, c)]
    torch.cuda.synchronize()
    got = [[], [], []]

    def run(i):
        with torch.cuda.device(0):
            for _ in range(20):
                got[i].append((a, b, c)[i]())

    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, results in zip(want, got):
        assert len(results) == 20
        for r in results:
            assert all(torch.equal(m, n) for m, n in zip(r, w))


def test_graphs_share_a_stream_s_workspace():
    """Graphs of two sizes on one stream, replayed in turn with eager calls
    that let the workspace grow."""
    rng = np.random.default_rng(4)
    x = smp._logits(rng, 3, 20000, "f32")
    y = smp._logits(rng, 20, 100000, "f16", peak=0.8)
    big = smp._logits(rng, 90, 131072, "bf16")
    u = torch.from_numpy(rng.random(90).astype(np.float32)).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        calls = [lambda: ltk.sample(x, u[:3], top_p=0.9, out=outs[0]),
                 lambda: ltk.sample(y, u[:20], top_p=0.98, top_k=50000,
                                    out=outs[1])]
        want = [ltk.sample(x, u[:3], top_p=0.9),
                ltk.sample(y, u[:20], top_p=0.98, top_k=50000)]
        outs = [tuple(torch.zeros_like(t) for t in w) for w in want]
        side.synchronize()
        graphs = []
        for call in calls:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                call()
        first = None
        for i in range(4):
            for g, w, o in zip(graphs, want, outs):
                for t in o:
                    t.zero_()
                g.replay()
                assert all(torch.equal(m, n) for m, n in zip(w, o))
            eager = ltk.sample(big, u, top_p=0.95)
            first = first or eager
            assert all(torch.equal(m, n) for m, n in zip(eager, first))
    side.synchronize()


@pytest.mark.parametrize("rows,cols", [(3000, 5000), (70, 1 << 20)])
def test_rows_in_batches(rows, cols):
    """More rows than one workspace holds give what a few at a time do."""
    rng = np.random.default_rng(rows)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16)
    x *= 2
    u = torch.rand(rows, generator=g, device="cuda")
    top_p = torch.from_numpy(np.where(np.arange(rows) % 3 == 0, 0.999,
                                      0.9).astype(np.float32)).cuda()
    got = ltk.sample(x, u, top_p=top_p, top_k=5000)
    torch.cuda.synchronize()
    for lo in range(0, rows, 100):
        part = slice(lo, min(lo + 100, rows))
        some = ltk.sample(x[part], u[part], top_p=top_p[part], top_k=5000)
        assert torch.equal(some[0], got[0][part])
        assert torch.equal(some[1], got[1][part])
    for r in rng.integers(0, rows, 2):
        lo = int(r)
        smp._check(x[lo:lo + 1], u[lo:lo + 1].cpu().numpy(),
                   top_p=float(top_p[lo]), top_k=5000,
                   got=(got[0][lo:lo + 1], got[1][lo:lo + 1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_beyond_a_million_logits(dtype):
    rng = np.random.default_rng(5)
    x = smp._logits(rng, 2, (1 << 20) + 77, dtype, peak=0.9)
    u = rng.random(2)
    smp._check(x, u, top_p=0.9)
    smp._check(x, u, top_k=30, min_p=0.01, temperature=0.7)
    smp._check(x, u)


@pytest.mark.parametrize("page", [512, 100])
def test_4_bit_rows_past_32_bits(page):
    """Rows (and scales) more than 2^32 bytes apart, the last pages of the
    cache: attention, and eviction from and to them."""
    rng = np.random.default_rng(6)
    dim, slots, blocks = 128, 700, 4
    pages = (1 << 32) // (page * 64) + 30
    dev = torch.device("cuda")
    used = -(-slots // page)
    table = np.arange(pages - used, pages, dtype=np.int32)[None, ::-1].copy()
    sizes = {"k": 64, "v": 64, "k_blocks": blocks, "v_blocks": blocks}
    big, small = {}, {}
    for name, n in sizes.items():
        step = 64 if name == "k_blocks" else n  # scales as far apart as rows
        x = torch.zeros(pages, 1, page, step, dtype=torch.uint8, device=dev)
        x = x[..., :n]
        bits = rng.integers(118, 128, (used, 1, page, n)) if "blocks" in name \
            else rng.integers(0, 256, (used, 1, page, n))
        small[name] = torch.from_numpy(bits.astype(np.uint8)).to(dev)
        x[pages - used:] = small[name]
        kind = torch.float8_e8m0fnu if "blocks" in name else \
            torch.float4_e2m1fn_x2
        big[name], small[name] = x.view(kind), small[name].view(kind)
    assert big["k"].numel() > 1 << 32
    lens = torch.tensor([slots], dtype=torch.int32, device=dev)
    q = base._q(rng, 1, 4, dim, "bf16", 0.05)
    tables = [torch.from_numpy(t).to(dev)
              for t in (table, table - (pages - used))]
    seen = torch.tensor([slots], dtype=torch.int32, device=dev)
    results = []
    for cache, t in zip((big, small), tables):
        w = torch.zeros(1, 1, used * page, device=dev)
        got = ltk.cache_attend(q, cache["k"], cache["v"], t, lens, weights=w,
                               k_blocks=cache["k_blocks"],
                               v_blocks=cache["v_blocks"])
        pos = torch.arange(used * page, dtype=torch.int32, device=dev)
        cut = ltk.cache_evict(cache["k"], cache["v"], t, lens, seen, w,
                              pos.view(1, 1, -1).contiguous(), 300,
                              k_blocks=cache["k_blocks"],
                              v_blocks=cache["v_blocks"])
        results.append((*got, w, *cut))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert float(results[0][2].sum()) == pytest.approx(4.0, abs=1e-3)
    for name in sizes:
        assert torch.equal(big[name].view(torch.uint8)[pages - used:],
                           small[name].view(torch.uint8)), name
        assert not big[name].view(torch.uint8)[:2].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [5003, 70001])
def test_settings_at_their_ends(cols, dtype):
    """Prefixes that are all but the whole row, next to nothing, and
    temperatures beyond any use."""
    print("ends", cols, dtype, flush=True)
    rng = np.random.default_rng(cols + 1)
    x = smp._logits(rng, 3, cols, dtype, peak=0.9)
    u = rng.random(3)
    nearly = float(np.nextafter(np.float32(1), np.float32(0)))
    for how in (dict(top_p=nearly), dict(top_p=1e-30), dict(min_p=1e-38),
                dict(temperature=1e-30, top_p=0.9),
                dict(temperature=1e-45), dict(temperature=1e30, top_p=0.5),
                dict(temperature=3e38), dict(top_k=cols - 1, top_p=nearly),
                dict(top_k=2 ** 31 - 1, min_p=1e-6)):
        smp._check(x, u, **how)


def test_workspaces_that_held_anything():
    """Neither the tickets nor the rest of a workspace say anything to the
    next call."""
    rng = np.random.default_rng(8)
    x = smp._logits(rng, 9, 60000, "f16", peak=0.7)
    u = torch.from_numpy(rng.random(9).astype(np.float32)).cuda()
    p = torch.tensor([1, .5, .9, .98, 1, .999, .3, .97, .95], device="cuda")
    want = ltk.sample(x, u, top_p=p, top_k=30000)
    _, dev, _ = ext._case4(2, [3000, 9000], 2, 64, 16)
    q = base._q(rng, 2, 32, 64, "bf16", 0.05)
    stream = torch.cuda.current_stream().cuda_stream
    for i in range(3):
        w = torch.zeros(2, 2, dev["table"].shape[1] * 16, device="cuda")
        ltk.cache_attend(q, dev["k"], dev["v"], dev["table"], dev["lens"],
                         weights=w, k_blocks=dev["k_blocks"],
                         v_blocks=dev["v_blocks"])
        assert ltk.lib.cache_debug_scramble(stream, 5 + i) == ltk.OK
        got = ltk.sample(x, u, top_p=p, top_k=30000)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
