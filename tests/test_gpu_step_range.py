"""The ends of a decoding step's numbers on the GPU, against the float64
oracle: tokens whose weight is next to nothing, and norm weights of the rows'
own type at both ends of its range.

Bounds are those of the calls' own tests.
"""
import numpy as np
import pytest
import torch

import oracle.step as st
import test_gpu_extend as ext
import test_gpu_sample as smp
import top_selection_two_amd as ltk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [3, 1000, 5003, 70001])
@pytest.mark.parametrize("gap,temperature", [(86, 1.0), (90, 1.0), (200, 1.0),
                                             (700, 1.0), (44, 0.25)])
def test_tokens_of_next_to_no_weight(dtype, cols, gap, temperature):
    """At u = 0 the first logit above -infinity is drawn, and past the end the
    last, however far they lie below the largest: their weights are above 0 in
    64 bits (down to e^-744)."""
    print("sample far", dtype, cols, gap, temperature, flush=True)
    x = torch.full((4, cols), -float("inf"), dtype=smp.TYPES[dtype])
    x[:, 0] = x[:, cols - 1] = -gap
    x[:2, cols // 2] = 0
    x[2, cols // 2] = x[2, cols // 3] = 8  # (cols = 3: one)
    x[3] = -gap
    x[3, cols // 2] = 0
    x = x.cuda()
    for u in (0.0, 1.0, 2.0 ** -149, 0.4):
        got = smp._check(x, [u] * 4, temperature=temperature)
        assert got[1].isfinite().all()
    assert smp._check(x, [0.0] * 4, temperature=temperature)[0].tolist() == \
        [0] * 4
    assert smp._check(x, [1.0] * 4, temperature=temperature)[0].tolist() == \
        [cols - 1] * 4


def _with_norm(rows, weight, eps, ctype, rot, dtype, q_heads=2):
    """cache_extend of rows [N, 64], a sequence of N tokens, with norm weights
    of the rows' own type, against the oracle."""
    n, dim = rows.shape
    x = rows.to(smp.TYPES[dtype])[:, None].expand(n, q_heads, dim)
    x = x.contiguous().cuda()
    g = torch.full((dim,), weight, dtype=x.dtype).cuda()
    rng = np.random.default_rng(n)
    dev, ref = ext._blank(rng, [0], [n], q_heads, dim, 16, ctype)
    freqs = np.geomspace(1, 0.01, rot // 2).astype(np.float32)
    starts = torch.tensor([0, n], dtype=torch.int32).cuda()
    _, got = ltk.cache_extend(
        x, x, dev["k"], dev["v"], dev["table"], dev["lens"], starts, q=x,
        freqs=torch.from_numpy(freqs).cuda() if rot else None, q_norm=g,
        k_norm=g, eps=eps, k_blocks=dev.get("k_blocks"),
        v_blocks=dev.get("v_blocks"))
    torch.cuda.synchronize()
    host = x.double().cpu().numpy()
    w = g.double().cpu().numpy()
    want, writes, _ = st.extend(host, host, host, ref, [0, n], None, w, w,
                                float(np.float32(eps)),
                                freqs if rot else None)
    have = got.double().cpu().numpy()
    size = np.abs(want).max(-1, keepdims=True) + np.zeros_like(want)
    ext._near(have, want, size, dtype)
    after = {m: ext._raw(dev[m]) for m in ("k", "k_blocks") if m in dev}
    for page, h, place, row, _, _, _, _ in writes:
        at = page, h, place
        if ctype == "e2m1":
            ext._same4(row, after["k"][at], after["k_blocks"][at])
        else:
            y = torch.from_numpy(after["k"][at]).view(
                ext.TYPES[ctype]).double().numpy()
            if ctype == "e4m3":
                row = np.clip(row, -448, 448)
            ext._near(y, row, np.abs(row).max(), ctype)


@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("ctype", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_weights_at_the_ends_of_bfloat16(ctype, rot, eps):
    """x g may lie beyond float32's range, above or below; x / size(x) g does
    not."""
    rng = np.random.default_rng(rot)
    signs = torch.from_numpy(rng.choice([-1.0, 1.0], (6, 64)))
    sizes = torch.tensor([3e38, 1.7e38, 2.0 ** 100, 1.0, 2.0 ** -70,
                          2.0 ** -120])[:, None]
    spread = torch.from_numpy(rng.uniform(0.5, 1.0, (6, 64)))
    for weight in (1.25, 2.0, 2.0 ** 80, 2.0 ** -30, 2.0 ** -90):
        print("norm", ctype, rot, eps, weight, flush=True)
        _with_norm((signs * sizes * spread).float(), weight, eps, ctype, rot,
                   "bf16")


@pytest.mark.parametrize("ctype", ["f16", "e4m3", "e2m1"])
def test_norm_weights_at_the_ends_of_float16(ctype):
    rng = np.random.default_rng(3)
    rows = torch.from_numpy(rng.uniform(-1, 1, (4, 64))).float()
    rows *= torch.tensor([65504.0, 1.0, 2.0 ** -12, 2.0 ** -20])[:, None]
    for weight in (1.5, 100.0, 2.0 ** -20):
        print("norm f16", ctype, weight, flush=True)
        _with_norm(rows, weight, 0.0, ctype, 64, "f16")


def test_what_counts_as_a_weight():
    """Without settings a row of at most 2^20 logits draws whatever has a
    weight in 64 bits; where weights are added as integers, one below half a
    unit (2^-51 of the largest here, 2^-41 of 2^20 + 1 logits) is none."""
    for cols, gap in ((2, 40.0), (2000, 40.0), ((1 << 20) + 1, 30.0)):
        print("sample units", cols, flush=True)
        x = torch.full((1, cols), -float("inf"))
        x[0, 0], x[0, cols - 1] = -gap, 0.0
        x = x.cuda()
        u = torch.zeros(1).cuda()
        for how in (dict(), dict(min_p=1e-38), dict(top_k=cols - 1, min_p=1e-38),
                    dict(top_p=0.9999999)):
            tokens, lp = ltk.sample(x, u, **how)
            if not how and cols < 1 << 20:
                assert tokens.tolist() == [0]
                assert abs(float(lp) + gap) <= gap * 2.0 ** -24
            else:
                assert tokens.tolist() == [cols - 1] and float(lp) == 0
