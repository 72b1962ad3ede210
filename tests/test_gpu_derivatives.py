"""Gradients that no call computes are errors, for each input on which new
outputs depend."""
import numpy as np
import pytest
import torch

import test_gpu_extend as ext
import top_selection_two_amd as ltk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["q", "q_norm", "freqs"])
def test_extend(name):
    rng = np.random.default_rng(1)
    q, k, v = ext._new(rng, [4], 2, 1, 64, "bf16")
    dev, _ = ext._blank(rng, [0], [4], 1, 64, 16, "bf16")
    d = dict(q=q, q_norm=torch.ones(64).cuda(), k_norm=torch.ones(64).cuda(),
             freqs=torch.ones(32).cuda())
    d[name] = d[name].detach().clone().requires_grad_()
    starts = torch.tensor([0, 4], dtype=torch.int32).cuda()

    def call(**kw):
        return ltk.cache_extend(k, v, dev["k"], dev["v"], dev["table"],
                                dev["lens"], starts, **d, **kw)[1]

    with pytest.raises(RuntimeError, match="cache_extend"):
        call().float().sum().backward()
    assert not call(out=torch.empty_like(q).contiguous()).requires_grad
    with torch.no_grad():
        assert not call().requires_grad


@pytest.mark.parametrize("name", ["logits", "temperature"])
def test_sample(name):
    d = dict(logits=torch.randn(2, 50).cuda(),
             temperature=torch.full((2,), 0.9).cuda(),
             u=torch.rand(2).cuda())
    d[name].requires_grad_()
    tokens, lp = ltk.sample(**d)
    assert not tokens.requires_grad
    with pytest.raises(RuntimeError, match="sample_logits"):
        lp.sum().backward()
    with torch.no_grad():
        assert not ltk.sample(**d)[1].requires_grad


@pytest.mark.parametrize("name", ["q", "k", "v", "weights", "k_scale",
                                  "v_scale"])
def test_attend(name):
    rng = np.random.default_rng(2)
    k = torch.randn(3, 2, 16, 64).cuda().to(torch.bfloat16)
    d = dict(q=torch.randn(1, 4, 64).cuda().to(torch.bfloat16), k=k,
             v=k.clone(), weights=torch.zeros(1, 2, 48).cuda(),
             k_scale=torch.ones(2).cuda(), v_scale=torch.ones(2).cuda())
    if name != "weights":
        d[name] = d[name].requires_grad_()
    else:
        d[name] = torch.zeros(1, 2, 48).cuda().requires_grad_() * 1
    table = torch.from_numpy(rng.permutation(3).astype(np.int32))
    out, lse = ltk.cache_attend(
        table=table.view(1, 3).cuda(),
        lens=torch.tensor([40], dtype=torch.int32).cuda(), **d)
    for x in (out, lse):
        with pytest.raises(RuntimeError, match="cache_attend"):
            x.float().sum().backward()
