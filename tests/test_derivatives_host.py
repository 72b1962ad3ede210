"""Forward-mode tangents are refused by the calls whose outputs would lose
them, before anything is launched (on the CPU: before the device is missed)."""
import pytest
import torch
from torch.autograd import forward_ad

import test_cache_host as base
import test_step_host as step
import top_selection_two_amd as ltk


def _dual(x):
    return forward_ad.make_dual(x, torch.ones_like(x))


@pytest.mark.parametrize("name", ["q", "k", "v", "weights", "k_scale",
                                  "v_scale"])
def test_attend(name):
    with forward_ad.dual_level():
        d = base._t(k_scale=torch.ones(4), v_scale=torch.ones(4))
        d = {n: d[n] for n in ("q", "k", "v", "table", "lens", "weights",
                               "k_scale", "v_scale")}
        with pytest.raises(ValueError, match="device"):
            ltk.cache_attend(**d)
        d[name] = _dual(d[name])
        with pytest.raises(NotImplementedError, match="cache_attend"):
            ltk.cache_attend(**d)
        out = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 8)
        with pytest.raises(ValueError, match="device"):
            ltk.cache_attend(**d, out=out)


@pytest.mark.parametrize("name", ["q", "q_norm", "freqs"])
def test_extend(name):
    with forward_ad.dual_level():
        d = step._t(q_norm=torch.ones(64), k_norm=torch.ones(64),
                    freqs=torch.ones(32))
        with pytest.raises(ValueError, match="device"):
            ltk.cache_extend(**d)
        x = d[name]
        d[name] = _dual(x)
        with pytest.raises(NotImplementedError, match="cache_extend"):
            ltk.cache_extend(**d)
        # rows alone, and queries that are given, have none anyway
        with pytest.raises(ValueError, match="device"):
            ltk.cache_extend(**dict(d, q=None))
        with pytest.raises(ValueError, match="device"):
            ltk.cache_extend(**d, out=torch.zeros_like(step._t()["q"]))


@pytest.mark.parametrize("name", ["logits", "temperature"])
def test_sample(name):
    with forward_ad.dual_level():
        d = dict(logits=torch.zeros(2, 9), temperature=torch.ones(2),
                 top_p=_dual(torch.ones(2)), u=torch.zeros(2))
        with pytest.raises(ValueError, match="device"):
            ltk.sample(**d)
        d[name] = _dual(d[name])
        with pytest.raises(NotImplementedError, match="sample_logits"):
            ltk.sample(**d)
        out = torch.zeros(2, dtype=torch.int64), torch.zeros(2)
        with pytest.raises(ValueError, match="device"):
            ltk.sample(**d, out=out)
