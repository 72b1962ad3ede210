"""The ends of a decoding step's numbers on the GPU, against the float64
oracle: tokens whose weight is next to nothing, and norm weights of the rows'
own type at both ends of its range.

Bounds are those of the calls' own tests.
"""
import numpy as np
import pytest
import torch

import test_gpu_sample as smp

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
