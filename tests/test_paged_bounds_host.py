"""The bounds of bounds_util catch a tenth of the V rows left out, and a few, where the coarser bound of
paged_util does not; and they hold for a model of the kernel's roundings."""
import math

import numpy as np
import pytest
import torch

import bounds_util as bu
import paged_util as pu


def inputs(dtype, n, D, seed=1):
    _, _, _, k, v = pu.make_cache(seed, [n], 1, D, 64, dtype)
    q = torch.randn((1, 2, 1, D), generator=torch.Generator().manual_seed(seed + 1)).to(pu.DT[dtype]).double().numpy()
    return q, k, v, 1 / math.sqrt(D)


@pytest.mark.parametrize("dtype,dropped", [("bf16", 500), ("bf16", 128), ("fp16", 500), ("fp16", 32)])
def test_planted_mistake_in_the_statement_is_caught(dtype, dropped):
    q, k, v, scale = inputs(dtype, 5001, 64)
    args = (q, k, v, [5000], [1], None, scale)
    o, lse, bound = bu.attention(*args, dtype)
    ref, rl = pu.attention(*args)
    assert np.allclose(o, ref, atol=1e-12) and np.allclose(lse, rl)
    wrong, _, _ = bu.attention(*args, dtype, drop=np.arange(1000, 1000 + dropped))
    assert (np.abs(wrong - o) > 2 * bound).any()
    if dtype == "bf16":
        assert np.abs(wrong - o).max() <= pu.tolerances(q, k, v, dtype, scale)[0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 40, 3000])
def test_bounds_hold_for_rounded_weights(dtype, n):
    q, k, v, scale = inputs(dtype, n, 64, seed=5)
    o, _, bound = bu.attention(q, k, v, [n - 1], [1], None, scale, dtype)
    for h in range(2):
        s = torch.from_numpy(k[0][0]).float() @ torch.from_numpy(q[0, h, 0]).float() * scale
        p = torch.exp(s - s.max())
        got = (p.to(pu.DT[dtype]).float() @ torch.from_numpy(v[0][0]).float() / p.sum()).to(pu.DT[dtype]).double().numpy()
        assert (np.abs(got - o[0, h, 0]) <= bound[0, h, 0]).all()
