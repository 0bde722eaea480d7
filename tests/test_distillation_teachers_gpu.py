"""A teacher's logits of any magnitude: the lowest float is a logit, and what is a float times the scale need not be one."""

import numpy as np
import pytest

from helpers import log
from logits_bounds import distillation as expected
from logits_bounds import within
from test_distillation_gpu import Case
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu

LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("scale", [0.5, 1.0, 2.0, 2.0 ** 20])
def test_the_ends_of_floats(dtype, scale):
    import torch
    log(f"CASE {dtype} {scale}")
    c = Case(dtype, 12, 32, 300, top=4, masked=0.0, spread=2.0 / scale, scale=scale)
    c.ids = np.stack([np.random.default_rng(i).permutation(300)[:4] for i in range(12)])
    rows = [[LOWEST] * 4, [LOWEST, -np.inf, -np.inf, -np.inf], [3e38, 2e38, 1e38, 0.0], [3.4e38, LOWEST, 0.0, -np.inf],
            [LOWEST, LOWEST, 1e30, 5.0], [-3e38, -3e38, LOWEST, -np.inf], [1e25, 1e25, 1e25, 1e25], [0.0, LOWEST, LOWEST, LOWEST],
            [-1e33, -1e33, -1e38, LOWEST], [1.0, 2.0, 3.0, LOWEST], [LOWEST / 2, LOWEST / 2, LOWEST, LOWEST],
            [3.0, 3.0, -np.inf, -np.inf]]
    c.teacher = np.array(rows, dtype=np.float32)
    if scale == 2.0 ** 20:
        c.teacher[[9, 11]] *= 2.0 ** -20
    o = c.run()
    # equal largest logits, or one far ahead: p has no rounding of the logits' in it
    t = np.where(np.isneginf(c.teacher), -np.inf, c.teacher.astype(np.float64))
    small = t.copy()
    for i in range(12):
        if i not in (9, 11):
            small[i] = np.where(t[i] == t[i].max(), 0.0, -1e4 / scale)
            small[i][np.isneginf(t[i])] = -np.inf
    want = expected(c.X.double().numpy(), c.W.double().numpy(), c.ids, small, c.scale, c.dloss, dtype == am.BF16)
    for x, name in zip(o, ("loss", "lse", "dX", "dW")):
        assert torch.isfinite(x).all(), name
        within(name, x, *want[name])
