"""The gradients of rows that are left out are zero, whatever the classes hold: a mask of minus infinity, or NaN."""

import numpy as np
import pytest

from helpers import log
from test_distillation_gpu import Case
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu

# vocabularies whose products with W are one piece, and cut; rows as they come, and gathered
SIZES = [(1, 24, 300), (40, 32, 600), (140, 32, 600), (300, 37, 900), (50, 64, 5003), (333, 384, 5003), (2100, 1032, 12001)]


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("value", [-float("inf"), float("nan")])
@pytest.mark.parametrize("n,d,vocab", SIZES)
def test_left_out_rows_have_no_gradient(dtype, value, n, d, vocab):
    import torch
    log(f"CASE {dtype} {n} {d} {vocab} {value}")
    c = Case(dtype, n, d, vocab, top=3, masked=0.4)
    c.ids[0] = -1
    c.X[:, 7] = 1.0
    c.W[:, 7] = 0.0
    c.W[np.arange(vocab) % 3 == 1, 7] = value
    off = ~((c.ids >= 0) & (c.ids < vocab) & (c.teacher != -np.inf)).any(1)
    o = c.run()
    off = torch.from_numpy(off).to(o[2].device)
    for x in o[:3]:
        assert not (x[off] != 0).any()
