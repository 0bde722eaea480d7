"""Distillation's weight gradient over more rows than workgroups, of which each piece of the contraction counts."""

import numpy as np
import pytest

import logits_bounds
from test_distillation_gpu import Case
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu


def test_dw_of_many_rows():
    """1000 rows, each about 1049 times: dW is theirs with those numbers as weights.  fp32, where a lost piece of the 512
    (2e-3 of the sum) is far past the bound."""
    import torch
    n, of = (1 << 20) + 700, 1000
    rows = torch.arange(n) % of
    c, e = Case(am.F32, of, 8, 40, top=3), Case(am.F32, 1, 8, 40, top=3)
    e.n, e.X, e.W, e.ids, e.teacher = n, c.X[rows], c.W, c.ids[rows.numpy()], c.teacher[rows.numpy()]
    e.dloss = c.dloss[rows.numpy()]
    got = e.run()[3]
    X, W = c.X.double().numpy(), c.W.double().numpy()
    times = np.bincount(rows.numpy(), minlength=of).astype(np.float64)
    want, bound = logits_bounds.distillation(X, W, c.ids, c.teacher.astype(np.float64), c.scale, c.dloss * times, False)["dW"]
    # beside that bound's sum over 1000 rows: the sums of 2049 rows a piece, 6 roundings for 16 of them, and of 512 pieces
    G = np.abs(logits_bounds.ds.gradient_of_logits(X, W, c.ids, c.teacher.astype(np.float64), c.scale)
               * (c.dloss * times)[:, None])
    bound = bound + (6 * (2049 // 16 + 1) + 512) * logits_bounds.U * (G.T @ np.abs(X))
    assert float((bound / (G.T @ np.abs(X))).max()) < 1e-3
    logits_bounds.within("dW", got, want, bound)
