"""The gradient of W with a weight of its own for every row: one rounding of G, weights and all, and no other
before the output's.  Rows that share no column leave one product in every element, so that roundings do not
average."""

import numpy as np
import pytest

from helpers import DEV, log
from test_cross_entropy_gpu import Case
from test_learned_neural_amd import atlasmem as am
from xent_bounds import U, expected, within

pytestmark = pytest.mark.gpu


def apart(dtype, rows, each, vocab, seed=0):
    """Rows that share no column."""
    import torch
    c = Case(dtype, rows, rows * each, vocab, masked=0.0, seed=seed)
    on = torch.zeros(c.X.shape, dtype=torch.bool)
    for i in range(rows):
        on[i, i * each:(i + 1) * each] = True
    c.X = torch.where(on, c.X, torch.zeros_like(c.X))
    return c


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("equal", [False, True])
def test_one_rounding_of_a_single_product(dtype, equal):
    c = apart(dtype, 8, 32, 300)
    if equal:
        c.dloss = np.where(np.arange(c.n) % 2, 0.37, -0.37).astype(np.float32)
    log(f"CASE weights {c.size()} equal {equal}")
    got = c.run()
    want = expected(c.X.double().numpy(), c.W.double().numpy(), c.labels, c.dloss, dtype == am.BF16)
    for i, name in enumerate(("loss", "lse", "dX", "dW")):
        within(name, got[i], *want[name])


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_dw_alone_and_with_dx_are_the_same_bits(dtype):
    import torch
    c = Case(dtype, 300, 64, 700)
    a, t, ws = c.run(), c.tensors(), c.workspace(True)
    for want_dX in (True, False):
        o = c.outputs()
        am.cross_entropy_backward(t[0], t[1], *c.size(), t[2], a[1], t[3], o[2] if want_dX else None, o[3], ws)
        torch.cuda.synchronize()
        assert torch.equal(o[3], a[3])


def test_weights_of_a_kind():
    """Weights of one size (and either sign), weights with zeros among them, one large weight, no weights:
    each against the same weights given to every row by hand."""
    import torch
    c = Case(am.BF16, 200, 64, 500, masked=0.3)
    rng = np.random.default_rng(5)
    for name, w in (("signs", np.where(rng.random(200) < 0.5, 0.3, -0.3)), ("zeros", np.where(rng.random(200) < 0.5, 0.3, 0.0)),
                    ("all_zero", np.zeros(200)), ("one_large", np.where(np.arange(200) == 7, 1e4, 1e-3)),
                    ("tiny", np.full(200, 1e-20)), ("none", None)):
        c.dloss = None if w is None else w.astype(np.float32)
        log(f"CASE weights of a kind: {name}")
        got = c.run()
        want = expected(c.X.double().numpy(), c.W.double().numpy(), c.labels, c.dloss, True)
        within("dX", got[2], *want["dX"])
        within("dW", got[3], *want["dW"])
