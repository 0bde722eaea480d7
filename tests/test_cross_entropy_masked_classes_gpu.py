"""Classes that are masked by the weight of a column of ones: minus infinity, the type's lowest value or a
large negative one.  Their probability is zero, and everything else is as if they were not there; the bounds are
those of the classes that are left."""

import numpy as np
import pytest

from helpers import DEV, log
from test_cross_entropy_gpu import Case
from test_learned_neural_amd import atlasmem as am
from xent_bounds import expected, within

pytestmark = pytest.mark.gpu


def masked_case(dtype, n, d, vocab, value, seed=0):
    import torch
    c = Case(dtype, n, d, vocab, seed=seed)
    rng = np.random.default_rng(seed + 1)
    masked = rng.random(vocab) < 0.1
    masked[[0, vocab - 1]] = True
    keep = np.flatnonzero(~masked)
    c.X[:, -1] = 1.0
    c.W[torch.from_numpy(masked), -1] = value if value is not None else torch.finfo(c.W.dtype).min
    live = c.labels >= 0
    c.labels[live] = keep[rng.integers(0, len(keep), live.sum())]
    return c, keep


@pytest.mark.parametrize("value", [-np.inf, None, -1e30], ids=["infinity", "lowest", "large"])
@pytest.mark.parametrize("dtype,n,d,vocab", [(am.F32, 60, 40, 500), (am.F32, 1300, 64, 3001), (am.BF16, 300, 64, 700)])
def test_masked_classes_are_not_there(dtype, n, d, vocab, value):
    import torch
    c, keep = masked_case(dtype, n, d, vocab, value)
    log(f"CASE masked classes {c.size()} {value}")
    loss, lse, dX, dW = (x.double().cpu().numpy() for x in c.run())
    place = np.full(vocab, -1)
    place[keep] = np.arange(len(keep))
    labels = np.where(c.labels >= 0, place[np.maximum(c.labels, 0)], -100)
    want = expected(c.X.double().numpy(), c.W.double().numpy()[keep], labels, c.dloss, dtype == am.BF16,
                    plain32=dtype == am.F32)
    within("loss", loss, *want["loss"])
    within("lse", lse, *want["lse"])
    within("dW", dW[keep], *want["dW"])
    out = np.setdiff1d(np.arange(vocab), keep)
    assert not dW[out].any()
    # the gradient of the column of ones takes G = 0 times minus infinity
    cols = slice(None) if value != -np.inf else slice(0, d - 1)
    # a masked class adds zeros to the sum, and rounds nothing
    within("dX", dX[:, cols], want["dX"][0][:, cols], want["dX"][1][:, cols])


@pytest.mark.parametrize("dtype", [am.F32, am.BF16])
def test_infinite_logits_are_as_the_definition_has_them(dtype):
    """A class of plus infinity for one row alone: that row has no finite loss, the others do."""
    import torch
    c = Case(dtype, 70, 16, 200, masked=0.0)
    c.X[:, -1] = 0.5
    c.X[9, -1] = -0.25
    c.W[50, -1] = -np.inf
    c.labels[c.labels == 50] = 49
    loss = c.run()[0]
    bad = ~torch.isfinite(loss.cpu())
    assert bad[9] and int(bad.sum()) == 1
