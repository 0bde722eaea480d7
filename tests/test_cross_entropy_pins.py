"""The fp64 oracle of the cross entropy: a case by hand, differences for its gradients; and the
library's refusals, which need no GPU."""

import numpy as np
import pytest

from oracle import cross_entropy as ce
from test_learned_neural_amd import atlasmem as am


def test_by_hand():
    X, W = np.array([[1.0], [2.0], [5.0]]), np.array([[0.0], [np.log(3.0)]])
    loss, lse = ce.forward(X, W, np.array([1, 0, -100]))
    assert np.allclose(loss, [np.log(4.0 / 3.0), np.log(10.0), 0.0])
    assert np.allclose(lse, [np.log(4.0), np.log(10.0), 0.0])
    dX, dW = ce.backward(X, W, np.array([1, 0, -100]), np.array([2.0, 1.0, 7.0]))
    assert np.allclose(dX, [[-0.5 * np.log(3.0)], [0.9 * np.log(3.0)], [0.0]])
    assert np.allclose(dW, [[0.5 - 1.8], [-0.5 + 1.8]])


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    X, W = rng.standard_normal((6, 4)), rng.standard_normal((5, 4))
    labels, w = np.array([0, 4, 2, -1, 5, 2]), rng.standard_normal(6)
    grads = ce.backward(X, W, labels, w)
    for which, a in enumerate((X, W)):
        for i in np.ndindex(a.shape):
            vals = []
            for h in (1e-6, -1e-6):
                p = [X.copy(), W.copy()]
                p[which][i] += h
                vals.append((ce.forward(p[0], p[1], labels)[0] * w).sum())
            d = (vals[0] - vals[1]) / 2e-6
            assert abs(d - grads[which][i]) <= 1e-7 * (1 + abs(d))


FAR = 1 << 36


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), am.E_INVALID), (dict(W=None), am.E_INVALID), (dict(labels=None), am.E_INVALID),
    (dict(loss=None), am.E_INVALID), (dict(lse=None), am.E_INVALID), (dict(ws=None), am.E_INVALID),
    (dict(bytes=100), am.E_INVALID), (dict(ws=6 * FAR + 8), am.E_INVALID), (dict(dtype=9), am.E_INVALID), (dict(n=-1), am.E_INVALID),
    (dict(d=0), am.E_INVALID), (dict(vocab=0), am.E_INVALID), (dict(d=16385), am.E_SHAPE),
    (dict(vocab=1 << 25), am.E_SHAPE), (dict(n=1 << 25), am.E_SHAPE),
    (dict(n=1 << 24, d=1, vocab=1 << 14), am.E_SHAPE), (dict(n=1 << 23, d=1, vocab=(1 << 14) + 1), am.E_SHAPE),
    (dict(n=1 << 20, vocab=1 << 19), am.E_SHAPE), (dict(d=1 << 14, vocab=1 << 20), am.E_SHAPE),
    (dict(lse=4 * FAR), am.E_INVALID), (dict(loss=FAR + 8), am.E_INVALID), (dict(ws=2 * FAR), am.E_INVALID),
    (dict(n=0), am.OK), (dict(n=0, X=None, W=None, labels=None, loss=None, lse=None, ws=None), am.OK),
])
def test_forward_refusals(kw, status):
    a = dict(X=FAR, W=2 * FAR, dtype=am.F32, n=40, d=16, vocab=100, labels=3 * FAR, loss=4 * FAR, lse=5 * FAR,
             ws=6 * FAR, bytes=1 << 30)
    a.update(kw)
    assert am.load().atlasmem_cross_entropy(a["X"], a["W"], a["dtype"], a["n"], a["d"], a["vocab"], a["labels"],
                                            a["loss"], a["lse"], a["ws"], a["bytes"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), am.E_INVALID), (dict(lse=None), am.E_INVALID), (dict(ws=None), am.E_INVALID),
    (dict(bytes=100), am.E_INVALID), (dict(dX=FAR), am.E_INVALID), (dict(dW=2 * FAR), am.E_INVALID),
    (dict(dX=8 * FAR, dW=8 * FAR), am.E_INVALID), (dict(dX=None, dW=None), am.OK), (dict(d=20000), am.E_SHAPE),
])
def test_backward_refusals(kw, status):
    a = dict(X=FAR, W=2 * FAR, n=40, d=16, vocab=100, labels=3 * FAR, lse=5 * FAR, dloss=7 * FAR, dX=8 * FAR,
             dW=9 * FAR, ws=6 * FAR, bytes=1 << 30)
    a.update(kw)
    assert am.load().atlasmem_cross_entropy_backward(a["X"], a["W"], am.BF16, a["n"], a["d"], a["vocab"], a["labels"],
                                                     a["lse"], a["dloss"], a["dX"], a["dW"], a["ws"], a["bytes"],
                                                     None) == status


def test_workspace_is_far_below_the_logits():
    n, d, vocab = 65536, 2048, 131072
    assert am.cross_entropy_workspace_bytes(am.BF16, n, d, vocab, True) < 4 * n * vocab // 10
    assert am.cross_entropy_workspace_bytes(am.BF16, n, d, vocab, False) > 0
    assert am.cross_entropy_workspace_bytes(am.BF16, 0, d, vocab, True) >= 0
    assert am.cross_entropy_workspace_bytes(am.BF16, n, 0, vocab) == -1
    assert am.cross_entropy_workspace_bytes(5, n, d, vocab) == -1
