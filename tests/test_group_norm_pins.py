"""The fp64 oracle of group norm: a case by hand, differences for its gradients; and the library's
refusals, which need no GPU."""

import ctypes

import numpy as np
import pytest

from oracle import group_norm as gn
from test_learned_neural_amd import atlasmem as am


def test_two_groups_by_hand():
    x = np.array([[[1.0, 3.0, 5.0, 5.0]]])
    y, mean, rstd = gn.forward(x, 2, np.array([1.0, 2.0, 1.0, 1.0]), np.array([0.0, 1.0, 0.5, -0.5]), 0.0 + 1e-30, False)
    assert np.allclose(mean, [[2.0, 5.0]])
    assert np.allclose(y, [[[-1.0, 3.0, 0.5, -0.5]]])
    assert np.isclose(rstd[0, 0], 1.0)


@pytest.mark.parametrize("silu", [False, True])
def test_gradients_against_differences(silu):
    rng = np.random.default_rng(0)
    n, L, C, G = 2, 3, 6, 2
    x, dy = rng.standard_normal((2, n, L, C))
    gamma, beta = rng.standard_normal((2, C))
    grads = gn.backward(x, dy, G, gamma, beta, 1e-3, silu)
    args = [x, gamma, beta]
    for which, (a, grad) in enumerate(zip(args, grads)):
        for i in np.ndindex(a.shape):
            vals = []
            for h in (1e-6, -1e-6):
                p = [b.copy() for b in args]
                p[which][i] += h
                vals.append((gn.forward(p[0], G, p[1], p[2], 1e-3, silu)[0] * dy).sum())
            d = (vals[0] - vals[1]) / 2e-6
            assert abs(d - grad[i]) <= 1e-6 * (1 + abs(d)), (which, i)


FAR = 1 << 32


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), am.E_INVALID), (dict(Y=None), am.E_INVALID), (dict(dtype=3), am.E_INVALID),
    (dict(act=2), am.E_INVALID), (dict(n=-1), am.E_INVALID), (dict(L=0), am.E_INVALID), (dict(C=0), am.E_INVALID),
    (dict(G=0), am.E_INVALID), (dict(G=3), am.E_INVALID), (dict(eps=-1.0), am.E_INVALID),
    (dict(eps=float("nan")), am.E_INVALID), (dict(C=1 << 17, G=1), am.E_SHAPE),
    (dict(n=1 << 30, G=8), am.E_SHAPE), (dict(L=1 << 40), am.E_SHAPE),
    (dict(L=5000, ws=None), am.E_INVALID), (dict(L=5000, bytes=16), am.E_INVALID),
    (dict(L=5000, ws=7 * FAR + 4), am.E_INVALID),        # not aligned
    (dict(Y=FAR + 32), am.E_INVALID),                    # partly over X
    (dict(mean=5 * FAR, rstd=5 * FAR), am.E_INVALID),    # two outputs in one place
    (dict(mean=2 * FAR), am.E_INVALID),                  # over Y
    (dict(n=0), am.OK), (dict(n=0, X=None, Y=None), am.OK),
])
def test_forward_refusals(kw, status):
    a = dict(X=FAR, dtype=am.F32, n=4, L=1, C=32, G=4, gamma=3 * FAR, beta=4 * FAR, eps=1e-5, act=0, Y=2 * FAR,
             mean=5 * FAR, rstd=6 * FAR, ws=7 * FAR, bytes=1 << 31)
    a.update(kw)
    st = am.load().atlasmem_group_norm(a["X"], a["dtype"], a["n"], a["L"], a["C"], a["G"], a["gamma"], a["beta"],
                                       ctypes.c_float(a["eps"]), a["act"], a["Y"], a["mean"], a["rstd"], a["ws"],
                                       a["bytes"], None)
    assert st == status


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), am.E_INVALID), (dict(dY=None), am.E_INVALID), (dict(mean=None), am.E_INVALID),
    (dict(rstd=None), am.E_INVALID), (dict(dX=None), am.E_INVALID), (dict(ws=None), am.E_INVALID),
    (dict(bytes=16), am.E_INVALID), (dict(dX=FAR + 16), am.E_INVALID), (dict(dX=2 * FAR + 4), am.E_INVALID),
    (dict(dgamma=8 * FAR, dbeta=8 * FAR), am.E_INVALID), (dict(dgamma=3 * FAR), am.E_INVALID),
    (dict(G=5), am.E_INVALID),
])
def test_backward_refusals(kw, status):
    a = dict(X=FAR, dY=2 * FAR, n=4, L=1, C=32, G=4, gamma=3 * FAR, beta=4 * FAR, mean=5 * FAR, rstd=6 * FAR,
             dX=7 * FAR, dgamma=8 * FAR, dbeta=9 * FAR, ws=10 * FAR, bytes=1 << 31)
    a.update(kw)
    st = am.load().atlasmem_group_norm_backward(a["X"], a["dY"], am.F32, a["n"], a["L"], a["C"], a["G"], a["gamma"],
                                                a["beta"], a["mean"], a["rstd"], 0, a["dX"], a["dgamma"], a["dbeta"],
                                                a["ws"], a["bytes"], None)
    assert st == status


def test_workspace_bytes():
    assert am.group_norm_workspace_bytes(100, 1, 256, 4) == 0
    assert am.group_norm_workspace_bytes(2, 4096, 512, 32) > 0
    assert am.group_norm_workspace_bytes(100, 1, 256, 4, True) > 0
    assert am.group_norm_workspace_bytes(100, 1, 256, 3) == -1
    assert am.group_norm_workspace_bytes(100, 0, 256, 4) == -1
