"""The fp64 oracle of linear attention: a case by hand, differences for its gradients; and the
library's refusals, which need no GPU."""

import ctypes

import numpy as np
import pytest

from oracle import linear_attention as la
from test_learned_neural_amd import atlasmem as am


def test_two_tokens_by_hand():
    q = np.array([[[[1.0, 2.0], [3.0, -1.0]]]])
    k = np.array([[[[1.0, 0.0], [0.5, 2.0]]]])
    v = np.array([[[[2.0], [4.0]]]])
    W0 = np.array([[[[8.0, 0.0]]]])
    y, W = la.forward(q, k, v, [np.log(0.5)], 0.1, W0)
    # W_1 = [4, 0] + [2, 0] = [6, 0], y = 0.6;  W_2 = [3, 0] + [2, 8] = [5, 8], y = 0.1 (15 - 8)
    assert np.allclose(y[0, 0, :, 0], [0.6, 0.7])
    assert np.allclose(W, [[[[5.0, 8.0]]]])


def test_nothing_is_kept_without_memory():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((1, 1, 4, 3)) for _ in range(3))
    y, _ = la.forward(q, k, v, [-np.inf], 1.0, rng.standard_normal((1, 1, 3, 3)))
    own = (q * k).sum(-1, keepdims=True) * v
    assert np.allclose(y, own)


@pytest.mark.parametrize("lengths", [None, [3, 0], [5, 2]])
def test_gradients_against_differences(lengths):
    rng = np.random.default_rng(1)
    B, H, T, dk, dv = 2, 2, 5, 3, 4
    q, k = rng.standard_normal((2, B, H, T, dk))
    v, dy = rng.standard_normal((2, B, H, T, dv))
    W0, dW = rng.standard_normal((2, B, H, dv, dk))
    g = np.array([-0.3, -1.1])
    args = {"q": q, "k": k, "v": v, "g": g, "W0": W0}

    def loss(a):
        y, W = la.forward(a["q"], a["k"], a["v"], a["g"], 0.7, a["W0"], lengths)
        return (y * dy).sum() + (W * dW).sum()

    grads = dict(zip(("q", "k", "v", "W0", "g"), la.backward(q, k, v, g, 0.7, W0, dy, dW, lengths)))
    for name, x in args.items():
        for i in np.ndindex(x.shape):
            h = 1e-6
            up, down = dict(args), dict(args)
            up[name], down[name] = x.copy(), x.copy()
            up[name][i] += h
            down[name][i] -= h
            d = (loss(up) - loss(down)) / (2 * h)
            assert abs(d - grads[name][i]) <= 1e-7 * (1 + abs(d)), (name, i)


def call(**kw):
    """A call whose pointers are never followed: apart from each other unless given."""
    a = dict(Q=1 << 20, K=2 << 20, V=3 << 20, dtype=am.F32, batch=1, heads=2, T=20, dk=8, dv=8, layout=am.HEADS_FIRST,
             g=4 << 20, lengths=None, scale=1.0, W0=5 << 20, Y=6 << 20, W_T=7 << 20, ws=8 << 20, bytes=1 << 30)
    a.update(kw)
    return am.load().atlasmem_linear_attention(
        a["Q"], a["K"], a["V"], a["dtype"], a["batch"], a["heads"], a["T"], a["dk"], a["dv"], a["layout"], a["g"],
        a["lengths"], ctypes.c_float(a["scale"]), a["W0"], a["Y"], a["W_T"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), am.E_INVALID), (dict(K=None), am.E_INVALID), (dict(V=None), am.E_INVALID),
    (dict(Y=None), am.E_INVALID), (dict(g=None), am.E_INVALID), (dict(dtype=2), am.E_INVALID),
    (dict(layout=2), am.E_INVALID), (dict(batch=0), am.E_INVALID), (dict(heads=0), am.E_INVALID),
    (dict(T=-1), am.E_INVALID), (dict(dk=0), am.E_INVALID), (dict(dv=-3), am.E_INVALID),
    (dict(dk=129), am.E_SHAPE), (dict(dv=129), am.E_SHAPE), (dict(batch=1 << 11, heads=1 << 10), am.E_SHAPE),
    (dict(heads=(1 << 16) + 1), am.E_SHAPE),
    (dict(T=1 << 31), am.E_SHAPE),
    (dict(T=5000, ws=None), am.E_INVALID), (dict(T=5000, bytes=100), am.E_INVALID),
    (dict(T=5000, ws=(9 << 30) + 8), am.E_INVALID),  # not aligned
    (dict(Y=(1 << 20) + 64), am.E_INVALID),          # over Q
    (dict(Y=(3 << 20)), am.E_INVALID),               # over V
    (dict(W_T=(5 << 20) + 16), am.E_INVALID),        # W_T inside W0, but not W0 itself
    (dict(W_T=6 << 20), am.E_INVALID),               # W_T over Y
    (dict(T=5000, Y=4 << 30, ws=5 << 20), am.E_INVALID),  # workspace over W0
])
def test_forward_refusals(kw, status):
    assert call(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dY=None), am.E_INVALID), (dict(dQ=None), am.E_INVALID), (dict(dK=None), am.E_INVALID),
    (dict(dV=None), am.E_INVALID), (dict(ws=None), am.E_INVALID), (dict(bytes=8), am.E_INVALID),
    (dict(dQ=1 << 20), am.E_INVALID), (dict(dV=13 << 20), am.E_INVALID), (dict(dW0=(9 << 20) + 4), am.E_INVALID),
    (dict(dk=200), am.E_SHAPE), (dict(T=-2), am.E_INVALID),
])
def test_backward_refusals(kw, status):
    a = dict(Q=1 << 20, K=2 << 20, V=3 << 20, T=20, dk=8, W0=5 << 20, dY=8 << 20, dW_T=9 << 20, dQ=11 << 20,
             dK=12 << 20, dV=13 << 20, dW0=14 << 20, dg=15 << 20, ws=16 << 20, bytes=1 << 30)
    if kw.get("dV") == 13 << 20:
        kw = dict(dK=13 << 20)                        # two outputs in one place
    a.update(kw)
    st = am.load().atlasmem_linear_attention_backward(
        a["Q"], a["K"], a["V"], am.F32, 1, 2, a["T"], a["dk"], 8, 0, 4 << 20, None, ctypes.c_float(1.0), a["W0"],
        a["dY"], a["dW_T"], a["dQ"], a["dK"], a["dV"], a["dW0"], a["dg"], a["ws"], a["bytes"], None)
    assert st == status


def test_workspace_bytes():
    assert am.linear_attention_workspace_bytes(am.BF16, 1, 8, 1, 64, 64) == 0          # single tokens need none
    assert am.linear_attention_workspace_bytes(am.BF16, 1, 1, 100000, 64, 64) > 0
    assert am.linear_attention_workspace_bytes(am.BF16, 1, 8, 0, 64, 64, True) > 0
    assert am.linear_attention_workspace_bytes(am.BF16, 1, 8, 8, 129, 64) == -1
    assert am.linear_attention_workspace_bytes(7, 1, 8, 8, 64, 64) == -1
