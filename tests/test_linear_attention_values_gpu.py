"""Linear attention with values that are no ordinary numbers: a NaN or infinity of one token reaches what the
recurrence lets it reach, and nothing before it (behind it for the adjoints)."""

import numpy as np
import pytest

from helpers import DEV, log
from test_learned_neural_amd import atlasmem as am
from test_linear_attention_gpu import Case
from test_linear_attention_largest_gpu import run

pytestmark = pytest.mark.gpu


# what a bad value of token t and column c may reach: tokens (from t on, up to t, t alone), and its column or all
REACH = {
    "v": {"Y": ("on", True), "dQ": ("on", False), "dK": ("at", False), "dV": None},
    "k": {"Y": ("on", False), "dQ": ("on", True), "dV": ("at", False), "dK": None},
    "q": {"Y": ("at", False), "dK": ("upto", True), "dV": ("upto", False), "dQ": None},
    "dy": {"dQ": ("at", False), "dK": ("upto", False), "dV": ("upto", True), "Y": None},
}
SHAPES = [
    dict(dtype=am.BF16, B=1, H=2, T=100, dk=64, dv=64),
    dict(dtype=am.F32, B=1, H=2, T=100, dk=64, dv=64),
    dict(dtype=am.BF16, B=2, H=1, T=333, dk=128, dv=40, lengths=[333, 290], layout=am.TOKENS_FIRST),
    dict(dtype=am.BF16, B=1, H=1, T=150, dk=37, dv=100),
    dict(dtype=am.F32, B=1, H=1, T=150, dk=128, dv=128),
    dict(dtype=am.F32, B=1, H=2, T=90, dk=33, dv=101),
    dict(dtype=am.BF16, B=1, H=2, T=12, dk=64, dv=64),
]


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("which", sorted(REACH))
@pytest.mark.parametrize("kw", SHAPES, ids=[f"{s['dtype']}x{s['T']}x{s['dk']}x{s['dv']}" for s in SHAPES])
def test_a_bad_value_reaches_no_token_that_it_should_not(kw, which, value):
    clean, c = Case(**kw), Case(**kw)
    T = kw["T"]
    t, col = (T * 2) // 3, 5
    c.host[which][0, 0, t, col] = value
    log(f"CASE {value} in {which} {c.size()} token {t}")
    a, b = run(clean), run(c)
    for name, reach in REACH[which].items():
        bad = np.zeros(a[name].shape, dtype=bool)
        if reach is not None:
            tokens = {"on": slice(t, None), "upto": slice(None, t + 1), "at": slice(t, t + 1)}[reach[0]]
            bad[0, 0, tokens, col if reach[1] else slice(None)] = True
        assert np.array_equal(a[name][~bad], b[name][~bad]), name
        if reach is not None and c.lengths is None:
            assert not np.isfinite(b[name][0, 0, t]).all(), name
    # the state takes it in and the other memories do not
    if which in ("k", "v"):
        assert not np.isfinite(b["W_T"][0, 0]).all()
        keep = np.ones(c.dv, dtype=bool)
        keep[col] = which != "v"
        if which == "v":
            assert np.array_equal(a["W_T"][0, 0][keep], b["W_T"][0, 0][keep])
    else:
        assert np.array_equal(a["W_T"], b["W_T"])
    others = np.ones(a["W_T"].shape[:2], dtype=bool)
    others[0, 0] = False
    for name in ("W_T", "dW0", "Y", "dQ", "dK", "dV"):
        assert np.array_equal(a[name][others], b[name][others]), name


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("B,T,dk,dv", [(64, 203, 128, 64), (1, 900, 64, 128), (64, 170, 50, 23)])
def test_many_bad_values_over_many_chunks(dtype, B, T, dk, dv):
    """In V, and for the gradients in Q: each column of one memory is clean up to its first (behind its last) one,
    and bad from there on."""
    kw = dict(dtype=dtype, B=B, H=8, T=T, dk=dk, dv=dv)
    clean = run(Case(**kw))
    rng = np.random.default_rng(T)
    log(f"CASE many bad values {kw}")
    for which, name, w in (("v", "Y", dv), ("q", "dK", dk)):
        c = Case(**kw)
        t, col = rng.integers(0, T, 25), rng.integers(0, w, 25)
        t[:3], col[:3] = (0, T - 1, T // 2), (0, w - 1, w // 2)
        for i in range(25):
            c.host[which][B - 1, 7, t[i], col[i]] = (np.nan, np.inf, -np.inf)[i % 3]
        got = run(c)
        bad = np.zeros(got[name].shape, dtype=bool)
        for i in range(25):
            bad[B - 1, 7, slice(t[i], None) if which == "v" else slice(None, t[i] + 1), col[i]] = True
        assert np.array_equal(got[name][~bad], clean[name][~bad])
        assert not np.isfinite(got[name][bad]).any()
        others = np.ones((B, 8), dtype=bool)
        others[B - 1, 7] = False
        for n in ("Y", "W_T", "dQ", "dK", "dV", "dW0"):
            assert np.array_equal(got[n][others], clean[n][others]), n
