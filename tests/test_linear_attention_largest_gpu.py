"""The lowest and largest finite floats are values of linear attention like others."""

import pytest

from helpers import DEV, log
from oracle import linear_attention as la
from test_learned_neural_amd import atlasmem as am
from test_linear_attention_gpu import Case, state_bound, term_bound, within

pytestmark = pytest.mark.gpu


def run(c):
    import torch
    d, Y = c.tensors(), c.out(c.dv)
    W_T = torch.full((c.B, c.H, c.dv, c.dk), 7.0, device=DEV)
    c.forward(d, Y, W_T, c.workspace(False))
    o = c.outputs()
    c.backward(d, o, c.workspace(True))
    torch.cuda.synchronize()
    got = {"Y": c.np64(Y), "W_T": W_T.double().cpu().numpy()}
    got.update({n: c.np64(o[n]) if n in ("dQ", "dK", "dV") else o[n].double().cpu().numpy() for n in o})
    return got


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("which", ["v", "k", "q", "dy"])
@pytest.mark.parametrize("T", [10, 100])
@pytest.mark.parametrize("dtype", [am.F32, am.BF16])
def test_the_largest_finite_values(dtype, T, which, sign):
    """The other operand is small enough for every product and sum to stay below the largest float."""
    import torch
    c = Case(dtype, 1, 2, T, 64, 48, seed=3)
    for n in ("q", "k", "v", "dy"):
        if n != which:
            c.host[n] = c.host[n] * 2.0 ** -6
    c.W0, c.dW = c.W0 * 2.0 ** -6, c.dW * 2.0 ** -6
    c.host[which][0, 1, T // 2, 7] = sign * float(torch.finfo(c.host[which].dtype).max)
    log(f"CASE largest {which} {c.size()}")
    got = run(c)
    args = [c.f64("q"), c.f64("k"), c.f64("v"), c.g, c.scale, c.W0, c.f64("dy"), c.dW]
    mags = [abs(x) if i not in (3, 4) else x for i, x in enumerate(args)]
    y, W = la.forward(*args[:6])
    ya, Wa = la.forward(*mags[:6])
    step = 2.0 ** -8 if dtype == am.BF16 else 2.0 ** -24
    e, es = term_bound(dtype, T, 64), state_bound(T, 64)
    within("Y", got["Y"], y, ya, step, e)
    within("W_T", got["W_T"], W, Wa, 2.0 ** -24, es)
    want, wa = la.backward(*args), la.backward(*mags)
    for i, n in enumerate(("dQ", "dK", "dV")):
        within(n, got[n], want[i], wa[i], step, e)
    within("dW0", got["dW0"], want[3], wa[3], 2.0 ** -24, es)
