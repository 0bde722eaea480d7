"""Linear attention where a workgroup walks many chunks: every LDS buffer is used many times, the state is
carried far, and the outputs of the parts of a wide x take turns.  Many memories (one segment each, the state
also in place), and fewer ones with several segments of many chunks.  Two sequences are compared with the fp64
oracle; the others' adjoints are zero, so that the decays' gradients are the two sequences' alone."""

import numpy as np
import pytest

from helpers import DEV, log
from oracle import linear_attention as la
from test_learned_neural_amd import atlasmem as am
from test_linear_attention_gpu import Case, state_bound, term_bound, within

pytestmark = pytest.mark.gpu

CHUNK = 32


def chunks_of_a_workgroup(c):
    """From the workspace, which holds a state for every segment where there are several."""
    states = am.linear_attention_workspace_bytes(*c.size(), False) // (4 * c.B * c.H * c.dk * c.dv)
    return -(-(-(-c.T // CHUNK)) // max(states, 1))


WIDTHS = [(64, 64), (128, 64), (64, 128), (128, 128), (72, 101)]
FORMS = {
    "one_segment": dict(B=128, H=4, T=301, least=10),
    "segments": dict(B=32, H=4, T=1500, least=8),
}


@pytest.mark.parametrize("dk,dv", WIDTHS)
@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_many_chunks(form, dtype, dk, dv):
    import torch
    f = FORMS[form]
    B, H, T = f["B"], f["H"], f["T"]
    lengths = [T - (b * 7) % 40 for b in range(B)]
    lengths[B - 1] = T - 133
    c = Case(dtype, B, H, T, dk, dv, layout=am.TOKENS_FIRST if dk == 64 else am.HEADS_FIRST, lengths=lengths, seed=dk + dv)
    assert chunks_of_a_workgroup(c) >= f["least"]
    if form == "one_segment":
        assert am.linear_attention_workspace_bytes(*c.size(), False) == 0
    at = [0, B - 1]
    others = np.setdiff1d(np.arange(B), at)
    c.host["dy"][others] = 0
    c.dW[others] = 0
    log(f"CASE many chunks {form} {c.size()} {chunks_of_a_workgroup(c)} chunks a workgroup")
    d, Y = c.tensors(), c.out(dv)
    W_T = torch.full((B, H, dv, dk), 7.0, device=DEV)
    c.forward(d, Y, W_T, c.workspace(False))
    o = c.outputs()
    c.backward(d, o, c.workspace(True))
    here = dict(d, W0=d["W0"].clone(), dW=d["dW"].clone())
    Y2, o2 = c.out(dv), c.outputs()
    o2["dW0"] = here["dW"]
    c.backward(here, o2, c.workspace(True))
    c.forward(here, Y2, here["W0"], c.workspace(False))
    torch.cuda.synchronize()
    assert torch.equal(Y, Y2) and torch.equal(W_T, here["W0"])
    assert all(torch.equal(o[n], o2[n]) for n in o)

    args = [c.f64("q")[at], c.f64("k")[at], c.f64("v")[at], c.g, c.scale, c.W0[at], c.f64("dy")[at], c.dW[at]]
    mags = [abs(x) if i not in (3, 4) else x for i, x in enumerate(args)]
    n = [lengths[b] for b in at]
    y, W = la.forward(*args[:6], n)
    ya, Wa = la.forward(*mags[:6], n)
    want, wa = la.backward(*args, n), la.backward(*mags, n)
    step = 2.0 ** -8 if dtype == am.BF16 else 2.0 ** -24
    e, es = term_bound(dtype, T, max(dk, dv)), state_bound(T, max(dk, dv))
    within("Y", c.np64(Y)[at], y, ya, step, e)
    within("W_T", W_T.double().cpu().numpy()[at], W, Wa, 2.0 ** -24, es)
    for i, name in enumerate(("dQ", "dK", "dV")):
        g = c.np64(o[name])
        within(name, g[at], want[i], wa[i], step, e)
        assert not g[others].any(), name
    dW0 = o["dW0"].double().cpu().numpy()
    within("dW0", dW0[at], want[3], wa[3], 2.0 ** -24, es)
    assert not dW0[others].any()
    within("dlog_decay", o["dlog_decay"].double().cpu().numpy(), want[4], wa[4], 2.0 ** -24, 2 * es)
