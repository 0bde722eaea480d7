"""Token log probabilities and distillation where a caller may trip: calls at the same time, equal calls, memory around
what a call may write, rows with a range of weights, and a row of each kind in one call."""

import numpy as np
import pytest

import logits_bounds
from helpers import DEV
from test_distillation_gpu import Case as Distill
from test_learned_neural_amd import atlasmem as am
from test_token_logprobs_gpu import Case as Logprobs

pytestmark = pytest.mark.gpu

GUARD = 4096


def guarded(nbytes):
    """(buffer, the nbytes of it that may be written)."""
    import torch
    b = torch.full((GUARD + nbytes + GUARD,), 171, dtype=torch.uint8, device=DEV)
    return b, b[GUARD:GUARD + nbytes]


def like(x):
    import torch
    b, v = guarded(x.numel() * x.element_size())
    return b, v.view(x.dtype).view(x.shape)


def clean(b):
    return bool((b[:GUARD] == 171).all()) and bool((b[-GUARD:] == 171).all())


LOGPROBS = [dict(dtype=am.BF16, n=1, d=37, vocab=130, top=64), dict(dtype=am.F32, n=65, d=41, vocab=1001, top=3),
            dict(dtype=am.BF16, n=300, d=72, vocab=16007, top=20), dict(dtype=am.BF16, n=1100, d=72, vocab=16003, top=25),
            dict(dtype=am.BF16, n=2100, d=2048, vocab=24001, top=3), dict(dtype=am.F32, n=700, d=1000, vocab=24001, top=2)]
DISTILL = [dict(dtype=am.BF16, n=1, d=37, vocab=131, top=128), dict(dtype=am.F32, n=65, d=41, vocab=1001, top=3),
           dict(dtype=am.BF16, n=1100, d=72, vocab=16003, top=8, spread=20.0),
           dict(dtype=am.BF16, n=4500, d=40, vocab=300, top=20), dict(dtype=am.F32, n=1300, d=24, vocab=140, top=2),
           dict(dtype=am.BF16, n=2100, d=1032, vocab=12001, top=16), dict(dtype=am.F32, n=500, d=400, vocab=24001, top=2)]


@pytest.mark.parametrize("kw", LOGPROBS)
def test_logprobs_write_what_is_theirs(kw):
    import torch
    c = Logprobs(**kw)
    a = c.run()
    outs, t = [like(x) for x in c.outputs()], [like(x) for x in c.tensors()]
    for (_, v), x in zip(t, c.tensors()):
        v.copy_(x)
    w, ws = guarded(am.token_logprobs_workspace_bytes(*c.size(), c.top))
    c.call([v for _, v in t], [v for _, v in outs], ws)
    torch.cuda.synchronize()
    assert all(clean(b) for b, _ in outs + t) and clean(w)
    assert all(torch.equal(x, v) for x, (_, v) in zip(a, outs))
    assert all(torch.equal(x, v) for x, (_, v) in zip(c.tensors(), t))


@pytest.mark.parametrize("kw", DISTILL)
def test_distillation_writes_what_is_its_own(kw):
    import torch
    c = Distill(**kw)
    a = c.run()
    outs, t = [like(x) for x in c.outputs()], [like(x) for x in c.tensors()]
    for (_, v), x in zip(t, c.tensors()):
        v.copy_(x)
    w, ws = guarded(am.distillation_workspace_bytes(*c.size(), True))
    k, kept = guarded(am.distillation_kept_bytes(c.dtype, c.n, c.vocab, c.top))
    c.call([v for _, v in t], [v for _, v in outs], (ws, kept))
    torch.cuda.synchronize()
    assert all(clean(b) for b, _ in outs + t) and clean(w) and clean(k)
    assert all(torch.equal(x, v) for x, (_, v) in zip(a, outs))
    assert all(torch.equal(x, v) for x, (_, v) in zip(c.tensors(), t))
    e, loss_ws = guarded(am.distillation_workspace_bytes(*c.size()))
    am.distillation(t[0][1], t[1][1], *c.size(), t[2][1], t[3][1], c.scale, outs[0][1], outs[1][1], loss_ws)
    torch.cuda.synchronize()
    assert clean(e) and torch.equal(outs[0][1], a[0])


@pytest.mark.parametrize("Case,kw", [(Logprobs, LOGPROBS[3]), (Distill, DISTILL[2]), (Distill, DISTILL[6])])
def test_equal_calls_give_equal_bits(Case, kw):
    import torch
    c = Case(**kw)
    a = c.run()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, c.run()))


def test_calls_at_the_same_time():
    """Two streams, a workspace each."""
    import torch
    cases = [Logprobs(**LOGPROBS[3]), Distill(**DISTILL[2])]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    state = [(c.tensors(), c.outputs(), c.workspace() if i == 0 else c.buffers()) for i, c in enumerate(cases)]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s, (t, o, w) in zip(cases, streams, state):
            c.call(t, o, w, stream=s)
    torch.cuda.synchronize()
    for w, (_, o, _) in zip(want, state):
        assert all(torch.equal(x, y) for x, y in zip(w, o))


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_weights_of_all_sizes(dtype):
    """Each row's dX is its own weight's; rows of tiny weights do not lose theirs beside a large one."""
    import torch
    c = Distill(dtype, 200, 48, 300, masked=0.0)
    c.dloss = np.ones(200, dtype=np.float32)
    a = c.run()
    c.dloss = (2.0 ** np.random.default_rng(1).integers(-40, 40, 200)).astype(np.float32)
    b = c.run()
    w = torch.from_numpy(c.dloss).to(DEV)
    assert torch.equal(a[2].float() * w[:, None], b[2].float())  # powers of two: no rounding of their own
    c.dloss = np.zeros(200, dtype=np.float32)
    z = c.run()
    assert not z[2].any() and not z[3].any()


def test_one_call_with_rows_of_each_kind():
    """Left out, NaN, masked throughout, near and far references, one entry: each as in a call of its own."""
    import torch
    c = Distill(am.BF16, 96, 64, 700, masked=0.0, top=4)
    c.X[:, 5] = 0.0
    c.W[:, 5] = 0.0
    c.W[3, 5] = 2000.0             # class 3 is out of reach, or all there is
    c.ids[c.ids == 3] = 4
    c.X[8:16, 5] = 1.0             # lse 2000 away from any reference
    c.ids[16:20] = -1
    c.ids[20:24, 1:] = -1
    c.ids[20:24, 0] = 7
    c.X[30, 0] = float("nan")
    o = c.run()
    t = c.tensors()
    for rows in (slice(0, 8), slice(8, 16), slice(16, 20), slice(20, 24), slice(30, 31)):
        e = Distill(am.BF16, rows.stop - rows.start, 64, 700, top=4)
        e.X, e.W, e.ids, e.teacher, e.dloss = c.X[rows], c.W, c.ids[rows], c.teacher[rows], c.dloss[rows]
        p = e.run()
        for i in (0, 1, 2):
            x, y = o[i][rows].double(), p[i].double()
            assert torch.equal(torch.isnan(x), torch.isnan(y))
            # 64 columns of other tiles: 2^-7 of bf16 gradients' largest, 1e-6 of the sums
            tol = 2.0 ** -7 if i == 2 else 1e-6
            x, y = torch.nan_to_num(x), torch.nan_to_num(y)
            assert float((x - y).abs().max()) <= tol * max(float(y.abs().max()), 1e-30), (rows, i)
    assert float(o[1][8]) > 1900 and torch.isnan(o[0][30]) and not o[2][16:20].any()
    assert t[0].shape == (96, 64)


def test_more_rows_than_workgroups():
    """A row's answer does not depend on its place, past 2^20 rows either."""
    import torch
    n, of = (1 << 20) + 700, 1000
    rows = torch.arange(n) % of
    c, e = Logprobs(am.BF16, of, 8, 40, top=3), Logprobs(am.BF16, 1, 8, 40, top=3)
    e.n, e.X, e.W, e.tokens = n, c.X[rows], c.W, c.tokens[rows.numpy()]
    b = e.run()
    assert all(torch.equal(y, y[:of][rows]) for y in b)
    want, ids = logits_bounds.logprobs(c.X.double().numpy(), c.W.double().numpy(), c.tokens, c.scale, c.top, True)
    assert np.array_equal(b[2][:of].cpu().numpy(), ids)
    for i, name in ((0, "logprob"), (1, "entropy"), (3, "top_logprobs")):
        logits_bounds.within(name, b[i][:of], *want[name])
    c, e = Distill(am.BF16, of, 8, 40, top=3), Distill(am.BF16, 1, 8, 40, top=3)
    e.n, e.X, e.W, e.ids, e.teacher = n, c.X[rows], c.W, c.ids[rows.numpy()], c.teacher[rows.numpy()]
    e.dloss = None if c.dloss is None else c.dloss[rows.numpy()]
    b = e.run()
    assert all(torch.equal(y, y[:of][rows]) for y in b[:3])
    want = logits_bounds.distillation(c.X.double().numpy(), c.W.double().numpy(), c.ids, c.teacher.astype(np.float64), c.scale,
                                      c.dloss, True)
    for y, name in zip(b, ("loss", "lse", "dX")):
        logits_bounds.within(name, y[:of], *want[name])
