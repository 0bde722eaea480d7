"""Softmax cross entropy over a large vocabulary against the fp64 oracle, through the C ABI.

Bounds from the arithmetic, u = 2^-24, A the sum of a product's absolute terms:
  z      ez = (r + 4 planes) u A: r = 6 (d / 16 + 1) + 16 fp32 roundings on a term's way (six products of
         planes), planes of an fp32 call dropping three products of 2^-25 and two residues of 2^-26
  lse    el = max ez + (|z - m| + 16) 2 u + (u |lse|) for hardware exponentials and the joins
  G      |G| (ez + el + (|z - lse| + 8) 2 u) (of the probability's part) and its rounding, 2^-8 in bf16,
         3 u in planes;  products with it as z
  dW     takes the rows of X times their weight over the largest one, another rounding of every term:
         2^-8 |G x| in bf16, 3 u in planes, and 3 u for the quotient, its product and the factor outside
and one rounding of the output (2^-8 for bf16, u for fp32).
"""

import numpy as np
import pytest

from helpers import DEV, log
from oracle import cross_entropy as ce
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Case:
    def __init__(self, dtype, n, d, vocab, seed=0, masked=0.2, spread=2.0, weights=True):
        import torch
        rng = np.random.default_rng(seed)
        self.dtype, self.n, self.d, self.vocab = dtype, n, d, vocab
        dt = torch.bfloat16 if dtype == am.BF16 else torch.float32
        self.X = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).to(dt)
        self.W = torch.from_numpy((spread * d ** -0.5 * rng.standard_normal((vocab, d))).astype(np.float32)).to(dt)
        self.labels = rng.integers(0, vocab, n)
        self.labels[rng.random(n) < masked] = -100
        self.dloss = rng.standard_normal(n).astype(np.float32) if weights else None

    def size(self):
        return (self.dtype, self.n, self.d, self.vocab)

    def workspace(self, backward):
        import torch
        return torch.full((am.cross_entropy_workspace_bytes(*self.size(), backward),), 0xFF, dtype=torch.uint8,
                          device=DEV)

    def tensors(self):
        import torch
        return (self.X.to(DEV), self.W.to(DEV), torch.from_numpy(self.labels).to(DEV),
                None if self.dloss is None else torch.from_numpy(self.dloss).to(DEV))

    def outputs(self):
        import torch
        X, W = self.X, self.W
        return (torch.full((self.n,), 7.0, device=DEV), torch.full((self.n,), 7.0, device=DEV),
                torch.full(X.shape, 7.0, dtype=X.dtype, device=DEV), torch.full(W.shape, 7.0, dtype=W.dtype, device=DEV))

    def call(self, t, o, ws, stream=None):
        am.cross_entropy(t[0], t[1], *self.size(), t[2], o[0], o[1], ws[0], stream=stream)
        am.cross_entropy_backward(t[0], t[1], *self.size(), t[2], o[1], t[3], o[2], o[3], ws[1], stream=stream)

    def run(self):
        import torch
        o = self.outputs()
        self.call(self.tensors(), o, (self.workspace(False), self.workspace(True)))
        torch.cuda.synchronize()
        return o


def within(name, got, want, bound):
    assert np.isfinite(got).all(), name
    ratio = float(np.max(np.abs(got - want) / (bound + 1e-30)))
    log(f"PARITY {name}: {ratio:.3f} of the bound")
    assert ratio <= 1.0, (name, ratio)


def check(c, block=2000):
    log(f"CASE {c.size()}")
    loss, lse, dX, dW = (x.double().cpu().numpy() for x in c.run())
    bf = c.dtype == am.BF16
    X, W = c.X.double().numpy(), c.W.double().numpy()
    out, gr = (2.0 ** -8, 2.0 ** -8) if bf else (U, 3 * U)

    def e_of(k):
        return (6 * (k // 16 + 1) + 16 + (0 if bf else 4)) * U

    want_dW, bound_dW = np.zeros(W.shape), np.zeros(W.shape)
    ez = e_of(c.d)
    for r in range(0, c.n, block):
        x, y = X[r:r + block], c.labels[r:r + block]
        w = np.ones(len(x)) if c.dloss is None else c.dloss[r:r + block].astype(np.float64)
        on = (y >= 0) & (y < c.vocab)
        wl, ws = ce.forward(x, W, y)
        A, z = np.abs(x) @ np.abs(W).T, x @ W.T
        far = np.abs(z - z.max(1, keepdims=True)).max(1)
        el = ez * A.max(1) + (far + 16) * 2 * U + U * np.abs(ws)
        within("lse", lse[r:r + block], ws, np.where(on, el, 0.0))
        within("loss", loss[r:r + block], wl, np.where(on, el + ez * A.max(1) + U * np.abs(wl), 0.0))
        G = ce.gradient_of_logits(x, W, y, w)
        P = G.copy()
        P[np.arange(len(x))[on], y[on]] += w[on]
        eG = np.abs(P) * (ez * A + el[:, None] + (np.abs(z - ws[:, None]) + 8) * 2 * U) + (gr + U) * np.abs(G)
        dx = G @ W
        eX = eG @ np.abs(W) + (e_of(c.vocab) + c.vocab / 512 * U) * (np.abs(G) @ np.abs(W)) + out * np.abs(dx)
        within("dX", dX[r:r + block], dx, eX)
        x0 = np.where(on[:, None], x, 0.0)
        want_dW += G.T @ x0
        bound_dW += eG.T @ np.abs(x0) + (e_of(c.n) + gr + 3 * U) * (np.abs(G).T @ np.abs(x0))
    within("dW", dW, want_dW, bound_dW + out * np.abs(want_dW))


CASES = [
    ("one_row", dict(dtype=am.BF16, n=1, d=64, vocab=1000, masked=0.0)),
    ("one_class", dict(dtype=am.F32, n=5, d=16, vocab=1)),
    ("one_column", dict(dtype=am.F32, n=9, d=1, vocab=50)),
    ("two_classes", dict(dtype=am.BF16, n=130, d=8, vocab=2)),
    ("odd_columns", dict(dtype=am.BF16, n=77, d=35, vocab=301)),
    ("odd_columns_f32", dict(dtype=am.F32, n=77, d=35, vocab=301)),
    ("tile", dict(dtype=am.BF16, n=128, d=64, vocab=128)),
    ("tile_and_one", dict(dtype=am.BF16, n=129, d=72, vocab=257)),
    ("tile_less_one", dict(dtype=am.F32, n=127, d=56, vocab=255)),
    ("ragged", dict(dtype=am.BF16, n=333, d=384, vocab=5003)),
    ("ragged_f32", dict(dtype=am.F32, n=210, d=136, vocab=3001)),
    ("unweighted", dict(dtype=am.F32, n=50, d=32, vocab=99, weights=False)),
    ("sharp", dict(dtype=am.BF16, n=100, d=64, vocab=500, spread=20.0)),
    ("sharp_f32", dict(dtype=am.F32, n=100, d=64, vocab=500, spread=20.0)),
    ("all_left_out", dict(dtype=am.BF16, n=40, d=32, vocab=60, masked=1.1)),
    ("large_tiles", dict(dtype=am.BF16, n=1100, d=72, vocab=16003)),
    ("large_tiles_f32", dict(dtype=am.F32, n=1500, d=40, vocab=12000)),
    ("large_tiles_wide_rows", dict(dtype=am.BF16, n=4300, d=4096, vocab=520)),
    ("middle_tiles", dict(dtype=am.BF16, n=700, d=904, vocab=4000)),
    ("middle_tiles_narrow_rows", dict(dtype=am.BF16, n=1500, d=100, vocab=12000)),
    ("pieces", dict(dtype=am.F32, n=22000, d=16, vocab=4200)),
]


@pytest.mark.parametrize("kw", [c[1] for c in CASES], ids=[c[0] for c in CASES])
def test_parity(kw):
    check(Case(**kw))


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_rows_left_out_may_hold_anything(dtype):
    import torch
    c = Case(dtype, 200, 64, 500, masked=0.0)
    c.labels[3], c.labels[50], c.labels[199] = -1, 500, -100
    a = c.run()
    for i, v in ((3, float("nan")), (50, float("inf")), (199, -float("inf"))):
        c.X[i, :] = v
    b = c.run()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for i in (3, 50, 199):
        assert float(b[0][i]) == 0.0 and float(b[1][i]) == 0.0 and not b[2][i].any()


def test_nan_stays_in_its_row():
    import torch
    c = Case(am.BF16, 140, 64, 500, masked=0.0)
    a = c.run()
    c.X[7, 3] = float("nan")
    b = c.run()
    assert torch.isnan(b[0][7]) and torch.isnan(b[1][7]) and torch.isnan(b[2][7]).all()
    keep = torch.arange(140, device=DEV) != 7
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[2][keep], b[2][keep])


def test_one_gradient_alone():
    import torch
    c = Case(am.BF16, 300, 64, 700)
    a, t, ws = c.run(), c.tensors(), c.workspace(True)
    for which in (2, 3):
        o = c.outputs()
        am.cross_entropy_backward(t[0], t[1], *c.size(), t[2], a[1], t[3], o[2] if which == 2 else None,
                                  o[3] if which == 3 else None, ws)
        torch.cuda.synchronize()
        assert torch.equal(o[which], a[which])


def test_no_rows():
    import torch
    W = torch.ones((30, 8), device=DEV)
    dW = torch.full_like(W, 7.0)
    am.cross_entropy_backward(None, W, am.F32, 0, 8, 30, None, None, None, None, dW, None)
    assert not dW.any()


def test_unaligned_and_other_streams():
    import torch
    c = Case(am.BF16, 150, 64, 700)
    a = c.run()
    t, o, ws, s = c.tensors(), c.outputs(), (c.workspace(False), c.workspace(True)), torch.cuda.Stream()
    torch.cuda.synchronize()
    c.call(t, o, ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, o))

    def shifted(x):
        b = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
        return b.copy_(x)

    o = [o[0], o[1], shifted(o[2]), shifted(o[3])]
    for x in o:
        x.fill_(7.0)
    c.call((shifted(t[0]), shifted(t[1]), t[2], t[3]), o, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, o))


def test_captured_and_replayed():
    import torch
    c = Case(am.BF16, 150, 64, 700)
    t, o, ws = c.tensors(), c.outputs(), (c.workspace(False), c.workspace(True))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.call(t, o, ws)
    for i in range(3):
        e = Case(am.BF16, 150, 64, 700, seed=20 + i)
        for dst, src in zip(t, e.tensors()):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(o, e.run()))


def test_offsets_past_32_bits():
    """More than 2^31 elements of W and dW: the last class is read and written where it is."""
    import torch
    n, d, vocab = 3, 4096, 530000
    X = torch.zeros((n, d), dtype=torch.bfloat16, device=DEV)
    W = torch.zeros((vocab, d), dtype=torch.bfloat16, device=DEV)
    X[0, -1] = X[1, 0] = 4.0
    W[-1, -1] = W[-2, 0] = 5.0
    labels = torch.tensor([vocab - 1, 0, -1], device=DEV)
    loss, lse = torch.empty((2, n), device=DEV)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    size = (am.BF16, n, d, vocab)
    am.cross_entropy(X, W, *size, labels, loss, lse,
                     torch.empty(am.cross_entropy_workspace_bytes(*size), dtype=torch.uint8, device=DEV))
    want = np.log(vocab - 1 + np.exp(20.0))
    assert np.allclose(lse.cpu()[:2], want, rtol=1e-6)
    assert np.allclose(loss.cpu(), [want - 20.0, want, 0.0], rtol=1e-3, atol=1e-6)
    am.cross_entropy_backward(X, W, *size, labels, lse, None, dX, dW,
                              torch.empty(am.cross_entropy_workspace_bytes(*size, True), dtype=torch.uint8, device=DEV))
    p = np.exp(20.0 - want)
    assert abs(float(dW[-1, -1]) - 4 * (p - 1)) <= 2.0 ** -6 * 4 * (1 - p)
    assert abs(float(dW[-2, 0]) - 4 * p) <= 2.0 ** -6 * 4 * p
    assert abs(float(dX[0, -1]) - 5 * (p - 1)) <= 2.0 ** -6 * 5 * (1 - p)
