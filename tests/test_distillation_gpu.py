"""Distillation from a teacher's top logits and its gradients against the fp64 oracle, through the C ABI.  Bounds: see
logits_bounds."""

import numpy as np
import pytest

from helpers import DEV, log
from logits_bounds import distillation as expected
from logits_bounds import within
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, dtype, n, d, vocab, top=5, seed=0, masked=0.2, spread=2.0, scale=1.0, weights=True, near=False):
        import torch
        rng = np.random.default_rng(seed)
        self.dtype, self.n, self.d, self.vocab, self.top, self.scale = dtype, n, d, vocab, top, scale
        dt = torch.bfloat16 if dtype == am.BF16 else torch.float32
        self.X = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).to(dt)
        self.W = torch.from_numpy((spread * d ** -0.5 * rng.standard_normal((vocab, d))).astype(np.float32)).to(dt)
        if near:  # side by side
            self.ids = (rng.integers(0, vocab, (n, 1)) + np.arange(top)) % vocab
        else:
            self.ids = np.stack([rng.permutation(vocab)[np.arange(top) % vocab] for _ in range(n)])
        self.ids[rng.random((n, top)) < 0.15] = -1
        self.ids[rng.random(n) < masked] = -100
        self.teacher = (10.0 + 2.0 * rng.standard_normal((n, top))).astype(np.float32)
        self.teacher[rng.random((n, top)) < 0.05] = -np.inf
        self.dloss = rng.standard_normal(n).astype(np.float32) if weights else None

    def size(self):
        return (self.dtype, self.n, self.d, self.vocab, self.top)

    def buffers(self):
        import torch
        return [torch.full((b,), 171, dtype=torch.uint8, device=DEV)
                for b in (am.distillation_workspace_bytes(*self.size(), True),
                          am.distillation_kept_bytes(self.dtype, self.n, self.vocab, self.top))]

    def tensors(self):
        import torch
        return (self.X.to(DEV), self.W.to(DEV), torch.from_numpy(self.ids).to(DEV), torch.from_numpy(self.teacher).to(DEV),
                None if self.dloss is None else torch.from_numpy(self.dloss).to(DEV))

    def outputs(self):
        import torch
        o = [torch.full((self.n,), 7.0, device=DEV) for _ in range(2)]
        return o + [torch.full(x.shape, 7.0, dtype=x.dtype, device=DEV) for x in (self.X, self.W)]

    def call(self, t, o, b, stream=None):
        am.distillation(t[0], t[1], *self.size(), t[2], t[3], self.scale, o[0], o[1], b[0], kept=b[1], stream=stream)
        am.distillation_backward(t[0], t[1], *self.size(), b[1], t[4], o[2], o[3], b[0], stream=stream)

    def run(self):
        import torch
        o = self.outputs()
        self.call(self.tensors(), o, self.buffers())
        torch.cuda.synchronize()
        return o


def check(c, plain32=False):
    import torch
    log(f"CASE {c.size()}")
    o = c.run()
    want = expected(c.X.double().numpy(), c.W.double().numpy(), c.ids, c.teacher.astype(np.float64), c.scale, c.dloss,
                    c.dtype == am.BF16, plain32)
    for x, name in zip(o, ("loss", "lse", "dX", "dW")):
        within(name, x, *want[name])
    # the loss alone
    t, e = c.tensors(), c.outputs()
    am.distillation(t[0], t[1], *c.size(), t[2], t[3], c.scale, e[0], e[1],
                    torch.full((am.distillation_workspace_bytes(*c.size()),), 171, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(e[0], o[0]) and torch.equal(e[1], o[1])
    return o


CASES = [
    ("one_row", dict(dtype=am.BF16, n=1, d=64, vocab=1000, masked=0.0)),
    ("one_class", dict(dtype=am.F32, n=5, d=16, vocab=1, top=1)),
    ("one_class_many_times", dict(dtype=am.BF16, n=5, d=16, vocab=1, top=7)),
    ("one_column", dict(dtype=am.F32, n=9, d=1, vocab=50)),
    ("two_classes", dict(dtype=am.BF16, n=130, d=8, vocab=2, top=2)),
    ("one_entry", dict(dtype=am.BF16, n=130, d=24, vocab=99, top=1)),
    ("most_entries", dict(dtype=am.BF16, n=50, d=24, vocab=300, top=128)),
    ("most_entries_near", dict(dtype=am.F32, n=50, d=24, vocab=301, top=127, near=True)),
    ("entries_past_a_wave", dict(dtype=am.BF16, n=21, d=24, vocab=300, top=65, near=True)),
    ("every_class_given_twice", dict(dtype=am.F32, n=20, d=24, vocab=40, top=80)),
    ("odd_columns", dict(dtype=am.BF16, n=77, d=35, vocab=301, scale=0.5)),
    ("odd_columns_f32", dict(dtype=am.F32, n=77, d=35, vocab=301, scale=1.5)),
    ("tile", dict(dtype=am.BF16, n=128, d=64, vocab=128)),
    ("tile_and_one", dict(dtype=am.BF16, n=129, d=72, vocab=257)),
    ("tile_less_one", dict(dtype=am.F32, n=127, d=56, vocab=255)),
    ("ragged", dict(dtype=am.BF16, n=333, d=384, vocab=5003, top=20)),
    ("ragged_f32", dict(dtype=am.F32, n=210, d=136, vocab=3001, top=20, near=True)),
    ("factors_rounded_up_f32", dict(dtype=am.F32, n=90, d=48, vocab=1001, scale=1.25)),
    ("factors_rounded_down_f32", dict(dtype=am.F32, n=90, d=48, vocab=1001, scale=0.7)),
    ("wide_rows_f32", dict(dtype=am.F32, n=5, d=1000, vocab=659, top=128)),
    ("rows_gathered_f32", dict(dtype=am.F32, n=500, d=400, vocab=24001, masked=0.5)),
    ("rows_gathered", dict(dtype=am.BF16, n=2100, d=1032, vocab=12001, top=16)),
    ("many_short_rows", dict(dtype=am.BF16, n=4500, d=40, vocab=300, top=20)),
    ("many_short_rows_f32", dict(dtype=am.F32, n=4200, d=23, vocab=130, top=64)),
    ("many_short_rows_far_references", dict(dtype=am.BF16, n=4100, d=64, vocab=200, top=3, spread=30.0)),
    ("as_many_rows_as_few", dict(dtype=am.BF16, n=64, d=520, vocab=3001, top=9)),
    ("as_many_rows_as_few_f32", dict(dtype=am.F32, n=64, d=260, vocab=3001, top=9)),
    ("hottest", dict(dtype=am.BF16, n=60, d=64, vocab=700, scale=2.0 ** -20)),
    ("unweighted", dict(dtype=am.F32, n=50, d=32, vocab=99, weights=False)),
    ("far_references", dict(dtype=am.BF16, n=100, d=64, vocab=500, spread=30.0)),
    ("far_references_f32", dict(dtype=am.F32, n=100, d=64, vocab=500, spread=30.0, scale=1.5)),
    ("all_left_out", dict(dtype=am.BF16, n=40, d=32, vocab=60, masked=1.1)),
    ("large_tiles", dict(dtype=am.BF16, n=1100, d=72, vocab=16003, top=8)),
    ("large_tiles_far_references", dict(dtype=am.BF16, n=1100, d=72, vocab=16003, top=3, spread=20.0)),
    ("middle_tiles_f32", dict(dtype=am.F32, n=1500, d=40, vocab=12000)),
    ("middle_tiles", dict(dtype=am.BF16, n=700, d=904, vocab=4000, top=32)),
    ("large_tiles_wide_rows", dict(dtype=am.BF16, n=4300, d=4096, vocab=520)),
]


@pytest.mark.parametrize("kw", [c[1] for c in CASES], ids=[c[0] for c in CASES])
def test_parity(kw):
    check(Case(**kw))


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_one_sure_class_is_cross_entropy(dtype):
    """Losses within two roundings of the sums of cross entropy's own."""
    import torch
    c = Case(dtype, 150, 64, 700, top=2)
    c.ids[:, 0] = np.random.default_rng(8).integers(0, 700, 150)
    c.ids[5, 0] = -100
    c.teacher[:, 0], c.teacher[:, 1] = 0.0, -np.inf
    o, t = c.run(), c.tensors()
    loss, lse = torch.empty(2, 150, device=DEV)
    am.cross_entropy(t[0], t[1], dtype, 150, 64, 700, t[2][:, 0].contiguous(), loss, lse,
                     torch.empty(am.cross_entropy_workspace_bytes(dtype, 150, 64, 700), dtype=torch.uint8, device=DEV))
    # logits of up to 9 in sums of 64 + 16 roundings of 2^-24
    assert torch.allclose(o[0], loss, rtol=0, atol=9 * 80 * 2.0 ** -24) and torch.allclose(o[1], lse, rtol=0, atol=9 * 80 * 2.0 ** -24)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("mask", [-float("inf"), float(np.finfo(np.float32).min)])
def test_masked_classes(dtype, mask):
    """Masked by a column of ones: probability zero.  Minus infinity makes dX's column of ones NaN."""
    import torch
    c = Case(dtype, 140, 32, 600, top=6, masked=0.1)
    if dtype == am.BF16 and mask != -float("inf"):
        mask = float(torch.finfo(torch.bfloat16).min)
    hidden = np.arange(600) % 3 == 1
    c.ids = np.where(c.ids >= 0, c.ids // 3 * 3, c.ids)
    c.X[:, 7] = 1.0
    c.W[:, 7] = 0.0
    c.W[hidden, 7] = mask
    o = c.run()
    X, W = c.X.double().numpy(), c.W.double().numpy()
    want = expected(X, W, c.ids, c.teacher.astype(np.float64), c.scale, c.dloss, dtype == am.BF16, plain32=True)
    others = np.arange(32) != 7
    for x, name in zip(o, ("loss", "lse", "dX", "dW")):
        v, b = want[name]
        if name == "dX":
            x, v, b = x[:, others], v[:, others], b[:, others]
        within(name, x, v, b)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_a_masked_class_of_the_teachers(dtype):
    """The teacher's likeliest class is impossible for the student: an infinite loss, a finite gradient."""
    import torch
    c = Case(dtype, 30, 32, 200, top=3, masked=0.0)
    c.X[:, 7] = 1.0
    c.W[:, 7] = 0.0
    c.W[11, 7] = -float("inf")
    c.ids[4], c.teacher[4] = [11, 20, 30], [12.0, 11.0, 10.0]
    c.ids[:4][c.ids[:4] == 11], c.ids[5:][c.ids[5:] == 11] = 12, 12
    o = c.run()
    assert torch.isposinf(o[0][4]) and torch.isfinite(o[1]).all() and torch.isfinite(o[0][torch.arange(30) != 4]).all()
    assert torch.isfinite(o[3]).all()
    G = -0.6652409557748219 * float(c.dloss[4])  # row 11 of dW: this row alone
    got, want = o[3][11].double().cpu().numpy(), G * c.X[4].double().numpy()
    assert np.allclose(got, want, rtol=2.0 ** -6 if dtype == am.BF16 else 1e-5, atol=0)


def test_teacher_values():
    """NaN stays in its row's loss; entries that do not count may hold anything."""
    import torch
    c = Case(am.BF16, 140, 64, 500, masked=0.1)
    c.ids[9] = [5, -1, 7, 500, 8]
    c.teacher[9] = [1, 2, 3, 4, 5]
    a = c.run()
    c.teacher[9, 1], c.teacher[9, 3] = np.nan, np.inf
    b = c.run()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    c.teacher[9, 2] = np.nan
    b = c.run()
    keep = torch.arange(140, device=DEV) != 9
    assert torch.isnan(b[0][9]) and torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1], b[1])
    assert torch.equal(a[2][keep], b[2][keep])


def test_equal_logits_in_any_order():
    import torch
    c = Case(am.BF16, 100, 64, 500, top=40, masked=0.0)
    a = check(c)
    order = np.random.default_rng(2).permutation(40)
    c.ids, c.teacher = c.ids[:, order].copy(), c.teacher[:, order].copy()
    b = check(c)
    assert torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_rows_left_out_may_hold_anything(dtype):
    import torch
    c = Case(dtype, 200, 64, 500, masked=0.0)
    c.ids[3], c.ids[50], c.teacher[199] = -1, 500, -np.inf
    a = c.run()
    for i, v in ((3, float("nan")), (50, float("inf")), (199, -float("inf"))):
        c.X[i, :] = v
    c.dloss[3], c.teacher[50] = np.nan, np.nan
    b = c.run()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for i in (3, 50, 199):
        assert not b[0][i] and not b[1][i] and not b[2][i].any()


def test_nan_stays_in_its_row():
    import torch
    c = Case(am.BF16, 140, 64, 500, masked=0.0)
    a = c.run()
    c.X[7, 3] = float("nan")
    b = c.run()
    assert torch.isnan(b[0][7]) and torch.isnan(b[1][7]) and torch.isnan(b[2][7]).all()
    keep = torch.arange(140, device=DEV) != 7
    assert all(torch.equal(a[i][keep], b[i][keep]) for i in (0, 1, 2))


def test_one_gradient_alone_and_twice():
    import torch
    c = Case(am.BF16, 300, 64, 700)
    t, b, a = c.tensors(), c.buffers(), c.outputs()
    c.call(t, a, b)
    for which in (2, 3, 2):
        o = c.outputs()
        am.distillation_backward(t[0], t[1], *c.size(), b[1], t[4], o[2] if which == 2 else None,
                                 o[3] if which == 3 else None, b[0])
        torch.cuda.synchronize()
        assert torch.equal(o[which], a[which])


def test_no_rows():
    import torch
    W = torch.ones((30, 8), device=DEV)
    dW = torch.full_like(W, 7.0)
    am.distillation_backward(None, None, am.F32, 0, 8, 30, 2, None, None, None, dW, None)
    assert not dW.any()


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_unaligned_and_other_streams(dtype):
    import torch
    c = Case(dtype, 150, 64, 700)
    a = c.run()
    t, o, b, s = c.tensors(), c.outputs(), c.buffers(), torch.cuda.Stream()
    torch.cuda.synchronize()
    c.call(t, o, b, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, o))

    def shifted(x):
        y = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
        return y.copy_(x)

    o = [shifted(x) for x in o]
    for x in o:
        x.fill_(7.0)
    c.call(tuple(shifted(x) for x in t), o, b)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, o))


def test_captured_and_replayed():
    import torch
    c = Case(am.BF16, 150, 64, 700, spread=12.0)
    t, o, b = c.tensors(), c.outputs(), c.buffers()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.call(t, o, b)
    for i in range(4):
        e = Case(am.BF16, 150, 64, 700, seed=20 + i, spread=(2.0, 40.0)[i % 2])
        for dst, src in zip(t, e.tensors()):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(o, e.run()))


def test_differences():
    """The gradient of the loss as it is computed, in fp32, along a direction in X and in W."""
    import torch
    c = Case(am.F32, 60, 16, 90, top=6)
    t, o, b = c.tensors(), c.outputs(), c.buffers()
    c.call(t, o, b)
    gen = torch.Generator(device=DEV).manual_seed(4)
    for which in (0, 1):
        step = torch.randn(t[which].shape, generator=gen, device=DEV)
        h = 2.0 ** -7
        ends = []
        for sign in (1.0, -1.0):
            moved = list(t)
            moved[which] = t[which] + sign * h * step
            e = c.outputs()
            am.distillation(moved[0], moved[1], *c.size(), t[2], t[3], c.scale, e[0], e[1], b[0])
            ends.append((e[0].double() * t[4].double()).sum())
        got = float((o[2 + which].double() * step.double()).sum())
        want = float(ends[0] - ends[1]) / (2 * h)
        # third derivatives: h^2 / 6 of a change of the logits by up to 4 a row; roundings: 2^-20 of each loss / h
        size = float((t[4].abs() * (1 if which == 0 else 1)).sum())
        assert abs(got - want) <= size * (h * h / 6 * 4 ** 3 + 2 * 10 * 2.0 ** -20 / h), (got, want)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,d,vocab,top", [(3, 2100, 400, 64), (9, 300, 500, 128), (256, 40, 300, 17), (257, 40, 300, 17),
                                           (256, 72, 300, 16), (2048, 40, 300, 16)])
def test_many_entries_of_few_rows(dtype, n, d, vocab, top):
    """On both sides of what decides how many lanes a row has."""
    check(Case(dtype, n, d, vocab, top=top))
