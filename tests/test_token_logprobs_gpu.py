"""Token log probabilities, entropies and top alternatives against the fp64 oracle, through the C ABI.  Bounds: see
logits_bounds; alternatives have to be the oracle's, in its order."""

import numpy as np
import pytest

from helpers import DEV, log
from logits_bounds import logprobs as expected
from logits_bounds import within
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, dtype, n, d, vocab, top=5, seed=0, masked=0.2, spread=2.0, scale=1.0, tokens=True, lean=0.0):
        import torch
        rng = np.random.default_rng(seed)
        self.dtype, self.n, self.d, self.vocab, self.top, self.scale = dtype, n, d, vocab, top, scale
        dt = torch.bfloat16 if dtype == am.BF16 else torch.float32
        X, W = rng.standard_normal((n, d)), spread * d ** -0.5 * rng.standard_normal((vocab, d))
        if lean:  # classes numbered by how frequent they are
            X += 0.5
            W -= lean * np.log1p(np.arange(vocab))[:, None] * 2.0 / d
        self.X = torch.from_numpy(X.astype(np.float32)).to(dt)
        self.W = torch.from_numpy(W.astype(np.float32)).to(dt)
        self.tokens = None
        if tokens:
            self.tokens = rng.integers(0, vocab, n)
            self.tokens[rng.random(n) < masked] = -100

    def size(self):
        return (self.dtype, self.n, self.d, self.vocab)

    def tensors(self):
        import torch
        return (self.X.to(DEV), self.W.to(DEV), None if self.tokens is None else torch.from_numpy(self.tokens).to(DEV))

    def outputs(self):
        import torch
        o = [torch.full((self.n,), 7.0, device=DEV) for _ in range(2)]
        if self.top:
            o += [torch.full((self.n, self.top), 7, dtype=torch.int64, device=DEV),
                  torch.full((self.n, self.top), 7.0, device=DEV)]
        return o

    def workspace(self):
        import torch
        size = am.token_logprobs_workspace_bytes(*self.size(), self.top)
        return torch.full((size,), 171, dtype=torch.uint8, device=DEV)

    def call(self, t, o, ws, stream=None):
        am.token_logprobs(t[0], t[1], *self.size(), t[2], None if t[2] is None else o[0], o[1], ws, scale=self.scale,
                          top=self.top, top_ids=o[2] if self.top else None, top_logprobs=o[3] if self.top else None,
                          stream=stream)

    def run(self):
        import torch
        o = self.outputs()
        self.call(self.tensors(), o, self.workspace())
        torch.cuda.synchronize()
        return o


def check(c, plain32=False):
    log(f"CASE {c.size()} {c.top}")
    o = c.run()
    want, ids = expected(c.X.double().numpy(), c.W.double().numpy(), c.tokens, c.scale, c.top, c.dtype == am.BF16, plain32)
    if c.top:
        got = o[2].cpu().numpy()
        assert np.array_equal(got, ids), (got != ids).sum()
        within("top_logprobs", o[3], *want["top_logprobs"])
    if c.tokens is not None:
        within("logprob", o[0], *want["logprob"])
    within("entropy", o[1], *want["entropy"])
    return o


CASES = [
    ("one_row", dict(dtype=am.BF16, n=1, d=64, vocab=1000, masked=0.0)),
    ("one_class", dict(dtype=am.F32, n=5, d=16, vocab=1, top=1)),
    ("one_column", dict(dtype=am.F32, n=9, d=1, vocab=50, top=3)),
    ("no_alternatives", dict(dtype=am.BF16, n=70, d=40, vocab=300, top=0)),
    ("no_tokens", dict(dtype=am.BF16, n=20, d=40, vocab=300, tokens=False)),
    ("every_class_an_alternative", dict(dtype=am.BF16, n=11, d=24, vocab=64, top=64)),
    ("most_alternatives", dict(dtype=am.F32, n=11, d=24, vocab=70, top=64)),
    ("odd_columns", dict(dtype=am.BF16, n=77, d=35, vocab=301)),
    ("odd_columns_f32", dict(dtype=am.F32, n=77, d=35, vocab=301, scale=0.5)),
    ("tile", dict(dtype=am.BF16, n=64, d=64, vocab=64)),
    ("tile_and_one", dict(dtype=am.BF16, n=65, d=72, vocab=65, scale=1.5)),
    ("tile_less_one", dict(dtype=am.F32, n=63, d=56, vocab=255)),
    ("groups_past_a_workgroup", dict(dtype=am.BF16, n=3, d=64, vocab=9001, top=64)),
    ("ragged", dict(dtype=am.BF16, n=333, d=384, vocab=5003, top=20, scale=1.25)),
    ("ragged_f32", dict(dtype=am.F32, n=210, d=136, vocab=3001, top=20)),
    ("factors_rounded_up_f32", dict(dtype=am.F32, n=90, d=48, vocab=1001, top=20, scale=1.25)),
    ("factors_rounded_down_f32", dict(dtype=am.F32, n=90, d=48, vocab=1001, top=20, scale=0.7)),
    ("wide_rows_f32", dict(dtype=am.F32, n=47, d=3616, vocab=1301, top=3)),
    ("hottest", dict(dtype=am.BF16, n=60, d=64, vocab=700, top=7, scale=2.0 ** -20)),
    ("coldest", dict(dtype=am.F32, n=60, d=64, vocab=700, top=7, scale=2.0 ** 20)),
    ("few_groups_many_alternatives", dict(dtype=am.BF16, n=17, d=80, vocab=642, top=64)),
    ("as_many_rows_as_few", dict(dtype=am.BF16, n=64, d=520, vocab=9001, top=20)),
    ("as_many_rows_as_few_f32", dict(dtype=am.F32, n=64, d=260, vocab=9001, top=20)),
    ("frequent_first", dict(dtype=am.BF16, n=200, d=128, vocab=20011, top=64, lean=1.0)),
    ("sharp", dict(dtype=am.BF16, n=100, d=64, vocab=500, spread=20.0)),
    ("sharp_f32", dict(dtype=am.F32, n=100, d=64, vocab=500, spread=20.0, scale=2.0)),
    ("all_left_out", dict(dtype=am.BF16, n=40, d=32, vocab=60, masked=1.1)),
    ("large_tiles", dict(dtype=am.BF16, n=1100, d=72, vocab=16003, top=20, lean=0.7)),
    ("middle_tiles", dict(dtype=am.BF16, n=700, d=904, vocab=4000, top=8)),
    ("middle_tiles_f32", dict(dtype=am.F32, n=1500, d=40, vocab=12000, top=8)),
    ("rows_gathered", dict(dtype=am.BF16, n=2100, d=2048, vocab=24001, top=3)),
    ("rows_gathered_f32", dict(dtype=am.F32, n=700, d=1000, vocab=24001, top=3, masked=0.5)),
]


@pytest.mark.parametrize("kw", [c[1] for c in CASES], ids=[c[0] for c in CASES])
def test_parity(kw):
    check(Case(**kw))


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,d,vocab,top", [(2, 33, 5000, 64), (300, 33, 1135, 64), (520, 300, 1000, 64), (1100, 33, 200, 20),
                                           (1100, 40, 90, 32), (1100, 5, 300, 1), (1100, 300, 2000, 10),
                                           (1100, 130, 5000, 32), (1100, 64, 20, 20)])
def test_first_choices(dtype, n, d, vocab, top):
    """Few and many rows of few and many classes, short and long: each way to the first alternatives."""
    check(Case(dtype, n, d, vocab, top=top))


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,d,vocab,top", [(300, 12, 700, 40), (1100, 12, 700, 20), (1100, 12, 9000, 8)])
def test_equal_logits_of_many_rows(dtype, n, d, vocab, top):
    """Small whole numbers, of which whole groups pass the last alternative: they go to the lowest index."""
    import torch
    c = Case(dtype, n, d, vocab, top=top)
    rng = np.random.default_rng(4)
    c.X = torch.from_numpy(rng.integers(-2, 3, c.X.shape).astype(np.float32)).to(c.X.dtype)
    c.W = torch.from_numpy(rng.integers(-1, 2, c.W.shape).astype(np.float32)).to(c.W.dtype)
    c.X[1::50] = 0.0
    check(c)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,vocab,top", [(5, 700, 20), (600, 9000, 64)])
def test_equal_logits_go_to_the_lowest_index(dtype, n, vocab, top):
    """Small whole numbers: few distinct logits, all exact."""
    import torch
    c = Case(dtype, n, 12, vocab, top=top, masked=0.0)
    rng = np.random.default_rng(3)
    c.X = torch.from_numpy(rng.integers(-2, 3, c.X.shape).astype(np.float32)).to(c.X.dtype)
    c.W = torch.from_numpy(rng.integers(-1, 2, c.W.shape).astype(np.float32)).to(c.W.dtype)
    c.X[1] = 0.0
    check(c)
    c.W[:] = 0.0
    check(c)


@pytest.mark.parametrize("vocab,alike", [(3000, 900), (70000, 3000)])
def test_logits_nearer_than_their_sums_round(vocab, alike):
    """Many classes apart by a few units in the last place of a weight, spread over the vocabulary and side by side."""
    import torch
    c = Case(am.F32, 6, 48, vocab, top=30, masked=0.0)
    rng = np.random.default_rng(5)
    row = 0.5 + torch.rand(48)
    c.X = (0.5 + torch.rand(6, 48)).float()
    for at in (np.arange(alike) + vocab // 3, rng.permutation(vocab)[:alike]):
        c.W[:] = -row
        c.W[at] = row
        for i in range(4):
            c.W[at, rng.integers(0, 48, alike)] *= torch.from_numpy((1 + rng.integers(-9, 9, alike) * 2.0 ** -23).astype(np.float32))
        check(c)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("mask", [-float("inf"), float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("n,vocab,left", [(4, 900, 3), (300, 3000, 1500), (40, 20000, 1)])
def test_masked_classes(dtype, mask, n, vocab, left):
    import torch
    c = Case(dtype, n, 32, vocab, top=8, masked=0.0)
    if dtype == am.BF16 and mask != -float("inf"):
        mask = float(torch.finfo(torch.bfloat16).min)
    hidden = np.random.default_rng(1).permutation(vocab)[left:]
    c.X[:, 7] = 1.0
    c.W[:, 7] = 0.0
    c.W[hidden, 7] = mask
    c.tokens = np.setdiff1d(np.arange(vocab), hidden)[np.arange(n) % left]
    o = check(c, plain32=True)
    if left < 8:
        assert (o[2].cpu() == -1).sum() == n * (8 - left)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("n,vocab", [(6, 900), (90, 2000), (1200, 9000)])
def test_classes_masked_in_some_rows(dtype, n, vocab):
    """A column of X says whether a row's classes are masked: the others' alternatives are all classes'."""
    import torch
    c = Case(dtype, n, 32, vocab, top=12, masked=0.0)
    mask = float(torch.finfo(c.X.dtype).min)
    hidden = np.random.default_rng(1).random(vocab) < 0.8
    c.X[:, 7] = torch.from_numpy((np.arange(n) % 2).astype(np.float32)).to(c.X.dtype)
    c.W[:, 7] = 0.0
    c.W[hidden, 7] = mask
    c.tokens = np.where(~hidden)[0][np.arange(n) % (~hidden).sum()]
    check(c, plain32=True)


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_a_row_without_a_class(dtype):
    import torch
    c = Case(dtype, 70, 16, 500, masked=0.0)
    a = c.run()
    c.X[:, 3] = 0.0
    c.W[:, 3] = -float("inf")
    c.X[9, 3] = 1.0
    c.X[:, 3] = torch.where(torch.arange(70) == 9, 1.0, 1.0).to(c.X.dtype)
    o = c.run()
    assert torch.isneginf(o[0]).all() and not o[1].any() and (o[2] == -1).all() and torch.isneginf(o[3]).all()
    assert torch.isfinite(a[0]).all()


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_and_infinity_stay_in_their_row(dtype, value):
    import torch
    c = Case(dtype, 140, 64, 500, masked=0.0)
    a = c.run()
    c.X[7, 3] = value
    b = c.run()
    assert torch.isnan(b[0][7]) and torch.isnan(b[1][7]) and (b[2][7] == -1).all() and torch.isnan(b[3][7]).all()
    keep = torch.arange(140, device=DEV) != 7
    assert all(torch.equal(x[keep], y[keep]) for x, y in zip(a, b))


@pytest.mark.parametrize("kw", [dict(n=200, d=64, vocab=500), dict(n=2100, d=2048, vocab=24001)])
def test_rows_left_out_may_hold_anything(kw):
    import torch
    c = Case(am.BF16, masked=0.0, **kw)
    c.tokens[3], c.tokens[50], c.tokens[199] = -1, c.vocab, -100
    a = c.run()
    for i, v in ((3, float("nan")), (50, float("inf")), (199, -float("inf"))):
        c.X[i, :] = v
    b = c.run()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for i in (3, 50, 199):
        assert not b[0][i] and not b[1][i] and (b[2][i] == -1).all() and not b[3][i].any()


def test_outputs_that_are_not_asked_for():
    import torch
    c = Case(am.BF16, 90, 64, 700)
    a, t, ws = c.run(), c.tensors(), c.workspace()
    o = c.outputs()
    am.token_logprobs(t[0], t[1], *c.size(), t[2], None, o[1], ws)
    am.token_logprobs(t[0], t[1], *c.size(), t[2], o[0], None, ws, top=c.top, top_ids=o[2], top_logprobs=o[3])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, o))


@pytest.mark.parametrize("dtype", [am.BF16, am.F32])
def test_unaligned_and_other_streams(dtype):
    import torch
    c = Case(dtype, 150, 64, 700)
    a = c.run()
    t, o, ws, s = c.tensors(), c.outputs(), c.workspace(), torch.cuda.Stream()
    torch.cuda.synchronize()
    c.call(t, o, ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, o))

    def shifted(x):
        b = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
        return b.copy_(x)

    o = [shifted(x) for x in o]
    for x in o:
        x.fill_(7)
    c.call(tuple(shifted(x) for x in t), o, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, o))


def test_captured_and_replayed():
    import torch
    c = Case(am.BF16, 150, 64, 700)
    t, o, ws = c.tensors(), c.outputs(), c.workspace()
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
    """More than 2^31 elements of W: the last classes are read where they are."""
    import torch
    n, d, vocab = 3, 4096, 530000
    X = torch.zeros((n, d), dtype=torch.bfloat16, device=DEV)
    W = torch.zeros((vocab, d), dtype=torch.bfloat16, device=DEV)
    X[0, -1] = X[1, 0] = 4.0
    W[-1, -1] = W[-2, 0] = 5.0
    tokens = torch.tensor([vocab - 1, 0, -1], device=DEV)
    logprob, entropy = torch.empty((2, n), device=DEV)
    ids, logs = torch.empty((n, 2), dtype=torch.int64, device=DEV), torch.empty((n, 2), device=DEV)
    size = (am.BF16, n, d, vocab)
    am.token_logprobs(X, W, *size, tokens, logprob, entropy,
                      torch.empty(am.token_logprobs_workspace_bytes(*size, 2), dtype=torch.uint8, device=DEV),
                      top=2, top_ids=ids, top_logprobs=logs)
    lse = np.log(vocab - 1 + np.exp(20.0))
    assert ids.tolist() == [[vocab - 1, 0], [vocab - 2, 0], [-1, -1]]
    # lse 20.001: one rounding of it is 1e-6, beside sums of 5e5 equal terms
    assert np.allclose(logs.cpu()[:2], [[20.0 - lse, -lse]] * 2, rtol=1e-6, atol=3e-6)
    assert np.allclose(logprob.cpu(), [20.0 - lse, -lse, 0.0], rtol=1e-6, atol=3e-6)
    H = lse - np.exp(20.0 - lse) * 20.0
    assert np.allclose(entropy.cpu(), [H, H, 0.0], rtol=1e-4, atol=1e-7)
