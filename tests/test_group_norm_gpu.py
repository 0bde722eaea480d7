"""Group norm with an activation against the fp64 oracle, through the C ABI.

Bounds from the arithmetic, with u = 2^-24 and r roundings on the longest way of a sum (a lane's 32
values, the halving of 64 lanes; over spans of positions 6 for each union of two partial sums, span / 4
of them in a lane, at most 256 lanes of a channel and splits * vectors / 64 in the reduction):
  mean  r u mean|x|;  xh: dxh = r u mean|x| rstd + (r + 10) u |xh|;  z: |gamma| dxh + 4 u (|gamma xh| + |beta|)
  silu  slope at most 1.1, itself within (|z| + 8) 2u of its value, the slope's slope at most 0.5
and the output's one rounding (2^-8 for bf16, u for fp32), carried through the formulas of the gradients.
"""

import numpy as np
import pytest

from helpers import DEV, log
from oracle import group_norm as gn
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


def ways(n, L, C):
    return 64 if L == 1 and C <= 256 else 64 + 6 * (L // 64 + 16 + 256 + 2048 * 4 // 64)


class Case:
    def __init__(self, dtype, n, L, C, G, silu, seed=0, offset=1.0, std=1.5, affine=True):
        import torch
        rng = np.random.default_rng(seed)
        self.dtype, self.n, self.L, self.C, self.G, self.silu = dtype, n, L, C, G, silu
        dt = torch.bfloat16 if dtype == am.BF16 else torch.float32
        x = rng.standard_normal((n, L, C)) * std + offset * rng.standard_normal(C)
        self.X = torch.from_numpy(x.astype(np.float32)).to(dt)
        self.dY = torch.from_numpy(rng.standard_normal((n, L, C)).astype(np.float32)).to(dt)
        self.gamma = (1 + 0.3 * rng.standard_normal(C)).astype(np.float32) if affine else None
        self.beta = (0.3 * rng.standard_normal(C)).astype(np.float32) if affine else None

    def size(self):
        return (self.dtype, self.n, self.L, self.C, self.G)

    def affine(self):
        import torch
        if self.gamma is None:
            return None, None
        return torch.from_numpy(self.gamma).to(DEV), torch.from_numpy(self.beta).to(DEV)

    def act(self):
        return am.ACT_SILU if self.silu else am.ACT_NONE

    def workspace(self, backward):
        import torch
        n = am.group_norm_workspace_bytes(self.n, self.L, self.C, self.G, backward)
        return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)

    def run(self, X=None, dY=None, Y=None, dX=None, stream=None, ws=None):
        import torch
        X = self.X.to(DEV) if X is None else X
        dY = self.dY.to(DEV) if dY is None else dY
        Y = torch.full_like(X, 7.0) if Y is None else Y
        dX = torch.full_like(X, 7.0) if dX is None else dX
        mean, rstd = torch.full((2, self.n, self.G), 7.0, device=DEV)
        ga, be = self.affine()
        dga, dbe = torch.full((2, self.C), 7.0, device=DEV)
        w = ws or (self.workspace(False), self.workspace(True))
        if stream is not None:
            torch.cuda.synchronize()
        am.group_norm(X, *self.size(), ga, be, EPS, self.act(), Y, mean=mean, rstd=rstd, workspace=w[0], stream=stream)
        am.group_norm_backward(X, dY, *self.size(), ga, be, mean, rstd, self.act(), dX, dgamma=dga, dbeta=dbe,
                               workspace=w[1], stream=stream)
        torch.cuda.synchronize()
        return Y, mean, rstd, dX, dga, dbe


def within(name, got, want, bound):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), name
    ratio = float(np.max(np.abs(got - want) / (bound + 1e-30)))
    log(f"PARITY {name}: {ratio:.3f} of the bound")
    assert ratio <= 1.0, (name, ratio)


def check(c):
    log(f"CASE {c.size()} silu {c.silu}")
    Y, mean, rstd, dX, dga, dbe = c.run()
    x, dy = c.X.double().numpy(), c.dY.double().numpy()
    ga = np.ones(c.C) if c.gamma is None else c.gamma.astype(np.float64)
    be = np.zeros(c.C) if c.beta is None else c.beta.astype(np.float64)
    y, m, rs = gn.forward(x, c.G, ga, be, EPS, c.silu)
    r = ways(c.n, c.L, c.C)
    out = 2.0 ** -8 if c.dtype == am.BF16 else U

    def spread(s):
        return np.repeat(s, c.C // c.G, axis=-1)[:, None, :]

    def mean_of(v):
        return v.reshape(c.n, c.L, c.G, -1).mean((1, 3))

    mx = mean_of(np.abs(x))
    xh = gn.normalised(x, c.G, m, rs)
    z = xh * ga + be
    dxh = r * U * spread(mx * rs) + (r + 10) * U * np.abs(xh)
    sh = (np.abs(z) + 8) * 2 * U if c.silu else 0.0
    dz_fwd = np.abs(ga) * dxh + 4 * U * (np.abs(ga * xh) + np.abs(be))
    slope = 1.1 if c.silu else 1.0
    within("Y", Y, y, out * np.abs(y) + slope * dz_fwd + sh * np.abs(z))
    within("mean", mean, m, r * U * mx + U * np.abs(m))
    within("rstd", rstd, rs, rs * (r + 10) * U + rs ** 3 * (r * U * mx) ** 2)
    dx, dg, db = gn.backward(x, dy, c.G, ga, be, EPS, c.silu)
    s = gn._sigmoid(z)
    dz = dy * (s * (1 + z * (1 - s))) if c.silu else dy
    e_dz = np.abs(dy) * (0.5 * dz_fwd + sh * 1.1) if c.silu else 0.0 * np.abs(dy)
    h = dz * ga
    e_h = np.abs(ga) * e_dz + U * np.abs(h)
    e_s1 = mean_of(e_h) + r * U * mean_of(np.abs(h))
    e_s2 = mean_of(e_h * np.abs(xh) + np.abs(h) * dxh) + r * U * mean_of(np.abs(h * xh))
    s1, s2 = spread(np.abs(mean_of(h))), spread(np.abs(mean_of(h * xh)))
    bound = spread(rs) * (e_h + spread(e_s1) + np.abs(xh) * spread(e_s2) + dxh * s2
                          + 4 * U * (np.abs(h) + s1 + np.abs(xh) * s2)) + ((r + 10) * U + out) * np.abs(dx)
    within("dX", dX, dx, bound)
    deep = r + c.n * c.L / 16
    within("dgamma", dga, dg, (e_dz * np.abs(xh) + np.abs(dz) * dxh + deep * U * np.abs(dz * xh)).sum((0, 1)))
    within("dbeta", dbe, db, (e_dz + deep * U * np.abs(dz)).sum((0, 1)))


CASES = [
    ("one_row", dict(dtype=am.BF16, n=1, L=1, C=1024, G=16, silu=True)),
    ("one_value", dict(dtype=am.F32, n=1, L=1, C=4, G=1, silu=False)),
    ("groups_of_one", dict(dtype=am.F32, n=5, L=1, C=7, G=7, silu=False)),
    ("heads", dict(dtype=am.BF16, n=700, L=1, C=512, G=4, silu=False)),
    ("heads_odd", dict(dtype=am.BF16, n=131, L=1, C=3 * 33, G=3, silu=True)),
    ("heads_100", dict(dtype=am.F32, n=77, L=1, C=500, G=5, silu=True)),
    ("wide_row", dict(dtype=am.BF16, n=33, L=1, C=2048, G=1, silu=True)),
    ("wider_than_a_wave", dict(dtype=am.F32, n=9, L=1, C=4104, G=1, silu=True)),
    ("odd_wider_than_a_wave", dict(dtype=am.BF16, n=9, L=1, C=1501, G=1, silu=False)),
    ("few_positions", dict(dtype=am.BF16, n=600, L=3, C=64, G=4, silu=True)),
    ("few_positions_odd", dict(dtype=am.F32, n=40, L=7, C=60, G=5, silu=False)),
    ("positions", dict(dtype=am.F32, n=3, L=1025, C=96, G=8, silu=True)),
    ("positions_bf16", dict(dtype=am.BF16, n=2, L=4999, C=40, G=2, silu=False)),
    ("positions_odd", dict(dtype=am.BF16, n=2, L=333, C=21, G=3, silu=True)),
    ("positions_wide", dict(dtype=am.F32, n=2, L=50, C=4096, G=2, silu=True)),
    ("many_samples", dict(dtype=am.F32, n=3000, L=40, C=24, G=2, silu=False)),
    ("heads_walked", dict(dtype=am.BF16, n=9001, L=1, C=1024, G=8, silu=True)),
    ("few_positions_walked", dict(dtype=am.F32, n=9001, L=2, C=512, G=8, silu=False)),
    ("no_affine", dict(dtype=am.BF16, n=50, L=1, C=256, G=2, silu=True, affine=False)),
    ("no_affine_positions", dict(dtype=am.F32, n=2, L=500, C=32, G=2, silu=True, affine=False)),
    ("far_from_zero", dict(dtype=am.F32, n=20, L=1, C=128, G=2, silu=False, offset=500.0, std=0.5)),
    ("far_from_zero_positions", dict(dtype=am.F32, n=2, L=600, C=32, G=32, silu=False, offset=300.0, std=0.5)),
]


@pytest.mark.parametrize("kw", [c[1] for c in CASES], ids=[c[0] for c in CASES])
def test_parity(kw):
    check(Case(**kw))


@pytest.mark.parametrize("L", [1, 300])
def test_gamma_alone_and_gradients_that_are_not_asked_for(L):
    import torch
    c = Case(am.F32, 6, L, 64, 4, True)
    X, dY, (ga, be) = c.X.to(DEV), c.dY.to(DEV), c.affine()
    for g, b, none in ((ga, None, torch.zeros_like(be)), (None, be, torch.ones_like(ga))):
        full = (ga, none) if b is None else (none, be)
        got = []
        for g_, b_ in ((g, b), full):
            Y, dX = torch.empty_like(X), torch.empty_like(X)
            mean, rstd = torch.empty((2, c.n, c.G), device=DEV)
            am.group_norm(X, *c.size(), g_, b_, EPS, c.act(), Y, mean=mean, rstd=rstd, workspace=c.workspace(False))
            Y2 = torch.empty_like(X)
            am.group_norm(X, *c.size(), g_, b_, EPS, c.act(), Y2, workspace=c.workspace(False))
            dga, dbe = torch.empty((2, c.C), device=DEV)
            dX2, dX3, dga2 = torch.empty_like(X), torch.empty_like(X), torch.empty_like(dga)
            back = (X, dY, *c.size(), g_, b_, mean, rstd, c.act())
            am.group_norm_backward(*back, dX, dgamma=dga, dbeta=dbe, workspace=c.workspace(True))
            am.group_norm_backward(*back, dX2, workspace=c.workspace(True))
            am.group_norm_backward(*back, dX3, dgamma=dga2, workspace=c.workspace(True))
            assert torch.equal(Y, Y2) and torch.equal(dX, dX2) and torch.equal(dX, dX3) and torch.equal(dga, dga2)
            got.append((Y, mean, rstd, dX, dga, dbe))
        assert all(torch.equal(p, q) for p, q in zip(*got))


def test_equal_values_give_beta():
    import torch
    c = Case(am.F32, 4, 1, 64, 2, False)
    c.X = torch.full_like(c.X, 3.25)
    Y, mean, rstd, *_ = c.run()
    assert torch.equal(Y.cpu(), torch.from_numpy(c.beta).expand(4, 1, 64))
    assert float(mean.min()) == 3.25 and abs(float(rstd.max()) * EPS ** 0.5 - 1) < 1e-6


@pytest.mark.parametrize("kw", [dict(n=40, L=1, C=256, G=2), dict(n=2, L=700, C=64, G=4)])
def test_in_place(kw):
    c = Case(am.BF16, silu=True, **kw)
    import torch
    a = c.run()
    X = c.X.to(DEV)
    ga, be = c.affine()
    am.group_norm(X, *c.size(), ga, be, EPS, c.act(), X, workspace=c.workspace(False))
    assert torch.equal(X, a[0])
    for over in ("X", "dY"):
        X, dY = c.X.to(DEV), c.dY.to(DEV)
        dX = X if over == "X" else dY
        am.group_norm_backward(X, dY, *c.size(), ga, be, a[1], a[2], c.act(), dX, workspace=c.workspace(True))
        torch.cuda.synchronize()
        assert torch.equal(dX, a[3])


@pytest.mark.parametrize("kw", [dict(n=50, L=1, C=256, G=4), dict(n=2, L=700, C=64, G=4)])
def test_unaligned_and_other_streams(kw):
    import torch
    c = Case(am.BF16, silu=True, **kw)
    a = c.run()
    b = c.run(stream=torch.cuda.Stream())
    assert all(torch.equal(x, y) for x, y in zip(a, b))

    def shifted(x):
        s = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
        return s.copy_(x)

    u = c.run(X=shifted(c.X), dY=shifted(c.dY), Y=shifted(c.X), dX=shifted(c.X))
    for x, y in zip(a, u):  # other lanes, other orders of the sums
        d = (x.double() - y.double()).abs().max() / x.double().abs().max()
        assert float(d) <= (2.0 ** -7 if x.dtype == torch.bfloat16 else 1e-5)


def test_a_sample_with_nan_stays_by_itself():
    import torch
    for kw in (dict(n=6, L=1, C=64, G=2), dict(n=6, L=300, C=64, G=2)):
        c = Case(am.F32, silu=True, **kw)
        a = c.run()
        c.X[2, 0, 3] = float("nan")
        c.X[4, 0, 40] = float("inf")
        b = c.run()
        for i in (0, 1, 3, 5):
            assert torch.equal(a[0][i], b[0][i]) and torch.equal(a[3][i], b[3][i])
        assert torch.isnan(b[0][2, :, :32]).all() and torch.equal(a[0][2, :, 32:], b[0][2, :, 32:])


def test_no_samples():
    import torch
    X = torch.zeros((0, 1, 16), device=DEV)
    dga, dbe = torch.full((2, 16), 7.0, device=DEV)
    ws = torch.zeros(16, dtype=torch.uint8, device=DEV)
    am.group_norm_backward(X, X, am.F32, 0, 1, 16, 2, None, None, None, None, 0, X, dgamma=dga, dbeta=dbe, workspace=ws)
    assert not dga.any() and not dbe.any()


@pytest.mark.parametrize("kw", [dict(n=50, L=1, C=256, G=4), dict(n=2, L=700, C=64, G=4)])
def test_captured_and_replayed(kw):
    import torch
    c = Case(am.BF16, silu=True, **kw)
    X, dY = c.X.to(DEV), c.dY.to(DEV)
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    mean, rstd = torch.empty((2, c.n, c.G), device=DEV)
    dga, dbe = torch.empty((2, c.C), device=DEV)
    ga, be = c.affine()
    w = c.workspace(False), c.workspace(True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        am.group_norm(X, *c.size(), ga, be, EPS, c.act(), Y, mean=mean, rstd=rstd, workspace=w[0])
        am.group_norm_backward(X, dY, *c.size(), ga, be, mean, rstd, c.act(), dX, dgamma=dga, dbeta=dbe, workspace=w[1])
    for i in range(3):
        d = Case(am.BF16, silu=True, seed=5 + i, **kw)
        d.gamma, d.beta = c.gamma, c.beta
        X.copy_(d.X)
        dY.copy_(d.dY)
        graph.replay()
        torch.cuda.synchronize()
        want = d.run()
        assert all(torch.equal(x, y) for x, y in zip((Y, mean, rstd, dX, dga, dbe), want))


def test_offsets_past_32_bits():
    import torch
    n, L, C = 1, 1100000, 2048
    X = torch.zeros((n, L, C), dtype=torch.bfloat16, device=DEV)
    X[0, -1, -1] = 4.0
    X[0, -1, 0] = -4.0
    Y = torch.empty_like(X)
    ws = torch.empty(am.group_norm_workspace_bytes(n, L, C, 2), dtype=torch.uint8, device=DEV)
    mean, rstd = torch.empty((2, n, 2), device=DEV)
    am.group_norm(X, am.BF16, n, L, C, 2, None, None, 0.0, am.ACT_NONE, Y, mean=mean, rstd=rstd, workspace=ws)
    count = L * C / 2
    want = (count - 1) ** 0.5    # one value 4 among zeros: (4 - 4 / count) / sqrt(16 (1 / count - 1 / count^2))
    assert abs(float(Y[0, -1, -1]) / want - 1) < 2 ** -7 and abs(float(Y[0, -1, 0]) / -want - 1) < 2 ** -7
