"""Linear attention with a decay for each head against the fp64 oracle, through the C ABI.

The bound of every element, from the arithmetic: |got - want| <= out |want| + e A, with A the sum of
the absolute values of the terms (the oracle on absolute inputs) and
  out  one rounding to the output type: 2^-8 for bf16, 2^-24 for fp32;
  e    computed operands in two bf16 planes, 2^-18 relative each, two in a product (bf16 calls), or
       in three planes, 2^-26 each and the dropped products 3 x 2^-25 (fp32 calls and every state);
       plus 2^-24 for each fp32 rounding on a term's way: at most 18 products of planes a step,
       (d / 16 + 8) steps for the outputs and 13 roundings for each further chunk the state passes,
       and the table of powers (an argument's rounding, at most 88 x 2^-24, and 2 ulp).
"""

import numpy as np
import pytest

from helpers import DEV, log
from oracle import linear_attention as la
from test_learned_neural_amd import atlasmem as am

pytestmark = pytest.mark.gpu


def roundings(T, d):
    return 18 * (d // 16 + 9) + 26 * (T // 64 + 1) + 92


def term_bound(dtype, T, d):
    planes = 2.0 ** -16 if dtype == am.BF16 else 2.0 ** -22
    return planes + roundings(T, d) * 2.0 ** -24


def state_bound(T, d):
    return 2.0 ** -22 + roundings(T, d) * 2.0 ** -24


def torch_dtype(dtype):
    import torch
    return torch.bfloat16 if dtype == am.BF16 else torch.float32


class Case:
    def __init__(self, dtype, B, H, T, dk, dv, layout=am.HEADS_FIRST, lengths=None, decays=None, seed=0, state=True):
        import torch
        self.dtype, self.B, self.H, self.T, self.dk, self.dv, self.layout = dtype, B, H, T, dk, dv, layout
        self.scale = dk ** -0.5
        rng = np.random.default_rng(seed)
        dt = torch_dtype(dtype)

        def rows(w):
            x = torch.from_numpy(rng.standard_normal((B, H, T, w)).astype(np.float32)).to(dt)
            return x

        self.host = dict(q=rows(dk), k=rows(dk), v=rows(dv), dy=rows(dv))
        self.g = np.asarray(decays if decays is not None else np.log1p(-2.0 ** -np.linspace(1, 9, H)), dtype=np.float32)
        z = rng.standard_normal((2, B, H, dv, dk)).astype(np.float32)
        self.W0, self.dW = (z[0], z[1]) if state else (np.zeros_like(z[0]), np.zeros_like(z[1]))
        self.state = state
        self.lengths = lengths

    def dev(self, name):
        x = self.host[name]
        if self.layout == am.TOKENS_FIRST:
            x = x.transpose(1, 2)
        return x.contiguous().to(DEV)

    def out(self, w, fill=7.0):
        import torch
        shape = (self.B, self.T, self.H, w) if self.layout == am.TOKENS_FIRST else (self.B, self.H, self.T, w)
        return torch.full(shape, fill, dtype=torch_dtype(self.dtype), device=DEV)

    def np64(self, t):
        a = t.double().cpu().numpy()
        return a.swapaxes(1, 2) if self.layout == am.TOKENS_FIRST else a

    def f64(self, name):
        return self.host[name].double().numpy()

    def size(self):
        return (self.dtype, self.B, self.H, self.T, self.dk, self.dv)

    def tensors(self):
        import torch
        d = {n: self.dev(n) for n in ("q", "k", "v", "dy")}
        d["g"] = torch.from_numpy(self.g).to(DEV)
        d["len"] = None if self.lengths is None else torch.tensor(self.lengths, dtype=torch.int32, device=DEV)
        d["W0"] = torch.from_numpy(self.W0).to(DEV) if self.state else None
        d["dW"] = torch.from_numpy(self.dW).to(DEV) if self.state else None
        return d

    def workspace(self, backward):
        import torch
        n = am.linear_attention_workspace_bytes(*self.size(), backward)
        return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device=DEV)  # NaN everywhere

    def forward(self, d, Y, W_T, ws, stream=None):
        am.linear_attention(d["q"], d["k"], d["v"], *self.size(), d["g"], self.scale, Y, W0=d["W0"], W_T=W_T,
                            lengths=d["len"], layout=self.layout, workspace=ws, stream=stream)

    def outputs(self):
        import torch
        return dict(dQ=self.out(self.dk), dK=self.out(self.dk), dV=self.out(self.dv),
                    dW0=torch.full((self.B, self.H, self.dv, self.dk), 7.0, device=DEV),
                    dlog_decay=torch.full((self.H,), 7.0, device=DEV))

    def backward(self, d, o, ws, stream=None):
        am.linear_attention_backward(d["q"], d["k"], d["v"], *self.size(), d["g"], self.scale, d["dy"], W0=d["W0"],
                                     dW_T=d["dW"], lengths=d["len"], layout=self.layout, workspace=ws, stream=stream,
                                     **o)


def within(name, got, want, A, out, e):
    bound = out * np.abs(want) + e * A + 1e-30
    ratio = float(np.max(np.abs(got - want) / bound)) if got.size else 0.0
    log(f"PARITY {name}: {ratio:.3f} of the bound")
    assert np.isfinite(got).all(), name
    assert ratio <= 1.0, (name, ratio)


def check_forward(c):
    import torch
    log(f"CASE forward {c.size()} layout {c.layout} lengths {c.lengths}")
    d, Y, ws = c.tensors(), c.out(c.dv), c.workspace(False)
    W_T = torch.full((c.B, c.H, c.dv, c.dk), 7.0, device=DEV)
    c.forward(d, Y, W_T, ws)
    torch.cuda.synchronize()
    q, k, v = c.f64("q"), c.f64("k"), c.f64("v")
    y, W = la.forward(q, k, v, c.g, c.scale, c.W0, c.lengths)
    ya, Wa = la.forward(abs(q), abs(k), abs(v), c.g, c.scale, abs(c.W0), c.lengths)
    step = 2.0 ** -8 if c.dtype == am.BF16 else 2.0 ** -24
    within("Y", c.np64(Y), y, ya, step, term_bound(c.dtype, c.T, c.dk))
    within("W_T", W_T.double().cpu().numpy(), W, Wa, 2.0 ** -24, state_bound(c.T, c.dk))


def check_backward(c):
    import torch
    log(f"CASE backward {c.size()} layout {c.layout} lengths {c.lengths}")
    d, o, ws = c.tensors(), c.outputs(), c.workspace(True)
    c.backward(d, o, ws)
    torch.cuda.synchronize()
    args = [c.f64("q"), c.f64("k"), c.f64("v"), c.g, c.scale, c.W0, c.f64("dy"), c.dW]
    want = la.backward(*args, c.lengths)
    mags = la.backward(*[abs(x) if i not in (3, 4) else x for i, x in enumerate(args)], c.lengths)
    step = 2.0 ** -8 if c.dtype == am.BF16 else 2.0 ** -24
    e, es = term_bound(c.dtype, c.T, max(c.dk, c.dv)), state_bound(c.T, max(c.dk, c.dv))
    for i, n in enumerate(("dQ", "dK", "dV")):
        within(n, c.np64(o[n]), want[i], mags[i], step, e)
    within("dW0", o["dW0"].double().cpu().numpy(), want[3], mags[3], 2.0 ** -24, es)
    # the tangent's shares: one more factor (a count) and one more product
    within("dlog_decay", o["dlog_decay"].double().cpu().numpy(), want[4], mags[4], 2.0 ** -24, 2 * es)


CASES = [
    ("one_token", dict(dtype=am.BF16, B=2, H=3, T=1, dk=64, dv=64)),
    ("two_tokens_f32", dict(dtype=am.F32, B=1, H=2, T=2, dk=20, dv=33, layout=am.TOKENS_FIRST)),
    ("width_one", dict(dtype=am.F32, B=1, H=2, T=5, dk=1, dv=1)),
    ("width_one_chunked", dict(dtype=am.BF16, B=1, H=2, T=70, dk=1, dv=1)),
    ("last_step", dict(dtype=am.BF16, B=1, H=4, T=16, dk=128, dv=128, layout=am.TOKENS_FIRST)),
    ("first_chunked", dict(dtype=am.BF16, B=1, H=4, T=17, dk=128, dv=128)),
    ("chunk_less_one", dict(dtype=am.F32, B=1, H=2, T=63, dk=32, dv=64)),
    ("chunk", dict(dtype=am.BF16, B=2, H=2, T=64, dk=64, dv=128)),
    ("chunk_and_one", dict(dtype=am.F32, B=1, H=2, T=65, dk=64, dv=32, layout=am.TOKENS_FIRST)),
    ("odd_widths", dict(dtype=am.BF16, B=1, H=3, T=150, dk=50, dv=23)),
    ("odd_widths_f32", dict(dtype=am.F32, B=1, H=3, T=150, dk=101, dv=66, layout=am.TOKENS_FIRST)),
    ("wide_narrow", dict(dtype=am.BF16, B=1, H=2, T=200, dk=128, dv=24)),
    ("narrow_wide", dict(dtype=am.BF16, B=1, H=2, T=200, dk=24, dv=128)),
    ("wide_narrow_padded", dict(dtype=am.BF16, B=3, H=2, T=600, dk=96, dv=40, lengths=[600, 0, 333],
                                layout=am.TOKENS_FIRST)),
    ("wide_narrow_odd_f32", dict(dtype=am.F32, B=1, H=3, T=555, dk=73, dv=33)),
    ("narrow_wide_segments", dict(dtype=am.BF16, B=2, H=1, T=1000, dk=36, dv=100, lengths=[999, 37])),
    ("segments", dict(dtype=am.BF16, B=1, H=3, T=1500, dk=64, dv=64, layout=am.TOKENS_FIRST)),
    ("segments_f32", dict(dtype=am.F32, B=1, H=2, T=900, dk=128, dv=128)),
    ("padded", dict(dtype=am.BF16, B=5, H=2, T=330, dk=64, dv=64, lengths=[330, 0, 1, 64, 257])),
    ("padded_rows", dict(dtype=am.F32, B=4, H=2, T=700, dk=40, dv=48, lengths=[1000, -3, 700, 65],
                         layout=am.TOKENS_FIRST)),
    ("padded_step", dict(dtype=am.F32, B=3, H=2, T=4, dk=40, dv=48, lengths=[4, 0, 2])),
    ("no_state", dict(dtype=am.BF16, B=1, H=2, T=100, dk=64, dv=64, state=False)),
    ("no_decay", dict(dtype=am.F32, B=1, H=2, T=300, dk=32, dv=32, decays=[0.0, -0.0])),
    ("no_memory", dict(dtype=am.F32, B=1, H=3, T=130, dk=32, dv=32, decays=[-np.inf, -200.0, -5.0])),
    ("no_memory_step", dict(dtype=am.F32, B=1, H=2, T=3, dk=32, dv=32, decays=[-np.inf, -30.0])),
]


@pytest.mark.parametrize("kw", [c[1] for c in CASES], ids=[c[0] for c in CASES])
def test_forward(kw):
    check_forward(Case(**kw))


@pytest.mark.parametrize("kw", [c[1] for c in CASES], ids=[c[0] for c in CASES])
def test_backward(kw):
    if kw.get("decays") is not None and not np.isfinite(kw["decays"]).all():
        kw = dict(kw, decays=[g if np.isfinite(g) else -150.0 for g in kw["decays"]])
    check_backward(Case(**kw))


def test_no_tokens():
    import torch
    c = Case(am.F32, 1, 2, 0, 8, 8)
    d, W_T = c.tensors(), torch.zeros((1, 2, 8, 8), device=DEV)
    c.forward(d, c.out(8), W_T, None)
    assert torch.equal(W_T, d["W0"])
    o = c.outputs()
    c.backward(d, o, c.workspace(True))
    assert torch.equal(o["dW0"], d["dW"]) and not o["dlog_decay"].any()


def test_infinite_forgetting_has_finite_gradients():
    import torch
    c = Case(am.F32, 1, 1, 100, 16, 16, decays=[-np.inf])
    d, o = c.tensors(), c.outputs()
    c.backward(d, o, c.workspace(True))
    torch.cuda.synchronize()
    want = la.backward(c.f64("q"), c.f64("k"), c.f64("v"), [-200.0], c.scale, c.W0, c.f64("dy"), c.dW)
    for i, n in enumerate(("dQ", "dK", "dV")):
        assert np.abs(c.np64(o[n]) - want[i]).max() <= 1e-5 * np.abs(want[i]).max()
    assert not o["dlog_decay"].any()


@pytest.mark.parametrize("T", [3, 200])
def test_padding_is_not_read(T):
    import torch
    lengths = [T - 1, 0, 1]
    c = Case(am.BF16, 3, 2, T, 32, 32, lengths=lengths)
    e = Case(am.BF16, 3, 2, T, 32, 32, lengths=lengths)
    for n in ("q", "k", "v", "dy"):
        for b, L in enumerate(lengths):
            e.host[n][b, :, L:] = float("nan")
    got = []
    for x in (c, e):
        d, Y, W_T = x.tensors(), x.out(32), torch.empty((3, 2, 32, 32), device=DEV)
        x.forward(d, Y, W_T, x.workspace(False))
        o = x.outputs()
        x.backward(d, o, x.workspace(True))
        got.append([Y, W_T, *o.values()])
    for a, b in zip(*got):
        assert torch.equal(a, b)
        assert torch.isfinite(a.float()).all()


@pytest.mark.parametrize("T", [1, 500])
def test_state_in_place_and_cut_into_calls(T):
    import torch
    c = Case(am.F32, 2, 2, T, 64, 48)
    d, Y, ws = c.tensors(), c.out(48), c.workspace(False)
    W_T = torch.empty_like(d["W0"])
    c.forward(d, Y, W_T, ws)
    Y2, W = c.out(48), d["W0"].clone()
    d2 = dict(d, W0=W)
    c.forward(d2, Y2, W, ws)
    assert torch.equal(Y, Y2) and torch.equal(W, W_T)
    # the same tokens in calls of 1, 7, 100 and the rest
    W, at = d["W0"].clone(), 0
    for n in (1, 7, 100, T):
        n = min(n, T - at)
        p = Case(am.F32, 2, 2, n, 64, 48)
        dp = dict(d, **{x: d[x][:, :, at:at + n].contiguous() for x in "qkv"}, W0=W)
        Yp = p.out(48)
        p.forward(dp, Yp, W, p.workspace(False))
        assert n == 0 or float((Yp - Y[:, :, at:at + n]).abs().max()) <= 1e-4 * float(Y.abs().max())
        at += n
    assert float((W - W_T).abs().max()) <= 1e-5 * float(W_T.abs().max())


@pytest.mark.parametrize("T,dv", [(70, 64), (900, 128), (900, 24)])
def test_gradients_that_are_not_asked_for_and_a_state_adjoint_in_place(T, dv):
    import torch
    c = Case(am.BF16, 1, 3, T, 72, dv)
    d, o = c.tensors(), c.outputs()
    c.backward(d, o, c.workspace(True))
    some = c.outputs()
    c.backward(d, dict(some, dW0=None, dlog_decay=None), c.workspace(True))
    for n in ("dQ", "dK", "dV"):
        assert float((some[n].float() - o[n].float()).abs().max()) <= 2 ** -7 * float(o[n].float().abs().max())
    A = d["dW"].clone()
    here = c.outputs()
    c.backward(dict(d, dW=A), dict(here, dW0=A), c.workspace(True))
    assert torch.equal(A, o["dW0"]) and torch.equal(here["dlog_decay"], o["dlog_decay"])
    for n in ("dQ", "dK", "dV"):
        assert torch.equal(here[n], o[n])


def test_unaligned_rows_equal_aligned_ones():
    import torch
    c = Case(am.BF16, 1, 2, 150, 64, 64)
    d, Y, W_T = c.tensors(), c.out(64), torch.empty((1, 2, 64, 64), device=DEV)
    c.forward(d, Y, W_T, c.workspace(False))

    def shifted(x):
        s = torch.empty(x.numel() + 1, dtype=x.dtype, device=DEV)[1:].view(x.shape)
        return s.copy_(x)

    d2 = dict(d, **{n: shifted(d[n]) for n in ("q", "k", "v", "W0")})
    Y2, W2 = shifted(c.out(64)), shifted(W_T)
    c.forward(d2, Y2, W2, c.workspace(False))
    assert torch.equal(Y, Y2) and torch.equal(W_T, W2)


def test_equal_calls_give_equal_bits_on_any_stream():
    import torch
    c = Case(am.BF16, 2, 3, 1000, 64, 64, lengths=[1000, 421])
    d = c.tensors()
    torch.cuda.synchronize()
    got = []
    for s in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        Y, W_T, o, w1, w2 = c.out(64), torch.empty_like(d["W0"]), c.outputs(), c.workspace(False), c.workspace(True)
        torch.cuda.synchronize()
        c.forward(d, Y, W_T, w1, stream=s)
        c.backward(d, o, w2, stream=s)
        got.append([Y, W_T, *o.values()])
    torch.cuda.synchronize()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("T", [1, 700])
def test_captured_and_replayed(T):
    import torch
    c = Case(am.BF16, 1, 2, T, 64, 64)
    d, Y, ws, wb = c.tensors(), c.out(64), c.workspace(False), c.workspace(True)
    W_T, o = torch.empty_like(d["W0"]), c.outputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.forward(d, Y, W_T, ws)
        c.backward(d, o, wb)
    for i in range(3):
        x = Case(am.BF16, 1, 2, T, 64, 64, seed=10 + i)
        new = x.tensors()
        for n in ("q", "k", "v", "dy", "W0", "dW"):
            d[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        Y2, W2, o2 = x.out(64), torch.empty_like(W_T), x.outputs()
        x.forward(new, Y2, W2, x.workspace(False))
        x.backward(new, o2, x.workspace(True))
        torch.cuda.synchronize()
        assert torch.equal(Y, Y2) and torch.equal(W_T, W2)
        assert all(torch.equal(o[n], o2[n]) for n in o)


def test_offsets_past_32_bits():
    """More than 2^31 elements of q: the last rows of the last head are read and written where they are."""
    import torch
    B, H, T, dk, dv = 1, 2, 8400000, 128, 8
    q = torch.zeros((B, H, T, dk), dtype=torch.bfloat16, device=DEV)
    k, v = torch.zeros_like(q), torch.zeros((B, H, T, dv), dtype=torch.bfloat16, device=DEV)
    q[0, 1, -1, 5] = 3.0
    k[0, 1, -2, 5] = 2.0
    v[0, 1, -2, 7] = 1.5
    g = torch.tensor([-1.0, -0.5], device=DEV)
    Y = torch.full_like(v, 9.0)
    n = am.linear_attention_workspace_bytes(am.BF16, B, H, T, dk, dv)
    am.linear_attention(q, k, v, am.BF16, B, H, T, dk, dv, g, 1.0, Y, workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    want = torch.tensor(3.0 * 2.0 * 1.5 * np.exp(-0.5)).bfloat16().float()
    assert abs(float(Y[0, 1, -1, 7]) - float(want)) <= 2.0 ** -7 * float(want)
    Y[0, 1, -1, 7] = 0
    assert not Y.any()
