"""A teacher's alternatives and the student that learns from them, together as they are used: linear attention (or the
memory itself) -> group norm -> log probabilities and alternatives of one model, -> distillation of another, and back.

Bars: the library's own parity bars for fp32 and bf16 paths (1e-4 and 2e-2 of the tensor's largest value), against the
same chain in fp64; the alternatives have to be those of the teacher's rows in fp64.
"""

import numpy as np
import pytest

import oracle
from helpers import BF16_TOL, DEV, F32_TOL, config_for, to_dev
from oracle import backward as bw
from oracle import distillation as ds
from oracle import group_norm as gn
from oracle import linear_attention as la
from oracle import token_logprobs as tl
from test_learned_neural_amd import atlasmem as am
from test_learned_neural_amd import synth
from test_training_path_gpu import EPS, Norm, check, torch_dtype, workspace

pytestmark = pytest.mark.gpu


class Teacher:
    """Alternatives of rows: what a student is given."""

    def __init__(self, dtype, n, d, W, tokens, top):
        import torch
        self.size, self.top = (dtype, n, d, len(W)), top
        self.W, self.tokens = torch.from_numpy(W).to(torch_dtype(dtype)).to(DEV), to_dev(tokens)
        self.logprob, self.entropy = torch.empty((2, n), device=DEV)
        self.ids = torch.empty((n, top), dtype=torch.int64, device=DEV)
        self.logs = torch.empty((n, top), device=DEV)
        self.ws = workspace(am.token_logprobs_workspace_bytes(*self.size, top))

    def forward(self, X):
        am.token_logprobs(X, self.W, *self.size, self.tokens, self.logprob, self.entropy, self.ws, top=self.top,
                          top_ids=self.ids, top_logprobs=self.logs)


class Student:
    def __init__(self, dtype, n, d, W, top, scale, dloss):
        import torch
        self.size, self.scale = (dtype, n, d, len(W), top), scale
        self.W, self.dloss = torch.from_numpy(W).to(torch_dtype(dtype)).to(DEV), to_dev(dloss)
        self.loss, self.lse = torch.empty((2, n), device=DEV)
        self.dW = torch.empty_like(self.W)
        self.ws = workspace(am.distillation_workspace_bytes(*self.size, True))
        self.kept = workspace(am.distillation_kept_bytes(dtype, n, len(W), top))

    def forward(self, X, ids, logs):
        am.distillation(X, self.W, *self.size, ids, logs, self.scale, self.loss, self.lse, self.ws, kept=self.kept)

    def backward(self, X, dX):
        am.distillation_backward(X, self.W, *self.size, self.kept, self.dloss, dX, self.dW, self.ws)


def rounded(x, dtype):
    import torch
    return torch.from_numpy(x.astype(np.float32)).to(torch_dtype(dtype)).float().numpy()


@pytest.mark.parametrize("dtype,captured", [(am.F32, False), (am.BF16, False), (am.BF16, True)])
def test_teacher_to_student_and_back(dtype, captured):
    import torch
    rng = np.random.default_rng(6)
    B, T, H, dk, dv, vocab, top, temper = 2, 260, 4, 32, 48, 1203, 12, 0.5
    n, d = B * T, H * dv
    dt = torch_dtype(dtype)
    host = {k: torch.from_numpy(rng.standard_normal((B, T, H, w)).astype(np.float32)).to(dt)
            for k, w in (("q", dk), ("k", dk), ("v", dv))}
    q, k, v = (host[x].to(DEV) for x in "qkv")
    g = np.log1p(-2.0 ** -np.linspace(2, 8, H)).astype(np.float32)
    gamma, beta = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32), (0.2 * rng.standard_normal(d)).astype(np.float32)
    Wt, Wv = (rounded(rng.standard_normal((vocab, d)) * 2 * d ** -0.5, dtype) for _ in range(2))
    tokens = rng.integers(0, vocab, n)
    tokens[rng.random(n) < 0.25] = -100                       # padding: no alternatives, and left out of the loss
    dloss = np.full(n, 1.0 / (tokens >= 0).sum(), dtype=np.float32)
    scale = dk ** -0.5
    size = (dtype, B, H, T, dk, dv)
    gd = to_dev(g)
    wa = workspace(am.linear_attention_workspace_bytes(*size, True))
    norm = Norm(dtype, n, H, dv, gamma, beta)
    teacher, student = Teacher(dtype, n, d, Wt, tokens, top), Student(dtype, n, d, Wv, top, temper, dloss)
    R = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).to(dt).to(DEV)   # the teacher's rows
    Y, Z, dZ, dY = (torch.empty((n, d), dtype=dt, device=DEV) for _ in range(4))
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty(H, device=DEV)

    def step():
        teacher.forward(R)
        am.linear_attention(q, k, v, *size, gd, scale, Y, layout=am.TOKENS_FIRST, workspace=wa)
        norm.forward(Y, Z)
        student.forward(Z, teacher.ids, teacher.logs)
        student.backward(Z, dZ)
        norm.backward(Y, dZ, dY)
        am.linear_attention_backward(q, k, v, *size, gd, scale, dY, dq, dk_, dv_, dlog_decay=dg, layout=am.TOKENS_FIRST,
                                     workspace=wa)

    outs = (teacher.ids, teacher.logs, student.loss, Z, student.dW, norm.dgamma, norm.dbeta, dq, dk_, dv_, dg)
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for _ in range(3):
            for o in outs:
                o.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, outs))
    else:
        step()
        torch.cuda.synchronize()

    lp, H_, ids, logs = tl.forward(R.double().cpu().numpy(), Wt.astype(np.float64), tokens, 1.0, top)
    assert np.array_equal(teacher.ids.cpu().numpy(), ids)
    f = {x: host[x].double().numpy().swapaxes(1, 2) for x in "qkv"}
    W0 = np.zeros((B, H, dv, dk))
    y, _ = la.forward(f["q"], f["k"], f["v"], g, scale, W0, [T] * B)
    rows = y.swapaxes(1, 2).reshape(n, 1, d)
    ga, be, Wd = gamma.astype(np.float64), beta.astype(np.float64), Wv.astype(np.float64)
    z, _, _ = gn.forward(rows, H, ga, be, EPS, True)
    wl, _ = ds.forward(z[:, 0], Wd, ids, logs, temper)
    dz, dW = ds.backward(z[:, 0], Wd, ids, logs, temper, dloss)
    dy, dga, dbe = gn.backward(rows, dz[:, None], H, ga, be, EPS, True)
    want = la.backward(f["q"], f["k"], f["v"], g, scale, W0, dy.reshape(B, T, H, dv).swapaxes(1, 2), W0, [T] * B)
    heads = lambda x: x.swapaxes(1, 2)
    check(f"student_{dtype}", BF16_TOL if dtype == am.BF16 else F32_TOL, logprob=(teacher.logprob, lp),
          entropy=(teacher.entropy, H_), logs=(teacher.logs, logs), loss=(student.loss, wl), Z=(Z, z[:, 0]),
          dW=(student.dW, dW), dgamma=(norm.dgamma, dga), dbeta=(norm.dbeta, dbe), dq=(dq, heads(want[0])),
          dk=(dk_, heads(want[1])), dv=(dv_, heads(want[2])), dlog_decay=(dg, want[4]))


def test_decoded_rows_have_the_prompts_alternatives():
    """One token of three users a call, against all tokens at once."""
    import torch
    rng = np.random.default_rng(7)
    B, T, d, vocab, top = 3, 150, 96, 4001, 10
    X = torch.from_numpy(rng.standard_normal((T, B, d)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    W = rounded(rng.standard_normal((vocab, d)) * 2 * d ** -0.5, am.BF16)
    tokens = rng.integers(0, vocab, T * B)
    whole, one = Teacher(am.BF16, T * B, d, W, tokens, top), Teacher(am.BF16, B, d, W, tokens[:B], top)
    whole.forward(X.view(T * B, d))
    for t in range(T):
        one.tokens.copy_(whole.tokens[t * B:(t + 1) * B])
        one.forward(X[t])
        rows = slice(t * B, (t + 1) * B)
        assert torch.equal(one.ids, whole.ids[rows])
        for a, b in ((one.logs, whole.logs), (one.logprob, whole.logprob), (one.entropy, whole.entropy)):
            assert float((a - b[rows]).abs().max()) <= F32_TOL * float(b.abs().max())


def test_a_students_gradient_trains_the_memory():
    """The memory's answers -> norm -> distillation; its gradient goes back through update_backward."""
    import torch
    inp = synth.make_inputs(4, "literal", batch=1, heads=2, T=256)
    s = inp.spec
    M, T, dv, H, n = s.n_mem, s.T, s.d_value, s.heads, s.batch * s.T
    rng = np.random.default_rng(8)
    vocab, d, top = 500, s.heads * dv, 6
    gamma, beta = np.ones(d, dtype=np.float32), np.zeros(d, dtype=np.float32)
    Wt, Wv = ((rng.standard_normal((vocab, d)) * d ** -0.5).astype(np.float32) for _ in range(2))
    R = rng.standard_normal((n, d)).astype(np.float32)
    dloss = np.ones(n, dtype=np.float32)

    def run():
        return [to_dev(x) for x in (inp.K, inp.Q, inp.V, inp.theta, inp.eta, inp.alpha)]

    mem = am.Memory(config_for(s), to_dev(inp.W0), to_dev(inp.S0))
    Y = torch.empty((M, T, dv), device=DEV)
    mem.update_chunked(*run(), None, T, Y)
    mem.close()
    rows = Y.view(s.batch, H, T, dv).transpose(1, 2).reshape(n, d).contiguous()
    norm = Norm(am.F32, n, H, dv, gamma, beta)
    teacher = Teacher(am.F32, n, d, Wt, np.zeros(n, dtype=np.int64), top)
    student = Student(am.F32, n, d, Wv, top, 1.0, dloss)
    Z, dZ, dR = (torch.empty_like(rows) for _ in range(3))
    teacher.forward(to_dev(R))
    norm.forward(rows, Z)
    student.forward(Z, teacher.ids, teacher.logs)
    student.backward(Z, dZ)
    norm.backward(rows, dZ, dR)
    dY = dR.view(s.batch, T, H, dv).transpose(1, 2).reshape(M, T, dv).contiguous()
    mem = am.Memory(config_for(s), to_dev(inp.W0), to_dev(inp.S0))
    dK, dQ, dV = (torch.empty((M, T, w), device=DEV) for w in (s.d_key, s.d_key, dv))
    gates = [torch.empty(inp.theta.shape, device=DEV) for _ in range(3)]
    dW0, dS0 = torch.empty((2, M, mem.P), device=DEV)
    mem.update_backward(*run(), T, dY, dK, dQ, dV, *gates, dW0, dS0, workspace(mem.backward_workspace_bytes(T)))
    torch.cuda.synchronize()
    mem.close()

    cfg = oracle.config_from(s)
    f = [synth.bf16_bits_to_f32(x).astype(np.float64) for x in (inp.K, inp.Q, inp.V)]
    y = oracle.run_inputs(inp)[0]
    _, _, ids, logs = tl.forward(R.astype(np.float64), Wt.astype(np.float64), None, 1.0, top)
    assert np.array_equal(teacher.ids.cpu().numpy(), ids)
    r = y.reshape(s.batch, H, T, dv).swapaxes(1, 2).reshape(n, 1, d)
    z, _, _ = gn.forward(r, H, gamma.astype(np.float64), beta.astype(np.float64), EPS, True)
    dz, dW = ds.backward(z[:, 0], Wv.astype(np.float64), ids, logs, 1.0, dloss.astype(np.float64))
    dy, _, _ = gn.backward(r, dz[:, None], H, gamma.astype(np.float64), beta.astype(np.float64), EPS, True)
    dyh = dy.reshape(s.batch, T, H, dv).swapaxes(1, 2).reshape(M, T, dv)
    want = [bw.outer_grads(cfg, oracle.unflatten(cfg, inp.W0[m].astype(np.float64)),
                           oracle.unflatten(cfg, inp.S0[m].astype(np.float64)), f[0][m], f[1][m], f[2][m],
                           inp.theta[m], inp.eta[m], inp.alpha[m], dyh[m], None, None) for m in range(M)]
    check("student_memory", BF16_TOL, dW=(student.dW, dW), dY=(dY, dyh), dK=(dK, np.stack([w["K"] for w in want])),
          dQ=(dQ, np.stack([w["Q"] for w in want])), dV=(dV, np.stack([w["V"] for w in want])))
