"""The operators around the memory run together as a user trains and decodes with them: linear
attention (or the memory itself) -> group norm of every head -> cross entropy, and back.

Bars: the library's own parity bars for fp32 and bf16 paths (1e-4 and 2e-2 of the tensor's largest
value), against the same chain in fp64.
"""

import numpy as np
import pytest

import oracle
from helpers import BF16_TOL, DEV, F32_TOL, config_for, log, maxrel, to_dev
from oracle import backward as bw
from oracle import cross_entropy as ce
from oracle import group_norm as gn
from oracle import linear_attention as la
from test_learned_neural_amd import atlasmem as am
from test_learned_neural_amd import synth

pytestmark = pytest.mark.gpu

EPS = 1e-5


def torch_dtype(dtype):
    import torch
    return torch.bfloat16 if dtype == am.BF16 else torch.float32


def workspace(n):
    import torch
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=DEV)


class Norm:
    """Group norm of the heads of `rows` rows of H * d channels, and its backward."""

    def __init__(self, dtype, rows, H, d, gamma, beta):
        import torch
        self.size = (dtype, rows, 1, H * d, H)
        self.gamma, self.beta = to_dev(gamma), to_dev(beta)
        self.mean, self.rstd = torch.empty((2, rows, H), device=DEV)
        self.ws = workspace(max(am.group_norm_workspace_bytes(rows, 1, H * d, H, b) for b in (False, True)))
        self.dgamma, self.dbeta = torch.empty((2, H * d), device=DEV)

    def forward(self, X, Y):
        am.group_norm(X, *self.size, self.gamma, self.beta, EPS, am.ACT_SILU, Y, self.mean, self.rstd, self.ws)

    def backward(self, X, dY, dX):
        am.group_norm_backward(X, dY, *self.size, self.gamma, self.beta, self.mean, self.rstd, am.ACT_SILU, dX,
                               self.dgamma, self.dbeta, self.ws)


class Loss:
    def __init__(self, dtype, n, d, W, labels, dloss):
        import torch
        self.size = (dtype, n, d, len(W))
        self.W = torch.from_numpy(W).to(torch_dtype(dtype)).to(DEV)
        self.labels, self.dloss = to_dev(labels), to_dev(dloss)
        self.loss, self.lse = torch.empty((2, n), device=DEV)
        self.dW = torch.empty_like(self.W)
        self.ws = workspace(max(am.cross_entropy_workspace_bytes(*self.size, b) for b in (False, True)))

    def forward(self, X):
        am.cross_entropy(X, self.W, *self.size, self.labels, self.loss, self.lse, self.ws)

    def backward(self, X, dX):
        am.cross_entropy_backward(X, self.W, *self.size, self.labels, self.lse, self.dloss, dX, self.dW, self.ws)


def check(name, tol, **pairs):
    errs = {k: maxrel(g.double().cpu().numpy(), r) for k, (g, r) in pairs.items()}
    log(f"PARITY {name}: " + " ".join(f"{k}={v:.2e}" for k, v in errs.items()) + f" (tol {tol:g})")
    assert all(v <= tol for v in errs.values()), errs


@pytest.mark.parametrize("dtype,captured", [(am.F32, False), (am.BF16, False), (am.F32, True)])
def test_mixer_norm_loss_and_back(dtype, captured):
    import torch
    rng = np.random.default_rng(3)
    B, T, H, dk, dv, vocab = 2, 300, 4, 32, 48, 1001
    n, d, lengths = B * T, H * dv, [300, 211]
    dt = torch_dtype(dtype)
    host = {k: torch.from_numpy(rng.standard_normal((B, T, H, w)).astype(np.float32)).to(dt)
            for k, w in (("q", dk), ("k", dk), ("v", dv))}
    q, k, v = (host[x].to(DEV) for x in "qkv")
    g = np.log1p(-2.0 ** -np.linspace(2, 8, H)).astype(np.float32)
    gamma = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    beta = (0.2 * rng.standard_normal(d)).astype(np.float32)
    Wv = torch.from_numpy((rng.standard_normal((vocab, d)) * 2 * d ** -0.5).astype(np.float32)).to(dt).float().numpy()
    labels = rng.integers(0, vocab, n)
    behind = (np.arange(T)[None, :] >= np.array(lengths)[:, None]).reshape(-1)
    labels[behind] = -100                                     # the padding's rows
    labels[rng.random(n) < 0.2] = -100                        # and a prompt's
    dloss = np.full(n, 1.0 / (labels >= 0).sum(), dtype=np.float32)
    scale = dk ** -0.5

    size = (dtype, B, H, T, dk, dv)
    gd, ld = to_dev(g), torch.tensor(lengths, dtype=torch.int32, device=DEV)
    wa = workspace(am.linear_attention_workspace_bytes(*size, True))
    norm, loss = Norm(dtype, n, H, dv, gamma, beta), Loss(dtype, n, d, Wv, labels, dloss)
    Y, Z, dZ, dY = (torch.empty((n, d), dtype=dt, device=DEV) for _ in range(4))
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty(H, device=DEV)

    def step():
        am.linear_attention(q, k, v, *size, gd, scale, Y, lengths=ld, layout=am.TOKENS_FIRST, workspace=wa)
        norm.forward(Y, Z)
        loss.forward(Z)
        loss.backward(Z, dZ)
        norm.backward(Y, dZ, dY)
        am.linear_attention_backward(q, k, v, *size, gd, scale, dY, dq, dk_, dv_, dlog_decay=dg, lengths=ld,
                                     layout=am.TOKENS_FIRST, workspace=wa)

    outs = (loss.loss, Z, loss.dW, norm.dgamma, norm.dbeta, dq, dk_, dv_, dg)
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for _ in range(3):
            for o in outs:
                o.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, outs))
    else:
        step()
        torch.cuda.synchronize()

    f = {x: host[x].double().numpy().swapaxes(1, 2) for x in "qkv"}
    W0 = np.zeros((B, H, dv, dk))
    y, _ = la.forward(f["q"], f["k"], f["v"], g, scale, W0, lengths)
    rows = y.swapaxes(1, 2).reshape(n, 1, d)
    ga, be = gamma.astype(np.float64), beta.astype(np.float64)
    z, _, _ = gn.forward(rows, H, ga, be, EPS, True)
    wl, _ = ce.forward(z[:, 0], Wv.astype(np.float64), labels)
    dz, dW = ce.backward(z[:, 0], Wv.astype(np.float64), labels, dloss)
    dy, dga, dbe = gn.backward(rows, dz[:, None], H, ga, be, EPS, True)
    dyh = dy.reshape(B, T, H, dv).swapaxes(1, 2)
    want = la.backward(f["q"], f["k"], f["v"], g, scale, W0, dyh, W0, lengths)
    heads = lambda x: x.swapaxes(1, 2)
    check(f"chain_{dtype}", BF16_TOL if dtype == am.BF16 else F32_TOL, loss=(loss.loss, wl), Z=(Z, z[:, 0]),
          dW=(loss.dW, dW), dgamma=(norm.dgamma, dga), dbeta=(norm.dbeta, dbe), dq=(dq, heads(want[0])),
          dk=(dk_, heads(want[1])), dv=(dv_, heads(want[2])), dlog_decay=(dg, want[4]))


def test_decoding_equals_the_prompt():
    """One token a call through the mixer and the norm, the state in place, against one call over all."""
    import torch
    rng = np.random.default_rng(4)
    B, T, H, d = 3, 40, 2, 64
    q, k, v = (to_dev(rng.standard_normal((B, T, H, d)).astype(np.float32)) for _ in range(3))
    g = to_dev(np.array([-0.2, -0.01], dtype=np.float32))
    gamma, beta = np.ones(H * d, dtype=np.float32), np.zeros(H * d, dtype=np.float32)
    Y, W_T = torch.empty_like(q), torch.empty((B, H, d, d), device=DEV)
    am.linear_attention(q, k, v, am.F32, B, H, T, d, d, g, 0.125, Y, W_T=W_T, layout=am.TOKENS_FIRST,
                        workspace=workspace(am.linear_attention_workspace_bytes(am.F32, B, H, T, d, d)))
    whole = Norm(am.F32, B * T, H, d, gamma, beta)
    Z = torch.empty_like(Y)
    whole.forward(Y, Z)
    W, step = torch.zeros_like(W_T), Norm(am.F32, B, H, d, gamma, beta)
    for t in range(T):
        y, z = torch.empty((2, B, 1, H, d), device=DEV)
        a = [x[:, t:t + 1].contiguous() for x in (q, k, v)]
        am.linear_attention(*a, am.F32, B, H, 1, d, d, g, 0.125, y, W0=W, W_T=W, layout=am.TOKENS_FIRST)
        step.forward(y, z)
        assert float((z[:, 0] - Z[:, t]).abs().max()) <= F32_TOL * float(Z.abs().max())
    assert float((W - W_T).abs().max()) <= F32_TOL * float(W_T.abs().max())


def test_the_losss_gradient_trains_the_memory():
    """The memory's answers -> norm -> loss; the loss's gradient goes back through update_backward."""
    import torch
    inp = synth.make_inputs(4, "literal", batch=1, heads=2, T=256)
    s = inp.spec
    M, T, dv = s.n_mem, s.T, s.d_value
    H, n = s.heads, s.batch * s.T
    rng = np.random.default_rng(5)
    vocab, d = 500, s.heads * dv
    gamma, beta = np.ones(d, dtype=np.float32), np.zeros(d, dtype=np.float32)
    Wv = (rng.standard_normal((vocab, d)) * d ** -0.5).astype(np.float32)
    labels = rng.integers(0, vocab, n)
    dloss = np.ones(n, dtype=np.float32)

    def run():
        return [to_dev(x) for x in (inp.K, inp.Q, inp.V, inp.theta, inp.eta, inp.alpha)]

    mem = am.Memory(config_for(s), to_dev(inp.W0), to_dev(inp.S0))
    Y = torch.empty((M, T, dv), device=DEV)
    mem.update_chunked(*run(), None, T, Y)
    mem.close()
    rows = Y.view(s.batch, H, T, dv).transpose(1, 2).reshape(n, d).contiguous()
    norm, loss = Norm(am.F32, n, H, dv, gamma, beta), Loss(am.F32, n, d, Wv, labels, dloss)
    Z, dZ, dR = (torch.empty_like(rows) for _ in range(3))
    norm.forward(rows, Z)
    loss.forward(Z)
    loss.backward(Z, dZ)
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
    r = y.reshape(s.batch, H, T, dv).swapaxes(1, 2).reshape(n, 1, d)
    z, _, _ = gn.forward(r, H, gamma.astype(np.float64), beta.astype(np.float64), EPS, True)
    dz, dW = ce.backward(z[:, 0], Wv.astype(np.float64), labels, dloss.astype(np.float64))
    dy, _, _ = gn.backward(r, dz[:, None], H, gamma.astype(np.float64), beta.astype(np.float64), EPS, True)
    dyh = dy.reshape(s.batch, T, H, dv).swapaxes(1, 2).reshape(M, T, dv)
    want = [bw.outer_grads(cfg, oracle.unflatten(cfg, inp.W0[m].astype(np.float64)),
                           oracle.unflatten(cfg, inp.S0[m].astype(np.float64)), f[0][m], f[1][m], f[2][m],
                           inp.theta[m], inp.eta[m], inp.alpha[m], dyh[m], None, None) for m in range(M)]
    check("memory_chain", BF16_TOL, dW=(loss.dW, dW), dY=(dY, dyh), dK=(dK, np.stack([w["K"] for w in want])),
          dQ=(dQ, np.stack([w["Q"] for w in want])), dV=(dV, np.stack([w["V"] for w in want])))
