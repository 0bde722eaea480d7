"""Expected values of token log probabilities and of distillation with its gradients, and how far each may be off,
elementwise, from the arithmetic (u = 2^-24, A the sum of a product's absolute terms, z' = scale z):
  z      ez = (r + 4 planes) u A: r = 6 (d / 16 + 1) + 16 fp32 roundings on a term's way, an fp32 call's planes
         dropping three products of 2^-25 and two residues of 2^-26; 2 d + 16 where fp32 instructions sum
         values that planes do not hold (plain32)
  e      exp(scale (z - m)): (3 |z' - m| + 8) u for the difference, its product and the hardware exponential
  lse    el = scale max ez + (3 max |z' - m| + 136) u + u |lse|: 64 sums in a lane, and the joins
  entropy  a change of the logits by ez moves it by sum p |log p + H| ez; its sums as lse's
  token, alternatives  their logits in 64 bits, rounded; el
  p      a product, a difference, two exponentials and a logarithm: (4 |t'| + 4 |t' - m| + 24) u
  G      q (scale ez + el + (|z' - lse| + 200) 2 u), up to 2^60 between a row's factor and lse; p's own; one
         rounding of G, 2^-8 in bf16, 3 u in planes
  dX, dW products with it as z; weights 4 u; dW's rows of X rounded with their weights, 2^-8 in bf16, 4 u else
and one rounding of an output (2^-8 for bf16, u for fp32).
"""

import numpy as np

from helpers import log
from oracle import distillation as ds
from oracle import token_logprobs as tl

U = 2.0 ** -24


def _product(k, bf16, plain32=False):
    return max(6 * (k // 16 + 1) + 16 + (0 if bf16 else 4), 2 * k + 16 if plain32 else 0) * U


def _logits(X, W, on, scale, bf16, plain32):
    X = np.where(on[:, None], X, 0.0)
    with np.errstate(invalid="ignore"):
        z = scale * (X @ W.T)
        A = np.abs(X) @ np.abs(W).T
    live = z > -1e30  # masked classes have no part in the sums
    z = np.where(live, z, -np.inf)
    m = z.max(1, keepdims=True)
    far = np.where(live, m - np.where(live, z, 0.0), 0.0)
    ez = scale * _product(X.shape[1], bf16, plain32) * np.where(live, A, 0.0)
    p = np.exp(z - m)
    lse = m[:, 0] + np.log(p.sum(1))
    el = ez.max(1) + (3 * np.minimum(far, 104).max(1) + 136) * U + U * np.abs(lse)
    return X, z, far, ez, p / p.sum(1, keepdims=True), lse, el


def logprobs(X, W, tokens, scale, top, bf16, plain32=False):
    """{name: (value, bound)} of logprob, entropy and top_logprobs, and top_ids."""
    on = np.ones(len(X), dtype=bool) if tokens is None else (tokens >= 0) & (tokens < len(W))
    with np.errstate(invalid="ignore", divide="ignore"):
        lp, H, ids, logs = tl.forward(X, W, tokens, scale, top)
    X, z, far, ez, p, lse, el = _logits(X, W, on, scale, bf16, plain32)
    live = np.isfinite(z)
    dist = np.minimum(far, 104)
    spread = (p * np.abs(np.where(live, z, 0.0) - lse[:, None] + H[:, None])).sum(1)
    eh = 2 * spread * ez.max(1) + ((p * dist * (3 * dist + 136)).sum(1) + 136 + 8 * np.abs(H)
                                   + np.abs(lse - z.max(1)) * 4) * U
    out = {"entropy": (H, np.where(on, eh, 0.0))}
    if tokens is not None:
        zt = z[np.arange(len(z)), np.where(on, tokens, 0)]
        out["logprob"] = (lp, np.where(on, el + 2 * U * np.abs(zt) + U * np.abs(lp), 0.0))
    if top:
        there = np.isfinite(logs) & on[:, None]
        out["top_logprobs"] = (logs, np.where(there, el[:, None] + 2 * U * np.abs(np.where(there, logs, 0.0)), 0.0))
    return out, ids


def distillation(X, W, ids, t, scale, dloss, bf16, plain32=False):
    """{name: (value, bound)} of loss, lse, dX, dW."""
    p, logp, on = ds.targets(ids, t, len(W), scale)
    loss, lse_want = ds.forward(X, W, ids, t, scale)
    X, z, far, ez, q, lse, el = _logits(X, W, on, scale, bf16, plain32)
    at = np.where((ids >= 0) & (ids < len(W)), ids, 0)
    st = np.where(p > 0, scale * np.where(np.isfinite(t), t, 0.0), 0.0)
    ep = (4 * np.abs(st) + 4 * np.abs(logp) + 24) * U
    zt = np.take_along_axis(np.where(np.isfinite(z), z, 0.0), at, 1)
    terms = p * (ep * (1 + np.abs(logp - zt + lse[:, None])) + el[:, None] + 2 * U * np.abs(zt)) \
        + 8 * U * p * np.abs(logp - zt + lse[:, None])
    out = {"loss": (loss, np.where(on, terms.sum(1), 0.0)), "lse": (lse_want, np.where(on, el, 0.0))}
    if dloss is None:
        dloss = np.ones(len(X))
    w = scale * np.where(on, dloss, 0.0)[:, None]
    G = ds.gradient_of_logits(X, W, ids, t, scale)
    rnd, gr, xr = (2.0 ** -8, 2.0 ** -8, 2.0 ** -8) if bf16 else (U, 3 * U, 4 * U)
    live = np.isfinite(z)
    eG = q * (ez + el[:, None] + (np.abs(np.where(live, z, 0.0) - lse[:, None]) + 200) * 2 * U)
    np.add.at(eG, (np.arange(len(G))[:, None], at), p * (ep + 4 * U))
    eG = np.abs(w) * (eG + (gr + 4 * U) * np.abs(G))
    G = G * w
    V = len(W)
    fin = np.where(np.isfinite(W), W, 0.0)
    dX, dW = G @ fin, G.T @ X
    eX = eG @ np.abs(fin) + (_product(V, bf16, plain32) + V / 512 * U) * (np.abs(G) @ np.abs(fin)) + rnd * np.abs(dX)
    eW = eG.T @ np.abs(X) + (_product(len(X), bf16, plain32) + xr) * (np.abs(G).T @ np.abs(X)) + rnd * np.abs(dW)
    out["dX"], out["dW"] = (dX, eX), (dW, eW)
    return out


def within(name, got, want, bound):
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else got
    same = (got == want) & np.isinf(want)
    assert np.isfinite(got[~same]).all(), name
    off = np.abs(np.where(same, 0.0, got) - np.where(same, 0.0, want)) / (bound + 1e-30)
    ratio = float(off.max()) if got.size else 0.0
    log(f"PARITY {name}: {ratio:.3f} of the bound")
    assert ratio <= 1.0, (name, ratio)
