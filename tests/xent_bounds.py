"""Expected values of a cross entropy call and how far each may be off, elementwise, from the arithmetic
(u = 2^-24, A the sum of a product's absolute terms):
  z      (r + 4 planes) u A: r = 6 (d / 16 + 1) + 16 fp32 roundings on a term's way, an fp32 call's planes
         dropping three products of 2^-25 and two residues of 2^-26
  lse    el = max ez + (|z - m| + 16) 2 u + u |lse| for hardware exponentials and the joins
  G      the probability's part |P| (ez + el + (|z - lse| + 8) 2 u), and one rounding of G, 2^-8 in bf16, 3 u in
         planes; its weight, a quotient and two products, 3 u
and one rounding of an output (2^-8 for bf16, u for fp32).
An fp32 call's products with values that planes do not hold (infinities, floats beyond bf16's largest) are fp32
sums, with at most two roundings a term: r = 2 d + 16 there (plain32).
"""

import numpy as np

from helpers import log
from oracle import cross_entropy as ce

U = 2.0 ** -24


def expected(X, W, labels, dloss, bf16, plain32=False):
    """{name: (value, bound)} of loss, lse, dX, dW for fp64 copies of the inputs."""
    n, d, vocab = len(X), X.shape[1], len(W)
    out, gr = (2.0 ** -8, 2.0 ** -8) if bf16 else (U, 3 * U)

    def e_of(k):
        return max(6 * (k // 16 + 1) + 16 + (0 if bf16 else 4), 2 * k + 16 if plain32 else 0) * U

    w = np.ones(n) if dloss is None else np.asarray(dloss, dtype=np.float64)
    on = (labels >= 0) & (labels < vocab)
    X = np.where(on[:, None], X, 0.0)
    loss, lse = ce.forward(X, W, labels)
    aX, aW = np.abs(X), np.abs(W)
    A, z = aX @ aW.T, X @ W.T
    ez = e_of(d)
    el = ez * A.max(1) + (np.abs(z - z.max(1, keepdims=True)).max(1) + 16) * 2 * U + U * np.abs(lse)
    G = ce.gradient_of_logits(X, W, labels, w)
    P = G.copy()
    P[np.arange(n)[on], labels[on]] += w[on]
    eG = np.abs(P) * (ez * A + el[:, None] + (np.abs(z - lse[:, None]) + 8) * 2 * U) + (gr + 3 * U) * np.abs(G)
    dX, dW = G @ W, G.T @ X
    eX = eG @ aW + (e_of(vocab) + vocab / 512 * U) * (np.abs(G) @ aW) + out * np.abs(dX)
    eW = eG.T @ aX + e_of(n) * (np.abs(G).T @ aX) + out * np.abs(dW)
    return {"loss": (loss, np.where(on, el + ez * A.max(1) + U * np.abs(loss), 0.0)), "lse": (lse, np.where(on, el, 0.0)),
            "dX": (dX, eX), "dW": (dW, eW)}


def within(name, got, want, bound):
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else got
    assert np.isfinite(got).all(), name
    ratio = float(np.max(np.abs(got - want) / (bound + 1e-30))) if got.size else 0.0
    log(f"PARITY {name}: {ratio:.3f} of the bound")
    assert ratio <= 1.0, (name, ratio)
