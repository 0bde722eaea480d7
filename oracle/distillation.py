"""Distillation from a teacher's top logits and its gradients in fp64; rows without an entry are left out."""

from __future__ import annotations

import numpy as np


def targets(ids, teacher, vocab, scale):
    """(p, log p, which rows count): entries that are no class, or minus infinity, have p 0 and log p 0."""
    given = (ids >= 0) & (ids < vocab) & (teacher != -np.inf)
    on = given.any(1)
    t = np.where(given, scale * np.where(given, teacher, 0.0), -np.inf)
    m = np.where(on, np.where(given, t, -np.inf).max(1), 0.0)[:, None]
    e = np.where(given, np.exp(t - m), 0.0)
    s = np.where(on, e.sum(1), 1.0)[:, None]
    return e / s, np.where(given, np.where(given, t, 0.0) - m - np.log(s), 0.0), on


def forward(X, W, ids, teacher, scale):
    """(loss, lse)"""
    p, logp, on = targets(ids, teacher, len(W), scale)
    z = scale * (np.where(on[:, None], X, 0.0) @ W.T)
    m = z.max(1)
    lse = m + np.log(np.exp(z - m[:, None]).sum(1))
    at = np.where((ids >= 0) & (ids < len(W)), ids, 0)
    logq = np.take_along_axis(z, at, 1) - lse[:, None]
    loss = np.where(p > 0, p * (logp - np.where(p > 0, logq, 0.0)), 0.0).sum(1)
    return np.where(on, loss, 0.0), np.where(on, lse, 0.0)


def gradient_of_logits(X, W, ids, teacher, scale):
    """dL/d(scale z) of each row's loss: q less the teacher's p."""
    p, _, on = targets(ids, teacher, len(W), scale)
    z = scale * (np.where(on[:, None], X, 0.0) @ W.T)
    G = np.exp(z - z.max(1, keepdims=True))
    G /= G.sum(1, keepdims=True)
    at = np.where((ids >= 0) & (ids < len(W)), ids, 0)
    np.add.at(G, (np.arange(len(G))[:, None], at), -p)
    return np.where(on[:, None], G, 0.0)


def backward(X, W, ids, teacher, scale, dloss):
    """(dX, dW)"""
    _, _, on = targets(ids, teacher, len(W), scale)
    G = gradient_of_logits(X, W, ids, teacher, scale) * (scale * np.where(on, dloss, 0.0))[:, None]
    return G @ W, G.T @ np.where(on[:, None], X, 0.0)
