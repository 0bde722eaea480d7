"""Log probabilities of given tokens, entropies and top alternatives in fp64; rows whose token is no class are left
out; classes whose product x w is -1e38 or less, or 1e32 or more below the row's largest, are masked and no
alternatives."""

from __future__ import annotations

import numpy as np


def forward(X, W, tokens, scale, top):
    """(logprob, entropy, top_ids, top_logprobs); tokens None: every row counts, logprob None."""
    vocab = len(W)
    on = np.ones(len(X), dtype=bool) if tokens is None else (tokens >= 0) & (tokens < vocab)
    raw = np.where(on[:, None], X, 0.0) @ W.T
    z, m_raw = scale * raw, raw.max(1)
    m = z.max(1)
    e = np.exp(z - m[:, None])
    s = e.sum(1)
    lse = m + np.log(s)
    p = e / s[:, None]
    entropy = np.where(on, -(p * np.where(p > 0, z - lse[:, None], 0.0)).sum(1), 0.0)
    logprob = None
    if tokens is not None:
        logprob = np.where(on, z[np.arange(len(z)), np.where(on, tokens, 0)] - lse, 0.0)
    order = np.argsort(-raw, axis=1, kind="stable")[:, :top]
    best = np.take_along_axis(raw, order, 1)
    there = on[:, None] & (best > -1e38) & (best > m_raw[:, None] - 1e32)
    logs = np.where(there, scale * best - lse[:, None], -np.inf)
    return logprob, entropy, np.where(there, order, -1), np.where(on[:, None], logs, 0.0)
