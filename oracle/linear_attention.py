"""Linear attention with a decay for each head, token by token in fp64, and its gradients.

W_t = lambda W_{t-1} + v_t k_t^T, y_t = scale W_t q_t, lambda = exp(log_decay[h]); arrays
[B, H, T, d], states [B, H, d_value, d_key].  Tokens at and behind lengths[b] do not exist.
"""

from __future__ import annotations

import numpy as np


def _lam(log_decay):
    return np.exp(np.asarray(log_decay, dtype=np.float64))[None, :, None, None]


def _live(lengths, t, B):
    n = np.full(B, np.iinfo(np.int64).max) if lengths is None else np.asarray(lengths)
    return (t < n)[:, None, None, None]


def forward(q, k, v, log_decay, scale, W0, lengths=None):
    """(y, W_T)"""
    B, H, T, _ = q.shape
    lam, W = _lam(log_decay), W0.astype(np.float64)
    y = np.zeros(v.shape)
    for t in range(T):
        on = _live(lengths, t, B)
        W = np.where(on, lam * W + v[:, :, t, :, None] * np.where(on, k[:, :, t, None, :], 0.0), W)
        y[:, :, t] = np.where(on[..., 0], scale * (W @ np.where(on, q[:, :, t, :, None], 0.0))[..., 0], 0.0)
    return y, W


def backward(q, k, v, log_decay, scale, W0, dy, dW_T, lengths=None):
    """(dq, dk, dv, dW0, dlog_decay)"""
    B, H, T, _ = q.shape
    lam = _lam(log_decay)
    states = [W0.astype(np.float64)]
    for t in range(T):
        on = _live(lengths, t, B)
        states.append(np.where(on, lam * states[-1] + v[:, :, t, :, None] * k[:, :, t, None, :], states[-1]))
    A = dW_T.astype(np.float64)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dlog = np.zeros(H)
    for t in reversed(range(T)):
        on = _live(lengths, t, B)
        dyt = scale * dy[:, :, t, :, None]
        At = A + dyt * q[:, :, t, None, :]
        dq[:, :, t] = np.where(on[..., 0], (np.swapaxes(states[t + 1], -1, -2) @ dyt)[..., 0], 0.0)
        dk[:, :, t] = np.where(on[..., 0], (np.swapaxes(At, -1, -2) @ v[:, :, t, :, None])[..., 0], 0.0)
        dv[:, :, t] = np.where(on[..., 0], (At @ k[:, :, t, :, None])[..., 0], 0.0)
        dlog += np.where(on, At * lam * states[t], 0.0).sum((0, 2, 3))
        A = np.where(on, lam * At, A)
    return dq, dk, dv, A, dlog
