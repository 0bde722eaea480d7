"""Group norm with an activation, channels last, in fp64: X [n, L, C], statistics of a group over its
positions and channels."""

from __future__ import annotations

import numpy as np


def _sigmoid(z):
    return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


def _grouped(x, groups):
    n, L, C = x.shape
    return x.reshape(n, L, groups, C // groups)


def statistics(x, groups, eps):
    """mean, rstd [n, groups]"""
    g = _grouped(x, groups)
    mean = g.mean((1, 3))
    var = ((g - mean[:, None, :, None]) ** 2).mean((1, 3))
    return mean, 1.0 / np.sqrt(var + eps)


def normalised(x, groups, mean, rstd):
    return ((_grouped(x, groups) - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(x.shape)


def forward(x, groups, gamma, beta, eps, silu):
    """(y, mean, rstd)"""
    mean, rstd = statistics(x, groups, eps)
    z = normalised(x, groups, mean, rstd) * gamma + beta
    return (z * _sigmoid(z) if silu else z), mean, rstd


def backward(x, dy, groups, gamma, beta, eps, silu):
    """(dx, dgamma, dbeta)"""
    mean, rstd = statistics(x, groups, eps)
    xh = normalised(x, groups, mean, rstd)
    z = xh * gamma + beta
    s = _sigmoid(z)
    dz = dy * (s * (1.0 + z * (1.0 - s))) if silu else dy
    h, g = _grouped(dz * gamma, groups), _grouped(xh, groups)
    dx = rstd[:, None, :, None] * (h - h.mean((1, 3), keepdims=True) - g * (h * g).mean((1, 3), keepdims=True))
    return dx.reshape(x.shape), (dz * xh).sum((0, 1)), dz.sum((0, 1))
