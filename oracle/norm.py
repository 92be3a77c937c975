"""RMS norm and its gradients in float64."""

import numpy as np


def forward(h, gamma, eps):
    """(y, rstd) of y = h rstd gamma, rstd = 1 / sqrt(mean(h^2) + eps) per row."""
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * gamma, rstd


def backward(dy, h, gamma, rstd, dres=None):
    """(dh, dgamma)."""
    up = dy * gamma
    c = np.mean(up * h, axis=1) * rstd ** 2
    dh = (up - h * c[:, None]) * rstd[:, None]
    if dres is not None:
        dh = dh + dres
    return dh, np.sum(dy * h * rstd[:, None], axis=0)
