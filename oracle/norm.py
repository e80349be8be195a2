"""Oracle: layer norm and root-mean-square norm, and their gradients.

Test infrastructure only (see ``oracle/__init__``).

Along each row x of n elements ("layer"; for "rms" the mean is 0):

    mean = sum(x) / n       var = sum((x - mean)^2) / n
    rstd = 1 / sqrt(var + eps)
    xhat = (x - mean) rstd  y = xhat w + b

and with g = dy w

    dx = rstd (g - sum(g) / n - xhat sum(g xhat) / n)   ("rms": without sum(g) / n)
    dw = column sums of dy xhat                          db = column sums of dy

float64 throughout.
"""

import numpy as np


def forward(x, w=None, b=None, eps=1e-5, kind="layer"):
    """y, mean, rstd"""
    mean = x.mean(axis=1) if kind == "layer" else np.zeros(x.shape[0])
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean, rstd


def backward(dy, x, mean, rstd, w=None, kind="layer"):
    """dx, dw, db for the statistics given."""
    xhat = (x - mean[:, None] if kind == "layer" else x) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = g - xhat * (g * xhat).mean(axis=1, keepdims=True)
    if kind == "layer":
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * rstd[:, None], (dy * xhat).sum(axis=0), dy.sum(axis=0)
