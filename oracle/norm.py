"""Layer normalisation and its gradients in binary64 (numpy).

y = h w + b with h = (x - mean) rstd, rstd = 1 / sqrt(var + eps), var the mean of squared
distances from the mean; dx = (v - mean(v) - h mean(v h)) rstd with v = dy w.
"""

import numpy as np


def layer_norm(x, w=None, b=None, eps=1e-5):
    """(y, h, mean, rstd) of rows of x; w and b default to ones and zeros."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1, keepdims=True)
    c = x - mean
    rstd = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    h = c * rstd
    y = h if w is None else h * np.asarray(w, np.float64)
    return (y if b is None else y + np.asarray(b, np.float64)), h, mean, rstd


def layer_norm_backward(x, w, dy, eps=1e-5):
    """(dx, dw, db) for the upstream dy."""
    _, h, _, rstd = layer_norm(x, eps=eps)
    dy = np.asarray(dy, np.float64)
    v = dy if w is None else dy * np.asarray(w, np.float64)
    dx = (v - v.mean(1, keepdims=True) - h * (v * h).mean(1, keepdims=True)) * rstd
    return dx, (dy * h).sum(0), dy.sum(0)
