"""Layer norm and its gradients -- oracle, TEST INFRASTRUCTURE ONLY.

    y = (x - mean) rstd w + b,   rstd = (var + eps)^(-1/2), biased variance
    dx = rstd (w dy - mean(w dy) - xhat mean(w dy xhat)),  dw = sum dy xhat,
    db = sum dy,   xhat = (x - mean) rstd

in float64.  Pinned by finite differences and by the row's own moments
(tests/test_oracle_linear_attention_pins.py).
"""
from __future__ import annotations

import numpy as np


def layer_norm(x, weight, bias=None, *, eps):
    """y, mean, rstd of float64 rows."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=-1)
    rstd = (((x - mean[..., None]) ** 2).mean(axis=-1) + eps) ** -0.5
    y = (x - mean[..., None]) * rstd[..., None] * weight
    return (y if bias is None else y + bias), mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd):
    """dx, dweight, dbias for [rows, D] inputs and given statistics."""
    f = lambda a: np.asarray(a, dtype=np.float64)
    dy, x, weight, mean, rstd = map(f, (dy, x, weight, mean, rstd))
    xhat = (x - mean[:, None]) * rstd[:, None]
    wdy = dy * weight
    dx = rstd[:, None] * (wdy - wdy.mean(axis=1, keepdims=True) -
                          xhat * (wdy * xhat).mean(axis=1, keepdims=True))
    return dx, (dy * xhat).sum(axis=0), dy.sum(axis=0)
