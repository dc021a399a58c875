"""Residual norm -- oracle, TEST INFRASTRUCTURE ONLY.

The norms around a block with its gate, residual scale and residual add, float64, rows [R, D]:

    t = residual + scale act(gate) rms(y) post_weight        out = rms(t) weight

The gradient is the chain rule step by step, from given statistics.  Pinned by the rows' moments and by
central finite differences (tests/test_oracle_recurrent_layer_pins.py).
"""
from __future__ import annotations

import numpy as np


def _f(v):
    return None if v is None else np.asarray(v, dtype=np.float64)


def _act(z, form):
    """Value and slope of the gate."""
    if z is None:
        return 1.0, 0.0
    if form == "linear":
        return z, np.ones_like(z)
    s = 1 / (1 + np.exp(-z))
    return z * s, s + z * s * (1 - s)


def rms(v, eps):
    """1 / sqrt(mean(v^2) + eps) of each row."""
    v = _f(v)
    return 1 / np.sqrt((v ** 2).mean(axis=1) + eps)


def total(y, residual, *, post_weight=None, gate=None, form="silu", scale=None, eps):
    """t [R, D]; gate already has a row for each of y's."""
    y, pw = _f(y), _f(post_weight)
    v = y if pw is None else y * rms(y, eps)[:, None] * pw
    return _f(residual) + v * _act(_f(gate), form)[0] * (1.0 if scale is None else _f(scale))


def residual_norm_backward(dout, dtotal, y, t, weight, rstd, *, post_weight=None, post_rstd=None,
                           gate=None, form="silu", scale=None):
    """dict of dy, dresidual, dgate (a row for each of y's), dweight, dpost_weight, dscale."""
    dout, y, t, w = _f(dout), _f(y), _f(t), _f(weight)
    pw, sc = _f(post_weight), 1.0 if scale is None else _f(scale)
    that = t * _f(rstd)[:, None]
    dthat = dout * w
    d = _f(rstd)[:, None] * (dthat - that * (dthat * that).mean(axis=1, keepdims=True))
    if dtotal is not None:
        d = d + _f(dtotal)
    value, slope = _act(_f(gate), form)
    yhat = y if pw is None else y * _f(post_rstd)[:, None]
    v = yhat if pw is None else yhat * pw
    dv = d * value * sc
    out = {"dresidual": d, "dweight": (dout * that).sum(axis=0),
           "dgate": d * v * slope * sc, "dscale": (d * v * value).sum(axis=0)}
    if pw is None:
        out["dy"] = dv
        return out
    dyhat = dv * pw
    out["dpost_weight"] = (dv * yhat).sum(axis=0)
    out["dy"] = _f(post_rstd)[:, None] * (dyhat - yhat * (dyhat * yhat).mean(axis=1, keepdims=True))
    return out
