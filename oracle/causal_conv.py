"""Causal depthwise convolution with sequence states -- oracle, TEST INFRASTRUCTURE ONLY.

Sequence by sequence in float64, over packed tokens [T, D] with the bounds ``offsets``; the
k - 1 places before a sequence are its state's rows (zero without one):

    c_t = bias + sum_i w_i u_{t - (k - 1) + i}      y_t = c_t sigmoid(c_t), or c_t

Pinned by the block oracle's convolution (numpy's ``convolve``), and by central finite differences
(tests/test_oracle_recurrent_layer_pins.py).
"""
from __future__ import annotations

import numpy as np


def _f(v):
    return np.asarray(v, dtype=np.float64)


def _places(u, offsets, state, q, k):
    before = np.zeros((k - 1, u.shape[1])) if state is None else _f(state)[q]
    return np.concatenate([before, u[offsets[q]:offsets[q + 1]]])


def causal_conv(u, weight, bias, offsets, *, silu, state=None):
    """y [T, D] (zero outside the sequences) and the last states [sequences, k - 1, D]."""
    u, w = _f(u), _f(weight)
    k, n = w.shape[1], len(offsets) - 1
    y = np.zeros_like(u)
    last = np.zeros((n, k - 1, u.shape[1]))
    for q in range(n):
        places = _places(u, offsets, state, q, k)
        for t in range(offsets[q], offsets[q + 1]):
            at = t - offsets[q]
            c = (w.T * places[at:at + k]).sum(axis=0) + (0.0 if bias is None else _f(bias))
            y[t] = c / (1 + np.exp(-c)) if silu else c
        last[q] = places[len(places) - (k - 1):]
    return y, last


def causal_conv_backward(u, weight, bias, offsets, dy, *, silu, state=None, dlast=None):
    """dict of du [T, D], dweight [D, k], dbias [D] and dstate [sequences, k - 1, D]."""
    u, w, dy = _f(u), _f(weight), _f(dy)
    k, n, D = w.shape[1], len(offsets) - 1, u.shape[1]
    out = {"du": np.zeros_like(u), "dweight": np.zeros_like(w), "dbias": np.zeros(D),
           "dstate": np.zeros((n, k - 1, D))}
    for q in range(n):
        places = _places(u, offsets, state, q, k)
        grad = np.zeros_like(places)
        if dlast is not None:
            grad[len(places) - (k - 1):] += _f(dlast)[q]
        for t in range(offsets[q], offsets[q + 1]):
            at = t - offsets[q]
            dz = dy[t]
            if silu:
                c = (w.T * places[at:at + k]).sum(axis=0) + (0.0 if bias is None else _f(bias))
                s = 1 / (1 + np.exp(-c))
                dz = dz * (s + c * s * (1 - s))
            grad[at:at + k] += w.T * dz
            out["dweight"] += (places[at:at + k] * dz).T
            out["dbias"] += dz
        out["du"][offsets[q]:offsets[q + 1]] = grad[k - 1:]
        out["dstate"][q] = grad[:k - 1]
    return out
