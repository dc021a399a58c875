"""Gated linear recurrence -- oracle, TEST INFRASTRUCTURE ONLY.

The recurrence and its adjoint, written out token by token in float64, over packed tokens
[T, D] whose sequences have the bounds ``offsets``:

    s = sigmoid(r), a = exp(A s), m = sqrt(1 - a^2), g = sigmoid(i)
    h_t = a_t h_{t-1} + m_t g_t x_t
    lam_t = dh_t + a_{t+1} lam_{t+1}        (after the last token: dlast)
    dx = lam m g                  di = lam m x g (1 - g)
    e  = lam (a h_{t-1} - g x a^2 / m)      (the gradient of log a)
    dr = e A s (1 - s)            dA = sum e s            dstate = a_1 lam_1

Pinned by the closed sum over earlier tokens and by central finite differences
(tests/test_oracle_recurrent_layer_pins.py).
"""
from __future__ import annotations

import numpy as np


def _f(v):
    return np.asarray(v, dtype=np.float64)


def _sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def _gates(i, r, A):
    s, g = _sigmoid(_f(r)), _sigmoid(_f(i))
    log_a = _f(A) * s
    return s, g, np.exp(log_a), np.sqrt(-np.expm1(2.0 * log_a))


def gated_recurrence(x, i, r, A, offsets, *, state=None):
    """h [T, D] (zero outside the sequences) and the last states [sequences, D]."""
    x = _f(x)
    _, g, a, m = _gates(i, r, A)
    n = len(offsets) - 1
    h = np.zeros_like(x)
    last = np.zeros((n, x.shape[1])) if state is None else _f(state).copy()
    for q in range(n):
        for t in range(offsets[q], offsets[q + 1]):
            last[q] = a[t] * last[q] + m[t] * g[t] * x[t]
            h[t] = last[q]
    return h, last


def gated_recurrence_backward(x, i, r, A, offsets, dh, *, state=None, dlast=None):
    """dict of dx, di, dr [T, D], dA [D] and dstate [sequences, D]."""
    x, dh, A = _f(x), _f(dh), _f(A)
    s, g, a, m = _gates(i, r, A)
    h, _ = gated_recurrence(x, i, r, A, offsets, state=state)
    n = len(offsets) - 1
    out = {k: np.zeros_like(x) for k in ("dx", "di", "dr")}
    out["dA"] = np.zeros(x.shape[1])
    out["dstate"] = np.zeros((n, x.shape[1])) if dlast is None else _f(dlast).copy()
    for q in range(n):
        psi = out["dstate"][q]
        for t in reversed(range(offsets[q], offsets[q + 1])):
            if t > offsets[q]:
                before = h[t - 1]
            else:
                before = np.zeros(x.shape[1]) if state is None else _f(state)[q]
            lam = dh[t] + psi
            out["dx"][t] = lam * m[t] * g[t]
            out["di"][t] = lam * m[t] * x[t] * g[t] * (1 - g[t])
            with np.errstate(divide="ignore", invalid="ignore"):
                slope = np.where(m[t] > 0, a[t] ** 2 / m[t], 0.0)
            e = lam * (a[t] * before - g[t] * x[t] * slope)
            out["dr"][t] = e * A * s[t] * (1 - s[t])
            out["dA"] += e * s[t]
            psi = a[t] * lam
        out["dstate"][q] = psi
    return out
