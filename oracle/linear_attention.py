"""Linear attention with a decay for each head -- oracle, TEST INFRASTRUCTURE ONLY.

The recurrence and its adjoint, written out token by token in float64, one
sequence and head at a time:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T          o_t = scale S_t^T q_t
    D_t = scale q_t dout_t^T + exp(g_{t+1}) D_{t+1}     (after the last: dlast)
    dq_t = scale S_t dout_t    dk_t = D_t v_t    dv_t = D_t^T k_t
    dg_t = exp(g_t) <D_t, S_{t-1}>               dS_0 = exp(g_1) D_1

Pinned by the closed sum over earlier tokens and by central finite differences
(tests/test_oracle_linear_attention_pins.py).
"""
from __future__ import annotations

import numpy as np


def _sequences(L_or_offsets, tokens):
    if np.ndim(L_or_offsets) == 0:
        n = int(L_or_offsets)
        return [(a, a + n) for a in range(0, tokens, n)] if n else []
    off = [int(x) for x in L_or_offsets]
    return list(zip(off[:-1], off[1:]))


def _inputs(q, k, v, log_decay):
    f = lambda a: np.asarray(a, dtype=np.float64)
    q, k, v, g = f(q), f(k), f(v), f(log_decay)
    T, H = v.shape[0], v.shape[1]
    rep = H // q.shape[1]
    g = np.broadcast_to(g, (T, H))
    return q, k, v, g, rep


def linear_attention(q, k, v, log_decay, offsets, *, scale, state=None):
    """o [T, H, dv] and the last states [sequences, H, dk, dv] for q, k [T, Hk, dk],
    v [T, H, dv], log_decay [T, H] or [H]; ``offsets`` the sequences' bounds."""
    q, k, v, g, rep = _inputs(q, k, v, log_decay)
    T, H, dv = v.shape
    dk = q.shape[2]
    seqs = _sequences(offsets, T)
    o = np.zeros((T, H, dv))
    last = np.zeros((len(seqs), H, dk, dv))
    for n, (a, b) in enumerate(seqs):
        for h in range(H):
            s = np.zeros((dk, dv)) if state is None else np.array(state[n, h], dtype=np.float64)
            for t in range(a, b):
                s = np.exp(g[t, h]) * s + np.outer(k[t, h // rep], v[t, h])
                o[t, h] = scale * (q[t, h // rep] @ s)
            last[n, h] = s
    return o, last


def linear_attention_backward(q, k, v, log_decay, offsets, dout, *, scale, state=None,
                              dlast=None):
    """Gradients of sum(dout * o) + sum(dlast * last): dq, dk [T, Hk, dk] (summed over the
    heads of a key head), dv, dlog_decay (of log_decay's shape) and dstate."""
    per_head = np.ndim(log_decay) == 1
    q, k, v, g, rep = _inputs(q, k, v, log_decay)
    dout = np.asarray(dout, dtype=np.float64)
    T, H, dv_ = v.shape
    dk_ = q.shape[2]
    seqs = _sequences(offsets, T)
    out = {"dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape),
           "dlog_decay": np.zeros((T, H)), "dstate": np.zeros((len(seqs), H, dk_, dv_))}
    for n, (a, b) in enumerate(seqs):
        for h in range(H):
            hk = h // rep
            s = np.zeros((dk_, dv_)) if state is None else np.array(state[n, h], dtype=np.float64)
            before = []
            for t in range(a, b):
                before.append(s)
                s = np.exp(g[t, h]) * s + np.outer(k[t, hk], v[t, h])
                out["dq"][t, hk] += scale * (s @ dout[t, h])
            D = (np.zeros((dk_, dv_)) if dlast is None
                 else np.array(dlast[n, h], dtype=np.float64))
            for t in range(b - 1, a - 1, -1):
                D = D + scale * np.outer(q[t, hk], dout[t, h])
                out["dk"][t, hk] += D @ v[t, h]
                out["dv"][t, h] = k[t, hk] @ D
                D = np.exp(g[t, h]) * D
                out["dlog_decay"][t, h] = np.sum(D * before[t - a])
            out["dstate"][n, h] = D
    if per_head:
        out["dlog_decay"] = out["dlog_decay"].sum(axis=0)
    return out
