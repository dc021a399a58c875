"""Pins for the oracles of the gated recurrence, the causal convolution with states and the
residual norm: closed forms, and every gradient against central finite differences (float64, tiny
inputs)."""
import numpy as np
import pytest

from oracle import block
from oracle import causal_conv as cc
from oracle import gated_recurrence as gr
from oracle import residual_norm as rn

OFFSETS = (0, 4, 4, 5, 9)


def differences(f, a, eps=1e-6):
    d = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        old = a[i]
        a[i] = old + eps
        hi = f()
        a[i] = old - eps
        lo = f()
        a[i] = old
        d[i] = (hi - lo) / (2 * eps)
    return d


def near(got, want):
    np.testing.assert_allclose(got, want, rtol=1e-6, atol=1e-7)


def recurrence_case(seed=1, D=3):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    T, q = OFFSETS[-1], len(OFFSETS) - 1
    return dict(x=n((T, D)), i=n((T, D)), r=n((T, D)), A=-rng.uniform(0.05, 2.0, D), state=n((q, D)),
                dh=n((T, D)), dlast=n((q, D)))


@pytest.mark.parametrize("name", ["x", "i", "r", "A", "state"])
def test_recurrence_gradients_match_finite_differences(name):
    c = recurrence_case()

    def loss():
        h, last = gr.gated_recurrence(c["x"], c["i"], c["r"], c["A"], OFFSETS, state=c["state"])
        return float((h * c["dh"]).sum() + (last * c["dlast"]).sum())

    got = gr.gated_recurrence_backward(c["x"], c["i"], c["r"], c["A"], OFFSETS, c["dh"],
                                       state=c["state"], dlast=c["dlast"])
    near(got["d" + name], differences(loss, c[name]))


def test_recurrence_is_the_sum_over_earlier_tokens():
    c = recurrence_case(2)
    h, last = gr.gated_recurrence(c["x"], c["i"], c["r"], c["A"], (0, 9), state=c["state"][:1])
    s = lambda v: 1 / (1 + np.exp(-v))
    log_a = c["A"] * s(c["r"])
    b = np.sqrt(1 - np.exp(log_a) ** 2) * s(c["i"]) * c["x"]
    G = np.cumsum(log_a, axis=0)
    for t in range(9):
        want = np.exp(G[t]) * c["state"][0] + sum(np.exp(G[t] - G[j]) * b[j] for j in range(t + 1))
        np.testing.assert_allclose(h[t], want, rtol=1e-12)
    np.testing.assert_array_equal(last[0], h[-1])


def test_recurrence_keeps_sequences_apart_and_goes_on_from_states():
    c = recurrence_case(3)
    a = (c["i"], c["r"])
    h, last = gr.gated_recurrence(c["x"], *a, c["A"], OFFSETS, state=c["state"])
    np.testing.assert_array_equal(last[1], c["state"][1])              # without tokens
    for q, (b, e) in enumerate(zip(OFFSETS[:-1], OFFSETS[1:])):
        cut = [v[b:e] for v in (c["x"], *a)]
        mid = (e - b) // 2
        h1, s1 = gr.gated_recurrence(*(v[:mid] for v in cut), c["A"], (0, mid),
                                     state=c["state"][q:q + 1])
        h2, s2 = gr.gated_recurrence(*(v[mid:] for v in cut), c["A"], (0, e - b - mid), state=s1)
        np.testing.assert_array_equal(np.concatenate([h1, h2]), h[b:e])
        np.testing.assert_array_equal(s2[0], last[q])


def conv_case(seed=4, D=2, k=3):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    T, q = OFFSETS[-1], len(OFFSETS) - 1
    return dict(u=n((T, D)), weight=n((D, k)), bias=n(D), state=n((q, k - 1, D)), dy=n((T, D)),
                dlast=n((q, k - 1, D)))


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("name", ["u", "weight", "bias", "state"])
def test_conv_gradients_match_finite_differences(name, k, silu):
    c = conv_case(k=k)

    def loss():
        y, last = cc.causal_conv(c["u"], c["weight"], c["bias"], OFFSETS, silu=silu,
                                 state=c["state"])
        return float((y * c["dy"]).sum() + (last * c["dlast"]).sum())

    got = cc.causal_conv_backward(c["u"], c["weight"], c["bias"], OFFSETS, c["dy"], silu=silu,
                                  state=c["state"], dlast=c["dlast"])
    near(got["d" + name], differences(loss, c[name]))


@pytest.mark.parametrize("k", [1, 3, 6])
def test_conv_is_the_blocks_convolution(k):
    rng = np.random.default_rng(5)
    u, w = rng.standard_normal((2, 10, 3)), rng.standard_normal((3, k))
    got, last = cc.causal_conv(u.reshape(20, 3), w, None, (0, 10, 20), silu=False)
    np.testing.assert_allclose(got.reshape(2, 10, 3), block.causal_conv1d(u, w), rtol=1e-12,
                               atol=1e-14)
    want = np.stack([[np.convolve(u[b, :, d], w[d, ::-1])[:10] for d in range(3)]
                     for b in range(2)])
    np.testing.assert_allclose(got.reshape(2, 10, 3), want.transpose(0, 2, 1), rtol=1e-12,
                               atol=1e-14)
    np.testing.assert_array_equal(last, u[:, 10 - (k - 1):])


def test_conv_goes_on_from_states():
    c = conv_case(6, k=4)
    y, last = cc.causal_conv(c["u"], c["weight"], c["bias"], (0, 9), silu=True,
                             state=c["state"][:1])
    for mid in (0, 1, 2, 5):
        y1, s1 = cc.causal_conv(c["u"][:mid], c["weight"], c["bias"], (0, mid), silu=True,
                                state=c["state"][:1])
        y2, s2 = cc.causal_conv(c["u"][mid:], c["weight"], c["bias"], (0, 9 - mid), silu=True,
                                state=s1)
        np.testing.assert_array_equal(np.concatenate([y1, y2]), y)
        np.testing.assert_array_equal(s2, last)


def norm_case(seed=7, R=3, D=5, post=True, gate=True, scale=True):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    return dict(y=n((R, D)), residual=n((R, D)), weight=n(D), post_weight=n(D) if post else None,
                gate=n((R, D)) if gate else None, scale=n(D) if scale else None, dout=n((R, D)),
                dtotal=n((R, D)))


@pytest.mark.parametrize("form", ["silu", "linear"])
@pytest.mark.parametrize("parts", [(1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)], ids=str)
def test_norm_gradients_match_finite_differences(parts, form):
    post, gate, scale = map(bool, parts)
    c = norm_case(post=post, gate=gate, scale=scale)
    eps = 1e-3
    opts = lambda: dict(post_weight=c["post_weight"], gate=c["gate"], form=form, scale=c["scale"])

    def loss():
        t = rn.total(c["y"], c["residual"], eps=eps, **opts())
        out = t * rn.rms(t, eps)[:, None] * c["weight"]
        return float((out * c["dout"]).sum() + (t * c["dtotal"]).sum())

    t = rn.total(c["y"], c["residual"], eps=eps, **opts())
    got = rn.residual_norm_backward(c["dout"], c["dtotal"], c["y"], t, c["weight"], rn.rms(t, eps),
                                    post_rstd=rn.rms(c["y"], eps), **opts())
    names = ["y", "residual", "weight"] + ["post_weight"] * post + ["gate"] * gate + ["scale"] * scale
    for name in names:
        near(got["d" + name], differences(loss, c[name]))


def test_norm_moments():
    c = norm_case(8, R=4, D=50)
    t = rn.total(c["y"], c["residual"], eps=0.0, post_weight=np.ones(50))
    np.testing.assert_allclose(((t - c["residual"]) ** 2).mean(axis=1), 1.0, rtol=1e-12)
    np.testing.assert_allclose((t * rn.rms(t, 0.0)[:, None] ** 1).std(axis=1) ** 2 +
                               (t * rn.rms(t, 0.0)[:, None]).mean(axis=1) ** 2, 1.0, rtol=1e-12)
