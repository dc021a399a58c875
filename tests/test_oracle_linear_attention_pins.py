"""Pins for the oracles of linear attention and layer norm: closed forms, and
every gradient against central finite differences (float64, tiny inputs)."""
import numpy as np
import pytest

from oracle import layer_norm as ln
from oracle import linear_attention as la


def _case(seed, offsets=(0, 4, 4, 9), Hk=1, H=2, dk=3, dv=2, per_head=False):
    rng = np.random.default_rng(seed)
    T, n = offsets[-1], len(offsets) - 1
    g = -rng.uniform(0.05, 1.0, (H,) if per_head else (T, H))
    return dict(q=rng.standard_normal((T, Hk, dk)), k=rng.standard_normal((T, Hk, dk)),
                v=rng.standard_normal((T, H, dv)), log_decay=g,
                state=rng.standard_normal((n, H, dk, dv))), dict(
        offsets=offsets, scale=0.7, dout=rng.standard_normal((T, H, dv)),
        dlast=rng.standard_normal((n, H, dk, dv)))


def _loss(c, p):
    o, s = la.linear_attention(c["q"], c["k"], c["v"], c["log_decay"], p["offsets"],
                               scale=p["scale"], state=c["state"])
    return float(np.sum(o * p["dout"]) + np.sum(s * p["dlast"]))


def _differences(f, a, eps=1e-6):
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


@pytest.mark.parametrize("per_head", [False, True], ids=["token", "head"])
@pytest.mark.parametrize("name", ["q", "k", "v", "log_decay", "state"])
def test_gradients_match_finite_differences(name, per_head):
    c, p = _case(11, per_head=per_head)
    got = la.linear_attention_backward(c["q"], c["k"], c["v"], c["log_decay"], p["offsets"],
                                       p["dout"], scale=p["scale"], state=c["state"],
                                       dlast=p["dlast"])["d" + name]
    np.testing.assert_allclose(got, _differences(lambda: _loss(c, p), c[name]), rtol=1e-6,
                               atol=1e-7)


def test_output_is_the_sum_over_earlier_tokens():
    c, p = _case(12, offsets=(0, 8))
    o, _ = la.linear_attention(c["q"], c["k"], c["v"], c["log_decay"], p["offsets"],
                               scale=p["scale"])
    G = np.cumsum(c["log_decay"], axis=0)
    for t in range(8):
        for h in range(2):
            want = sum(np.exp(G[t, h] - G[j, h]) * (c["q"][t, 0] @ c["k"][j, 0]) * c["v"][j, h]
                       for j in range(t + 1))
            np.testing.assert_allclose(o[t, h], p["scale"] * want, rtol=1e-12)


def test_sequences_do_not_meet_and_an_empty_one_keeps_its_state():
    c, p = _case(13)
    args = dict(scale=p["scale"], state=c["state"])
    _, s = la.linear_attention(c["q"], c["k"], c["v"], c["log_decay"], p["offsets"], **args)
    np.testing.assert_array_equal(s[1], c["state"][1])
    c["v"][:4] = 1e3
    _, s2 = la.linear_attention(c["q"], c["k"], c["v"], c["log_decay"], p["offsets"], **args)
    np.testing.assert_array_equal(s2[2], s[2])
    assert np.abs(s2[0] - s[0]).max() > 1


@pytest.mark.parametrize("name", ["x", "weight", "bias"])
def test_norm_gradients_match_finite_differences(name):
    rng = np.random.default_rng(5)
    c = dict(x=rng.standard_normal((3, 7)), weight=rng.standard_normal(7),
             bias=rng.standard_normal(7))
    dy = rng.standard_normal((3, 7))
    _, mean, rstd = ln.layer_norm(c["x"], c["weight"], c["bias"], eps=1e-3)
    got = dict(zip(("x", "weight", "bias"),
                   ln.layer_norm_backward(dy, c["x"], c["weight"], mean, rstd)))[name]
    loss = lambda: float(np.sum(dy * ln.layer_norm(c["x"], c["weight"], c["bias"], eps=1e-3)[0]))
    np.testing.assert_allclose(got, _differences(loss, c[name]), rtol=1e-6, atol=1e-7)


def test_norm_rows_have_the_moments_asked_for():
    x = np.random.default_rng(6).standard_normal((4, 50)) * 3 + 2
    y, mean, rstd = ln.layer_norm(x, np.ones(50), eps=0.0)
    np.testing.assert_allclose(y.mean(axis=1), 0, atol=1e-12)
    np.testing.assert_allclose((y ** 2).mean(axis=1), 1, rtol=1e-12)
    np.testing.assert_allclose(mean, x.mean(axis=1))
    np.testing.assert_allclose(rstd, 1 / x.std(axis=1))
