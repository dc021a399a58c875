"""The gated recurrence's gradients at gates far from zero, where a sigmoid's slope s (1 - s) is as small
as its complement 1 - s: against float64 with the complements formed as 1 / (1 + exp(gate)).

Bounds as in test_gated_recurrence_gpu.py, but with the slopes' true sizes: a slope's relative error is that of
its two factors.  With e = exp(-r) the complement is e s: e is off by |r| + 2 units of 2^-24 (the
exponential's argument is rounded), s by |r| + 4 and the product by one, 2 |r| + 7 in all; where s <= 1/2
the complement is 1 - s, off by s's share of |r| + 4 and half a unit.  Both are inside the bound's 2 units =
128 + 4 n + 4 (max |r| + max |i| + 4).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_support import host64  # noqa: E402
from recurrent_support import ULP, check, lay, offsets_kw  # noqa: E402
from selective_state_space_54_amd import mssm  # noqa: E402
from test_gated_recurrence_gpu import make, sizes_of  # noqa: E402


def gradients(x, i, r, A, dh, offsets):
    """dx, di, dr and the sizes of the terms of dr, in float64."""
    g, gc, s, sc = (1 / (1 + np.exp(v)) for v in (-i, i, -r, r))
    a, m = np.exp(A * s), np.sqrt(-np.expm1(2 * A * s))
    dx, di, dr = (np.zeros_like(x) for _ in range(3))
    for b, e in zip(offsets[:-1], offsets[1:]):
        before = np.zeros_like(x)
        for t in range(b + 1, e):
            before[t] = a[t - 1] * before[t - 1] + m[t - 1] * g[t - 1] * x[t - 1]
        psi = np.zeros(x.shape[1])
        for t in reversed(range(b, e)):
            lam = dh[t] + psi
            dx[t] = lam * m[t] * g[t]
            di[t] = dx[t] * x[t] * gc[t]
            dr[t] = lam * (a[t] * before[t] - g[t] * x[t] * a[t] ** 2 / m[t]) * A * s[t] * sc[t]
            psi = a[t] * lam
    return dx, di, dr


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("low,high", [(4.0, 9.0), (8.0, 16.0), (16.0, 40.0)])
@pytest.mark.parametrize("sign", [1, -1])
def test_slopes_far_from_zero(dtype, low, high, sign):
    c = make(int(low), [90, 40], 130, dtype, packed=True, rates=(0.01, 4.0))
    rng = np.random.default_rng(int(high))
    for n in ("i", "r"):
        c[n] = torch.from_numpy(sign * rng.uniform(low, high, c[n].shape)).to(c[n].dtype)
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    got = mssm.gated_recurrence_bwd(x, i, r, c["A"].cuda(), dh, **offsets_kw(c))
    X, I, R, A, dh = (host64(c[n]) for n in ("x", "i", "r", "A", "dh"))
    dx, di, dr = gradients(X, I, R, A, dh, c["offsets"])
    units, H, M = sizes_of(c, False, False)
    g, gc, s, sc = (1 / (1 + np.exp(v)) for v in (-I, I, -R, R))
    a, m = np.exp(A * s), np.sqrt(-np.expm1(2 * A * s))
    unit = (2 * units + 2 * np.abs(A * s) * (np.abs(R) + 4)) * ULP
    term = M * (a * H + g * np.abs(X) * a ** 2 / m)
    check("dx", got["dx"], dx, unit * M * m * g, dtype)
    check("dinput_gate", got["dinput_gate"], di, unit * M * m * g * gc * np.abs(X), dtype)
    check("ddecay_gate", got["ddecay_gate"], dr, unit * term * np.abs(A) * s * sc, dtype)
    assert (host64(got["dinput_gate"])[X != 0] != 0).mean() > 0.99


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gates_at_the_ends(dtype):
    """Gates of plus and minus 100 and infinity have no slope that a float32 number holds."""
    c = make(60, [130], 66, dtype)
    ends = torch.tensor([100.0, -100.0, float("inf"), float("-inf")])
    for n, shift in (("i", 0), ("r", 1)):
        c[n] = ends.roll(shift).repeat(130 * 66 // 4 + 1)[:130 * 66].view(130, 66).to(c[n].dtype)
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    got = mssm.gated_recurrence_bwd(x, i, r, c["A"].cuda(), dh)
    for n in ("dinput_gate", "ddecay_gate"):
        assert (got[n].float().abs() < 1e-37).all(), n
    assert torch.isfinite(got["dx"].float()).all() and torch.isfinite(got["dA"]).all()
