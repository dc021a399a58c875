"""The gated linear recurrence on the GPU (prompts, single tokens, gradient) against the float64
oracle on the same inputs.

Bounds.  Per channel, with the inputs' absolute values for x, dh and the states the recurrence and
its adjoint give sizes H_t >= |h_t| and M_t >= |lambda_t|.  In units of 2^-24: a sigmoid is off by
|gate| + 4 of its value (exp2's argument is rounded), a_t by 1 for its rounding and by
|A s| (|r| + 4) for what s is off.  What reaches a token from an earlier one has been multiplied
by exp(-sum |A s|) <= 1 / (e sum |A s|), so those add up to less than half of max |r| + 4; the
roundings of a and of each sum decay like the state, 2 n for a memory of n = 1 / (1 - a) tokens; the
input term's factors are two sigmoids, m (6 and half of s) and three products: (|i| + 4) + 10 +
(|r| + 4) / 2.  Together h_t is off by less than (64 + 2 n + 2 (max |r| + max |i| + 4)) 2^-24 max H,
and the adjoint alike with M.  The gradients are products of those with factors of the same
kind: twice that, and |A s| (|r| + 4) more for their own a (twice, as a^2); dA's bound is the sum of its
terms' (partial sums of at most 128 terms: 128 units more).
bfloat16 results are rounded once more: 2^-8 of the value.
A s below 2^-126, the smallest normal float32, may count as zero: m = sqrt(1 - exp(2 A s)) is then off
by at most sqrt(2 2^-126), and A s / m by half of that.  So may a below 2^-126, a factor of e.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_support import host64  # noqa: E402
from oracle import gated_recurrence as gr  # noqa: E402
from recurrent_support import (DT, ULP, check, fused, lay, offsets_kw, offsets_of,  # noqa: E402
                               shifted, tensor)
from selective_state_space_54_amd import mssm  # noqa: E402
from test_graph_gpu import capture, replay_and_check  # noqa: E402


def make(seed, lengths, D, dtype, packed=False, rates=(0.001, 0.5), gates=1.0):
    rng = np.random.default_rng(seed)
    T, n = int(np.sum(lengths)), len(lengths)
    c = {"lengths": lengths, "offsets": offsets_of(lengths), "packed": packed, "D": D}
    for name in ("x", "i", "r", "dh"):
        c[name] = tensor(rng, (T, D), dtype, gates if name in ("i", "r") else 1.0)
    lo, hi = np.log(rates[0]), np.log(rates[1])
    c["A"] = torch.from_numpy(-np.exp(rng.uniform(lo, hi, D))).float()
    c["state"] = torch.from_numpy(rng.standard_normal((n, D))).float()
    c["dlast"] = torch.from_numpy(rng.standard_normal((n, D))).float()
    return c


def sizes_of(c, with_state, with_dlast):
    """Per channel: the bound's units of 2^-24, and the largest H and M."""
    i, r, A = (host64(c[k]) for k in ("i", "r", "A"))
    x, dh = np.abs(host64(c["x"])), np.abs(host64(c["dh"]))
    state = np.abs(host64(c["state"])) if with_state else None
    dlast = np.abs(host64(c["dlast"])) if with_dlast else None
    T = len(x)
    a = np.exp(A / (1 + np.exp(-r)))
    longest = max(list(c["lengths"]) + [1])
    n = np.minimum(longest, 1 / (1 - a.max(axis=0))) if T else np.ones(c["D"])
    h, last = gr.gated_recurrence(x, i, r, A, c["offsets"], state=state)
    H = np.maximum(np.abs(h).max(axis=0, initial=0.0), np.abs(last).max(axis=0, initial=0.0))
    if with_state:
        H = np.maximum(H, state.max(axis=0))
    M = np.zeros(c["D"])
    for q, (b, e) in enumerate(zip(c["offsets"][:-1], c["offsets"][1:])):
        psi = dlast[q] if with_dlast else np.zeros(c["D"])
        M = np.maximum(M, psi)
        for t in reversed(range(b, e)):
            lam = dh[t] + psi
            M = np.maximum(M, lam)
            psi = a[t] * lam
    gates = [np.where(np.isfinite(v), np.abs(v), 0.0).max(axis=0, initial=0.0) for v in (i, r)]
    units = 64 + 2 * n + 2 * (gates[0] + gates[1] + 4)
    return units, H, M


def check_forward(c, dtype, *, with_state, inputs=None):
    x, i, r = inputs or lay(c, "x", "i", "r")
    A = c["A"].cuda()
    kw = dict(state=c["state"].cuda() if with_state else None, **offsets_kw(c))
    h, last = mssm.gated_recurrence(x, i, r, A, return_state=True, **kw)
    only = mssm.gated_recurrence(x, i, r, A, **kw)
    again, saved = mssm.gated_recurrence(x, i, r, A, return_saved=True, **kw)
    torch.cuda.synchronize()
    assert torch.equal(h, only) and torch.equal(h, again)
    assert h.dtype == DT[dtype] and h.shape == x.shape and last.dtype == torch.float32
    state = host64(c["state"]) if with_state else None
    want, want_last = gr.gated_recurrence(*(host64(c[k]) for k in ("x", "i", "r", "A")),
                                          c["offsets"], state=state)
    units, H, _ = sizes_of(c, with_state, False)
    bound = units * ULP * H
    check("h", h, want, bound, dtype)
    check("last state", last, want_last, bound, "fp32")


def check_backward(c, dtype, *, with_state, with_dlast):
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    A = c["A"].cuda()
    kw = dict(state=c["state"].cuda() if with_state else None, **offsets_kw(c))
    dlast = c["dlast"].cuda() if with_dlast else None
    got = mssm.gated_recurrence_bwd(x, i, r, A, dh, dstate=dlast, **kw)
    saved = mssm.gated_recurrence(x, i, r, A, return_saved=True, **kw)[1]
    from_saved = mssm.gated_recurrence_bwd(x, i, r, A, dh, dstate=dlast, saved=saved, **kw)
    torch.cuda.synchronize()
    for k in got:
        assert torch.equal(got[k], from_saved[k]), k
    assert set(got) == {"dx", "dinput_gate", "ddecay_gate", "dA"} | ({"dstate"} if with_state else set())
    X, I, R, A64, dh64 = (host64(c[k]) for k in ("x", "i", "r", "A", "dh"))
    state = host64(c["state"]) if with_state else None
    want = gr.gated_recurrence_backward(X, I, R, A64, c["offsets"], dh64, state=state,
                                        dlast=host64(c["dlast"]) if with_dlast else None)
    units, H, M = sizes_of(c, with_state, with_dlast)
    s, g = 1 / (1 + np.exp(-R)), 1 / (1 + np.exp(-I))
    unit = (2 * units + 2 * np.abs(A64 * s) * (np.abs(R) + 4)) * ULP
    a = np.exp(A64 * s)
    m = np.sqrt(-np.expm1(2 * A64 * s))
    term = M * (a * H + g * np.abs(X) * a ** 2 / np.where(m > 0, m, np.inf))
    lost = M * g * np.where(np.abs(A64 * s) < 2.0 ** -126, 2.0 ** -62.5, 0.0)
    check("dx", got["dx"], want["dx"], unit * M * m * g + lost, dtype)
    check("dinput_gate", got["dinput_gate"], want["di"], (unit * M * m * g + lost) * np.abs(X), dtype)
    check("ddecay_gate", got["ddecay_gate"], want["dr"],
          unit * term * np.abs(A64) * s + lost * np.abs(X) +
          M * (H + g * np.abs(X)) * 2.0 ** -126 * np.abs(A64) * s, dtype)
    check("dA", got["dA"], want["dA"], ((unit + 128 * ULP) * term * s).sum(axis=0), "fp32")
    if with_state:
        check("dstate", got["dstate"], want["dstate"], 2 * units * ULP * M, "fp32")


# around a wavefront's tokens (16; float32: 8), a tile's (128; 64) and several tiles
LENGTHS = [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 700]
WIDTHS = [1, 2, 3, 63, 64, 65, 66, 127, 128, 129, 200, 333]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L", LENGTHS)
def test_lengths(dtype, L):
    check_forward(make(L, [L, L], 70, dtype), dtype, with_state=L % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(dtype, D):
    check_forward(make(D, [150, 150], D, dtype), dtype, with_state=True)


PACKED = [[0, 1, 16, 0, 235, 1, 0], [1, 1, 1], [0, 0], [500, 3, 129], [5], [16, 16, 128, 128, 64],
          [1] * 40 + [0] * 30 + [2] * 20 + [0] * 70 + [3]]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths", PACKED, ids=lambda v: str(v)[:40])
@pytest.mark.parametrize("D", [40, 129])
def test_packed(dtype, lengths, D):
    c = make(9, lengths, D, dtype, packed=True)
    check_forward(c, dtype, with_state=True)
    check_forward(c, dtype, with_state=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L", LENGTHS)
def test_gradient_lengths(dtype, L):
    check_backward(make(20 + L, [L, L], 70, dtype), dtype, with_state=L % 2 == 1,
                   with_dlast=L % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", WIDTHS)
def test_gradient_widths(dtype, D):
    check_backward(make(30 + D, [150, 150], D, dtype), dtype, with_state=True, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths", PACKED, ids=lambda v: str(v)[:40])
def test_packed_gradient(dtype, lengths):
    c = make(29, lengths, 129, dtype, packed=True)
    check_backward(c, dtype, with_state=True, with_dlast=True)
    check_backward(c, dtype, with_state=True, with_dlast=False)
    check_backward(c, dtype, with_state=False, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths,packed", [([5000], False), ([3000, 0, 2500, 1], True)], ids=str)
def test_many_tiles(dtype, lengths, packed):
    """States that remember thousands of tokens, over many tiles."""
    c = make(31, lengths, 66, dtype, packed=packed, rates=(1e-4, 1e-2))
    check_forward(c, dtype, with_state=True)
    check_backward(c, dtype, with_state=True, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rates_and_gates_at_the_ends(dtype):
    """No decay at all, decays around the switch to the series, to zero at once; closed and
    wide open gates."""
    c = make(32, [100, 200], 130, dtype, packed=True, rates=(1e-6, 30.0))
    c["A"][:4] = torch.tensor([0.0, -0.25, -0.5, -500.0])
    c["r"][::17] = 60.0
    c["r"][5::17] = -60.0
    c["r"][6] = float("inf")
    c["r"][7] = float("-inf")
    c["i"][::13] = -100.0
    c["i"][1::13] = 100.0
    c["A"][0] = -1e-30                              # (zero itself: the next test)
    check_forward(c, dtype, with_state=True)
    c["r"] = c["r"].clamp(-60, 60)
    check_backward(c, dtype, with_state=True, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("packed", [False, True])
def test_tiles_that_forget_what_was_before(dtype, packed):
    """Several tiles, beside channels of long memory some whose decays over a tile come to zero."""
    c = make(31, [700, 700], 130, dtype, packed, rates=(1e-4, 200.0))
    check_forward(c, dtype, with_state=True)
    check_backward(c, dtype, with_state=True, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_rate_of_zero_keeps_the_state(dtype):
    c = make(33, [70], 66, dtype)
    c["A"][:] = 0.0
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    A, state, dlast = c["A"].cuda(), c["state"].cuda(), c["dlast"].cuda()
    h, last = mssm.gated_recurrence(x, i, r, A, state=state, return_state=True)
    g = mssm.gated_recurrence_bwd(x, i, r, A, dh, state=state, dstate=dlast)
    torch.cuda.synchronize()
    assert torch.equal(last, state)
    assert torch.equal(h, state[:, None].to(DT[dtype]).expand_as(h))
    for n in ("dx", "dinput_gate", "ddecay_gate"):
        assert not g[n].float().any(), n
    assert torch.isfinite(g["dA"]).all()
    want = host64(dh)[0].sum(axis=0) + host64(dlast)[0]
    np.testing.assert_allclose(host64(g["dstate"])[0], want, rtol=1e-5,
                               atol=71 * ULP * float(np.abs(host64(dh)).sum(axis=1).max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [1, 40, 129, 200])
def test_step(dtype, D):
    c = make(40, [1] * 5, D, dtype)
    x, i, r = (c[k].cuda() for k in ("x", "i", "r"))
    state = c["state"].cuda()
    h = mssm.gated_recurrence_step(x, i, r, c["A"].cuda(), state)
    torch.cuda.synchronize()
    want, last = gr.gated_recurrence(*(host64(c[k]) for k in ("x", "i", "r", "A")), c["offsets"],
                                     state=host64(c["state"]))
    units, H, _ = sizes_of(c, True, False)
    check("h", h, want, units * ULP * H, dtype)
    check("state", state, last, units * ULP * H, "fp32")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_steps_go_on_from_a_prompt(dtype):
    c = make(41, [160, 160], 129, dtype)
    x, i, r = lay(c, "x", "i", "r")
    A = c["A"].cuda()
    h, state = mssm.gated_recurrence(*(t[:, :140].contiguous() for t in (x, i, r)), A,
                                     return_state=True)
    outs = [h]
    for t in range(140, 160):
        outs.append(mssm.gated_recurrence_step(x[:, t], i[:, t], r[:, t], A, state)[:, None])
    torch.cuda.synchronize()
    want, last = gr.gated_recurrence(*(host64(c[k]) for k in ("x", "i", "r", "A")), c["offsets"])
    units, H, _ = sizes_of(c, False, False)
    check("h", torch.cat(outs, 1), want, units * ULP * H, dtype)
    check("state", state, last, units * ULP * H, "fp32")


def everything(c, x, i, r, dh, state, dlast, **kw):
    A = c["A"].cuda()
    h, last, saved = mssm.gated_recurrence(x, i, r, A, state=state, return_state=True,
                                           return_saved=True, **kw)
    g = mssm.gated_recurrence_bwd(x, i, r, A, dh, state=state, dstate=dlast, saved=saved, **kw)
    g2 = mssm.gated_recurrence_bwd(x, i, r, A, dh, state=state, dstate=dlast, **kw)
    return [h, last] + [g[k] for k in sorted(g)] + [g2[k] for k in sorted(g2)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [66, 129])
def test_views_and_unaligned_tensors(dtype, D):
    """Slices of a fused projection, and pointers past a 16-byte boundary: the same numbers."""
    c = make(43, [260, 260], D, dtype)
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    state, dlast = c["state"].cuda(), c["dlast"].cuda()
    dense = everything(c, x, i, r, dh, state, dlast)
    views = everything(c, *fused(x, i, r), dh, state, dlast)
    moved = everything(c, *(shifted(t) for t in (x, i, r, dh, state, dlast)))
    for a, b, d in zip(dense, views, moved):
        assert torch.equal(a, b) and torch.equal(a, d)
    for t in range(3):
        s1, s2 = state.clone(), state.clone()
        v = [u[:, t] for u in fused(x, i, r)]
        assert torch.equal(mssm.gated_recurrence_step(*v, c["A"].cuda(), s1),
                           mssm.gated_recurrence_step(*(u.contiguous() for u in v), c["A"].cuda(), s2))
        assert torch.equal(s1, s2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeats_are_the_same_bit_for_bit(dtype):
    c = make(44, [1500, 0, 700, 800], 300, dtype, packed=True)
    args = lay(c, "x", "i", "r", "dh") + [c["state"].cuda(), c["dlast"].cuda()]
    kw = offsets_kw(c)
    first = everything(c, *args, **kw)
    for _ in range(5):
        for a, b in zip(first, everything(c, *args, **kw)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_values_that_are_not_finite_stay_in_their_sequence_and_channel(dtype):
    lengths = [150, 40, 1, 200, 5]
    c = make(45, lengths, 130, dtype, packed=True)
    kw = offsets_kw(c)
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    state, dlast = c["state"].cuda(), c["dlast"].cuda()
    clean = everything(c, x, i, r, dh, state, dlast, **kw)
    bad = [t.clone() for t in (x, i, r, dh, state, dlast)]
    bad[0][3, 5] = float("nan")          # sequence 0, channel 5
    bad[1][170, 6] = float("nan")        # sequence 1, channel 6
    bad[2][200, 7] = float("nan")        # sequence 3, channel 7
    bad[3][393, 8] = float("inf")        # sequence 4, channel 8
    bad[4][0, 9] = float("inf")
    bad[5][3, 10] = float("nan")
    hit = {(0, 5), (1, 6), (3, 7), (4, 8), (0, 9), (3, 10)}
    off = c["offsets"]
    keep = torch.ones(off[-1], 130, dtype=torch.bool, device="cuda")
    keep_seq = torch.ones(5, 130, dtype=torch.bool, device="cuda")
    for q, ch in hit:
        keep[off[q]:off[q + 1], ch] = False
        keep_seq[q, ch] = False
    for a, b in zip(clean, everything(c, *bad, **kw)):
        if a.dim() == 1:
            rest = torch.ones(130, dtype=torch.bool, device="cuda")
            rest[[5, 6, 7, 8, 9, 10]] = False
        else:
            rest = keep if a.shape[0] == off[-1] else keep_seq
        assert torch.equal(a[rest], b[rest])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tokens_outside_the_sequences_are_left_alone(dtype):
    """Rows before the first and behind the last sequence hold NaN; their outputs stay as they
    were, and nothing else changes."""
    lengths, front, back = [70, 0, 200], 21, 300
    c = make(46, lengths, 130, dtype, packed=True)
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    state, dlast, A = c["state"].cuda(), c["dlast"].cuda(), c["A"].cuda()
    want = everything(c, x, i, r, dh, state, dlast, **offsets_kw(c))
    nan = lambda n: torch.full((n, 130), float("nan"), dtype=x.dtype, device="cuda")
    px, pi, pr, pdh = (torch.cat([nan(front), t, nan(back)]) for t in (x, i, r, dh))
    off = torch.from_numpy(c["offsets"] + front).cuda()
    T = len(px)
    sizes = (3, T, 130, DT[dtype])
    ws = lambda **k: torch.empty(mssm.mssm_gated_recurrence_workspace_size(*sizes, packed=True, **k),
                                 dtype=torch.uint8, device="cuda")
    h = torch.full_like(px, 7.0)
    last = torch.empty(3, 130, device="cuda")
    mssm.mssm_gated_recurrence_fwd(px, pi, pr, A, h, ws(), state=state, last_state=last,
                                   seq_offsets=off)
    grads = {k: torch.full_like(px, 7.0) for k in ("dx", "dinput_gate", "ddecay_gate")}
    grads |= {"dA": torch.empty(130, device="cuda"), "dstate": torch.empty(3, 130, device="cuda")}
    mssm.mssm_gated_recurrence_bwd(px, pi, pr, A, pdh, grads, ws(backward=True), state=state,
                                   dstate=dlast, seq_offsets=off)
    torch.cuda.synchronize()
    for t in [h] + [grads[k] for k in ("dx", "dinput_gate", "ddecay_gate")]:
        assert (t[:front] == 7.0).all() and (t[T - back:] == 7.0).all()
    inner = lambda t: t[front:T - back]
    got = [inner(h), last] + [grads[k] if grads[k].shape[0] != T else inner(grads[k])
                              for k in sorted(grads)]
    # the tiles lie otherwise: the same values to the bounds, the same order of terms apart
    units, _, _ = sizes_of(c, True, True)
    for a, b in zip(got, want):
        assert torch.isfinite(a.float()).all()
        a, b = host64(a), host64(b)
        tol = 2 * (2.0 ** -8 if dtype == "bf16" and a.shape[0] == len(x) else 0.0) * np.abs(b)
        scale = np.abs(b).max(axis=0) + np.sqrt((b ** 2).mean())
        assert (np.abs(a - b) <= tol + 16 * units * ULP * scale).all()


def test_offsets_that_do_not_fit_are_kept_inside():
    """Offsets below 0 and past the tokens count as 0 and the tokens."""
    c = make(47, [50, 60], 70, "fp32", packed=True)
    x, i, r = lay(c, "x", "i", "r")
    A = c["A"].cuda()
    good = mssm.gated_recurrence(x, i, r, A, seq_offsets=torch.tensor([0, 50, 110]).cuda())
    wild = mssm.gated_recurrence(x, i, r, A, seq_offsets=torch.tensor([-5, 50, 1 << 40]).cuda())
    torch.cuda.synchronize()
    assert torch.equal(good, wild)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_a_graph(dtype):
    c = make(48, [300, 5, 900], 130, dtype, packed=True)
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    A, state, dlast = c["A"].cuda(), c["state"].cuda(), c["dlast"].cuda()
    off = offsets_kw(c)
    sizes = (3, 1205, 130, DT[dtype])
    empty = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
    ws = [empty(mssm.mssm_gated_recurrence_workspace_size(*sizes, packed=True, backward=b, saved=True))
          for b in (False, True)]
    saved = empty(mssm.mssm_gated_recurrence_saved_size(*sizes, packed=True))
    h, last = torch.empty_like(x), torch.empty_like(state)
    grads = {k: torch.empty_like(x) for k in ("dx", "dinput_gate", "ddecay_gate")}
    grads |= {"dA": torch.empty_like(A), "dstate": torch.empty_like(state)}

    def run():
        mssm.mssm_gated_recurrence_fwd(x, i, r, A, h, ws[0], state=state, last_state=last,
                                       saved=saved, **off)
        mssm.mssm_gated_recurrence_bwd(x, i, r, A, dh, grads, ws[1], saved=saved, state=state,
                                       dstate=dlast, **off)

    run()
    torch.cuda.synchronize()
    outputs = [h, last] + list(grads.values())
    expected = [t.clone() for t in outputs]
    replay_and_check(capture(run), outputs, expected,
                     lambda: mssm.gated_recurrence(x, i, r, A, **off))


def test_on_another_stream():
    """Workspace and outputs belong to the stream that the call runs on."""
    c = make(49, [2000], 200, "bf16")
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    A = c["A"].cuda()
    want = mssm.gated_recurrence(x, i, r, A)
    wg = mssm.gated_recurrence_bwd(x, i, r, A, dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        h = mssm.gated_recurrence(x, i, r, A, stream=s)
        g = mssm.gated_recurrence_bwd(x, i, r, A, dh, stream=s)
        s.synchronize()
        assert torch.equal(h, want)
        for k in g:
            assert torch.equal(g[k], wg[k])


def test_refusals():
    c = make(50, [20, 20], 40, "bf16")
    x, i, r, dh = lay(c, "x", "i", "r", "dh")
    A, state = c["A"].cuda(), c["state"].cuda()
    f = mssm.gated_recurrence
    with pytest.raises(ValueError, match="GPU"):
        f(c["x"], i, r, A)
    with pytest.raises(ValueError, match="batch, L, D"):
        f(x[0], i, r, A)
    with pytest.raises(TypeError, match="input_gate has dtype"):
        f(x, i.float(), r, A)
    with pytest.raises(TypeError, match="decay_gate must be a torch.Tensor"):
        f(x, i, None, A)
    with pytest.raises(ValueError, match="decay_gate has shape"):
        f(x, i, r[:, :5], A)
    with pytest.raises(TypeError, match="A has dtype"):
        f(x, i, r, A.bfloat16())
    with pytest.raises(ValueError, match="A has shape"):
        f(x, i, r, A[:5])
    with pytest.raises(ValueError, match="x must hold its channels densely"):
        f(x.transpose(1, 2).contiguous().transpose(1, 2), i, r, A)
    with pytest.raises(ValueError, match="state has shape"):
        f(x, i, r, A, state=state[:1])
    with pytest.raises(TypeError, match="seq_offsets has dtype"):
        f(x[0], i[0], r[0], A, seq_offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError, match="dtype"):
        f(x.half(), i.half(), r.half(), A)
    with pytest.raises(mssm.MssmError, match="INVALID_VALUE"):          # the state itself
        mssm.mssm_gated_recurrence_fwd(x, i, r, A, torch.empty_like(x), None, state=state,
                                       last_state=state)
    big = [t.repeat(1, 20, 1) for t in (x, i, r, dh)]
    with pytest.raises(mssm.MssmError, match="WORKSPACE"):
        mssm.mssm_gated_recurrence_fwd(*big[:3], A, torch.empty_like(big[0]), None)
    with pytest.raises(mssm.MssmError, match="WORKSPACE"):
        mssm.gated_recurrence_bwd(*big[:3], A, big[3], saved=torch.empty(8, dtype=torch.uint8,
                                                                         device="cuda"))
    with pytest.raises(ValueError, match="unknown gradient"):
        mssm.mssm_gated_recurrence_bwd(x, i, r, A, dh, {"dz": x}, None)
    with pytest.raises(ValueError, match="must be"):
        mssm.gated_recurrence_step(x, i, r, A, state)


def test_nothing_to_do():
    for shape in ((0, 5, 40), (2, 0, 40), (2, 5, 0)):
        x = torch.zeros(shape, device="cuda")
        A = -torch.ones(shape[2], device="cuda")
        state = torch.ones(shape[0], shape[2], device="cuda")
        h, last = mssm.gated_recurrence(x, x, x, A, state=state, return_state=True)
        g = mssm.gated_recurrence_bwd(x, x, x, A, x, state=state, dstate=2 * state)
        torch.cuda.synchronize()
        assert h.shape == shape and g["dx"].shape == shape
        assert torch.equal(last, state) and torch.equal(g["dstate"], 2 * state)
        assert not g["dA"].any()
