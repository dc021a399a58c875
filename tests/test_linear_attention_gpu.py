"""Linear attention with a decay for each head on the GPU (prompt, single
tokens, gradient) against the float64 recurrence on the same inputs.

Tolerances, |err| <= a |ref| + b rms, rms the root mean square of the reference
over a head's tokens:
  bfloat16 results: 2^-8 |ref| + 2^-6 rms.  The output's rounding is at most 2^-8
    of it.  The rounded operands (decayed scores between runs of 16 tokens, state)
    err by at most 2^-8 each, independently, with a deviation of some 2^-9.5, so a
    sum of such products errs by about 2^-9.5 rms; five of those deviations for the
    largest of many, times sqrt(2) for two roundings, is 2^-6.7 rms.
  float32 results: 2e-5 (|ref| + rms): sums of up to a few hundred products at
    2^-24 each, in any order, stay under 300 * 2^-24 = 1.8e-5 of their sizes.
  states and their gradients (float32 from either type): the same 2e-5.
  dlog_decay: 1e-4 (|ref| + rms): it is put together from partial sums over 256
    tokens of either sign, each with the error above; for one decay a head the
    rms is over the heads.
"""
import numpy as np
import pytest

from gpu_support import host64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from oracle import linear_attention as la  # noqa: E402
from selective_state_space_54_amd import mssm  # noqa: E402
from test_graph_gpu import capture, replay_and_check  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _tensor(rng, shape, dtype, scale=1.0):
    return torch.from_numpy(scale * rng.standard_normal(shape)).to(DT[dtype])


def make(seed, lengths, Hk, H, dk, dv, dtype, per_head=False, packed=False, decay=(0.001, 1.0)):
    """CPU tensors of `dtype` and what the calls take; log decays spread over
    orders of magnitude, as those of heads of different memory are."""
    rng = np.random.default_rng(seed)
    T, n = sum(lengths), len(lengths)
    lead = (T,) if packed else (n, lengths[0] if n else 0)
    g = -np.exp(rng.uniform(*np.log(decay), (H,) if per_head else lead + (H,)))
    c = dict(q=_tensor(rng, lead + (Hk, dk), dtype), k=_tensor(rng, lead + (Hk, dk), dtype),
             v=_tensor(rng, lead + (H, dv), dtype), log_decay=torch.from_numpy(g).float(),
             state=_tensor(rng, (n, H, dk, dv), "fp32"),
             dout=_tensor(rng, lead + (H, dv), dtype),
             dlast=_tensor(rng, (n, H, dk, dv), "fp32"))
    c["offsets"] = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    c["packed"] = packed
    return c


def tokens(t, packed, trailing):
    a = host64(t)
    return a if packed else a.reshape((-1,) + a.shape[a.ndim - trailing:])


def oracle_inputs(c):
    p = c["packed"]
    g = c["log_decay"]
    return (tokens(c["q"], p, 2), tokens(c["k"], p, 2), tokens(c["v"], p, 2),
            host64(g) if g.dim() == 1 else tokens(g, p, 1), c["offsets"])


def on_gpu(c, *names):
    return [c[n].cuda() for n in names]


def offsets_kw(c):
    return {"seq_offsets": torch.from_numpy(c["offsets"]).cuda()} if c["packed"] else {}


def check(name, got, want, kind, heads_axis=-2):
    """kind: 'bf16', 'fp32' or 'decay'; want has the heads at heads_axis."""
    got = np.asarray(got, dtype=np.float64).reshape(want.shape)
    assert np.isfinite(got).all(), f"{name} is not finite"
    if not want.size:
        return
    axes = tuple(i for i in range(want.ndim) if i != heads_axis % want.ndim)
    rms = np.sqrt(np.mean(want ** 2, axis=axes if want.ndim > 1 else None, keepdims=True))
    a, b = {"bf16": (2.0 ** -8, 2.0 ** -6), "fp32": (2e-5, 2e-5), "decay": (1e-4, 1e-4)}[kind]
    ratio = float((np.abs(got - want) / (a * np.abs(want) + b * rms + 1e-30)).max())
    assert ratio <= 1.0, f"{name}: error {ratio:.3g} of the tolerance"


def check_forward(c, dtype, *, with_state, scale=None):
    q, k, v, g = on_gpu(c, "q", "k", "v", "log_decay")
    state = c["state"].cuda() if with_state else None
    dk = c["q"].shape[-1]
    kw = dict(scale=scale, state=state, **offsets_kw(c))
    o, last = mssm.linear_attention(q, k, v, g, return_state=True, **kw)
    o_only = mssm.linear_attention(q, k, v, g, **kw)
    torch.cuda.synchronize()
    want_o, want_s = la.linear_attention(*oracle_inputs(c),
                                         scale=dk ** -0.5 if scale is None else scale,
                                         state=host64(c["state"]) if with_state else None)
    assert o.dtype == DT[dtype] and o.shape == v.shape and last.dtype == torch.float32
    check("o", host64(o), want_o, dtype)
    check("o without the last state", host64(o_only), want_o, dtype)
    check("last state", host64(last), want_s, "fp32", 1)


def check_backward(c, dtype, *, with_state, with_dlast):
    q, k, v, g, dout = on_gpu(c, "q", "k", "v", "log_decay", "dout")
    state = c["state"].cuda() if with_state else None
    dlast = c["dlast"].cuda() if with_dlast else None
    got = mssm.linear_attention_bwd(q, k, v, g, dout, scale=0.3, state=state, dstate=dlast,
                                    **offsets_kw(c))
    torch.cuda.synchronize()
    want = la.linear_attention_backward(
        *oracle_inputs(c), tokens(c["dout"], c["packed"], 2), scale=0.3,
        state=host64(c["state"]) if with_state else None,
        dlast=host64(c["dlast"]) if with_dlast else None)
    assert set(got) == {"dq", "dk", "dv", "dlog_decay"} | ({"dstate"} if with_state else set())
    for n in ("dq", "dk", "dv"):
        assert got[n].dtype == DT[dtype]
        check(n, host64(got[n]), want[n], dtype)
    check("dlog_decay", host64(got["dlog_decay"]), want["dlog_decay"], "decay",
          -1 if g.dim() > 1 else 0)
    if with_state:
        check("dstate", host64(got["dstate"]), want["dstate"], "fp32", 1)


# lengths around one token, one chunk (64; float32: 32) and sequences cut into segments
LENGTHS = [1, 2, 31, 33, 63, 64, 65, 200, 700]
# key heads, heads, dk, dv: heads that share keys in pairs and not; tiles cut on either side
HEADS = [(1, 1, 16, 16), (2, 4, 64, 64), (1, 3, 48, 80), (3, 3, 112, 32), (1, 2, 16, 128),
         (2, 2, 128, 16), (1, 5, 128, 128), (2, 8, 80, 112)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L", LENGTHS)
def test_prompt_lengths(dtype, L):
    check_forward(make(L, [L, L], 2, 4, 64, 48, dtype), dtype, with_state=L % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_prompt_heads(dtype, heads):
    check_forward(make(7, [150], *heads, dtype, per_head=heads[0] == heads[1]), dtype,
                  with_state=True, scale=1.7)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", [(1, 1, 16, 16), (2, 4, 64, 64), (1, 3, 48, 80), (1, 1, 128, 128)],
                         ids=str)
@pytest.mark.parametrize("per_head", [False, True], ids=["token", "head"])
def test_long_prompts_are_cut_into_segments(dtype, heads, per_head):
    c = make(8, [1500], *heads, dtype, per_head=per_head, decay=(1e-4, 0.1))
    assert mssm.mssm_linear_attention_workspace_size(1, 1500, *heads, DT[dtype]) > 0
    check_forward(c, dtype, with_state=True)


PACKED = [[0, 1, 64, 0, 235, 1, 0], [1, 1, 1], [0, 0], [700, 3, 129], [5]]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths", PACKED, ids=str)
@pytest.mark.parametrize("heads", [(1, 2, 64, 64), (3, 3, 32, 96)], ids=str)
def test_packed_prompts(dtype, lengths, heads):
    c = make(9, lengths, *heads, dtype, packed=True)
    check_forward(c, dtype, with_state=True)
    check_forward(c, dtype, with_state=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("L", LENGTHS)
def test_gradient_lengths(dtype, L):
    check_backward(make(20 + L, [L, L], 2, 4, 48, 64, dtype), dtype, with_state=L % 2 == 1,
                   with_dlast=L % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_gradient_heads(dtype, heads):
    check_backward(make(27, [150], *heads, dtype, per_head=heads[0] == heads[1]), dtype,
                   with_state=True, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("per_head", [False, True], ids=["token", "head"])
def test_gradient_over_segments(dtype, per_head):
    check_backward(make(28, [1500], 1, 3, 48, 80, dtype, per_head=per_head, decay=(1e-4, 0.1)),
                   dtype, with_state=False, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lengths", PACKED, ids=str)
@pytest.mark.parametrize("per_head", [False, True], ids=["token", "head"])
def test_packed_gradient(dtype, lengths, per_head):
    check_backward(make(29, lengths, 1, 2, 64, 32, dtype, packed=True, per_head=per_head), dtype,
                   with_state=True, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_step(dtype, heads):
    Hk, H, dk, dv = heads
    c = make(40, [1, 1, 1], Hk, H, dk, dv, dtype, per_head=Hk == H)
    q, k, v, g = on_gpu(c, "q", "k", "v", "log_decay")
    state = c["state"].cuda()
    o = mssm.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g if g.dim() == 1 else g[:, 0], state)
    torch.cuda.synchronize()
    want_o, want_s = la.linear_attention(*oracle_inputs(c), scale=dk ** -0.5,
                                         state=host64(c["state"]))
    check("o", host64(o), want_o, dtype)
    check("state", host64(state), want_s, "fp32", 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_steps_go_on_from_a_prompt(dtype):
    """A prompt, then single tokens, give what the whole prompt gives."""
    c = make(41, [90, 90], 2, 4, 64, 64, dtype)
    q, k, v, g = on_gpu(c, "q", "k", "v", "log_decay")
    cut = lambda t, a, b: t[:, a:b].contiguous()
    o, state = mssm.linear_attention(*(cut(t, 0, 70) for t in (q, k, v, g)), return_state=True)
    outs = [o]
    for t in range(70, 90):
        outs.append(mssm.linear_attention_step(q[:, t], k[:, t], v[:, t], g[:, t].contiguous(),
                                               state)[:, None])
    torch.cuda.synchronize()
    want_o, want_s = la.linear_attention(*oracle_inputs(c), scale=64 ** -0.5)
    check("o", host64(torch.cat(outs, 1)), want_o, dtype)
    check("state", host64(state), want_s, "fp32", 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_last_state_may_be_the_state(dtype):
    """Also for empty sequences and for sequences without tokens at all."""
    for lengths, packed in (([300], False), ([0, 70, 0], True), ([0, 0], False), ([0], True)):
        c = make(42, lengths, 2, 2, 32, 64, dtype, packed=packed)
        q, k, v, g = on_gpu(c, "q", "k", "v", "log_decay")
        state = c["state"].cuda()
        o = torch.empty_like(v)
        n = mssm.mssm_linear_attention_workspace_size(
            len(lengths), sum(lengths) if packed else lengths[0], 2, 2, 32, 64, DT[dtype],
            packed=packed)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        mssm.mssm_linear_attention_fwd(q, k, v, g, o, ws, scale=0.5, state=state, last_state=state,
                                       **offsets_kw(c))
        torch.cuda.synchronize()
        want_o, want_s = la.linear_attention(*oracle_inputs(c), scale=0.5,
                                             state=host64(c["state"]))
        check("o", host64(o), want_o, dtype)
        check("state", host64(state), want_s, "fp32", 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_views_into_a_fused_projection(dtype):
    """q, k, v as slices of one [batch, L, ..] tensor; the same numbers as dense copies."""
    rng = np.random.default_rng(43)
    B, L, Hk, H, dk, dv = 2, 130, 2, 4, 48, 32
    cols = (Hk * dk, Hk * dk, H * dv)
    u = _tensor(rng, (B, L, sum(cols) + 8), dtype).cuda()
    q, k, v = torch.split(u[..., :-8], cols, dim=-1)
    q, k, v = q.unflatten(-1, (Hk, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (H, dv))
    g = -torch.rand(B, L, H, device="cuda")
    dout = _tensor(rng, (B, L, H, dv), dtype).cuda()
    dense = [t.contiguous() for t in (q, k, v)]
    for a, b in zip(mssm.linear_attention(q, k, v, g, return_state=True),
                    mssm.linear_attention(*dense, g, return_state=True)):
        assert torch.equal(a, b)
    a = mssm.linear_attention_bwd(q, k, v, g, dout)
    b = mssm.linear_attention_bwd(*dense, g, dout)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    s1, s2 = (torch.zeros(B, H, dk, dv, device="cuda") for _ in range(2))
    assert torch.equal(mssm.linear_attention_step(q[:, 3], k[:, 3], v[:, 3], g[:, 3].contiguous(), s1),
                       mssm.linear_attention_step(*(t[:, 3].contiguous() for t in dense),
                                                  g[:, 3].contiguous(), s2))
    assert torch.equal(s1, s2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_unaligned_tensors(dtype):
    """Every pointer one element (state: one float) past a 16-byte boundary: the same numbers."""
    c = make(44, [200], 2, 4, 64, 48, dtype)
    names = ("q", "k", "v", "log_decay", "state", "dout", "dlast")
    shifted, dense = {}, {}
    for n in names:
        dense[n] = c[n].cuda()
        big = torch.empty(dense[n].numel() + 1, dtype=dense[n].dtype, device="cuda")
        big[1:] = dense[n].flatten()
        shifted[n] = big[1:].view(dense[n].shape)

    def run(t):
        o, s = mssm.linear_attention(t["q"], t["k"], t["v"], t["log_decay"], state=t["state"],
                                     return_state=True)
        gr = mssm.linear_attention_bwd(t["q"], t["k"], t["v"], t["log_decay"], t["dout"],
                                       state=t["state"], dstate=t["dlast"])
        st = t["state"]
        one = mssm.linear_attention_step(t["q"][:, 5], t["k"][:, 5], t["v"][:, 5],
                                         t["log_decay"][0, 5][None].contiguous(), st)
        return [o, s, one, st.clone()] + [gr[n] for n in sorted(gr)]

    for a, b in zip(run(dense), run(shifted)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decays_at_the_ends(dtype):
    """A decay of one (log 0), to zero (minus infinity, the type's lowest value), slowly
    and by very much in one token."""
    c = make(45, [150], 1, 4, 32, 32, dtype)
    g = c["log_decay"]
    g[..., 0] = 0.0
    g[:, ::40, 1] = float("-inf")
    g[:, 1::40, 1] = torch.finfo(torch.float32).min
    g[..., 2] = float("-inf")                      # every token on its own
    g[:, 70, 3] = -300.0
    g[:, 71:, 3] = -1e-6
    check_forward(c, dtype, with_state=True)
    check_backward(c, dtype, with_state=True, with_dlast=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_not_finite_values_stay_in_their_sequence_and_head(dtype):
    c = make(46, [70, 65, 1, 80], 2, 4, 32, 48, dtype, packed=True)
    kw = offsets_kw(c)
    q, k, v, g, dout, state = on_gpu(c, "q", "k", "v", "log_decay", "dout", "state")
    clean = mssm.linear_attention(q, k, v, g, state=state, return_state=True, **kw)
    clean_g = mssm.linear_attention_bwd(q, k, v, g, dout, state=state, **kw)
    v[71, 3] = float("nan")
    v[135, 2] = float("inf")
    q[80, 1] = float("inf")
    dout[72, 3] = float("nan")
    got = mssm.linear_attention(q, k, v, g, state=state, return_state=True, **kw)
    got_g = mssm.linear_attention_bwd(q, k, v, g, dout, state=state, **kw)
    torch.cuda.synchronize()
    keep = torch.ones(216, dtype=torch.bool, device="cuda")
    keep[70:136] = False                           # sequences 1 and 2, heads 2 and 3
    for a, b in ((got[0], clean[0]), (got_g["dv"], clean_g["dv"]),
                 (got_g["dlog_decay"], clean_g["dlog_decay"])):
        assert torch.equal(a[keep], b[keep])
        assert torch.equal(a[~keep][:, :2], b[~keep][:, :2])
    for n in ("dq", "dk"):
        assert torch.equal(got_g[n][keep], clean_g[n][keep])
        assert torch.equal(got_g[n][~keep][:, :1], clean_g[n][~keep][:, :1])
    for i in (0, 3):
        assert torch.equal(got[1][i], clean[1][i])
        assert torch.equal(got_g["dstate"][i], clean_g["dstate"][i])
    assert torch.isnan(got[0][71:135, 3]).all()    # and they are not lost where they belong
    assert not torch.isfinite(got[0][135, 2]).any()


def test_no_tokens_sequences_or_heads():
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
    f = lambda *s: e(*s, dt=torch.float32)
    o, s = mssm.linear_attention(e(0, 5, 2, 16), e(0, 5, 2, 16), e(0, 5, 2, 16), f(0, 5, 2),
                                 return_state=True)
    assert o.shape == (0, 5, 2, 16) and s.shape == (0, 2, 16, 16)
    o, s = mssm.linear_attention(e(2, 0, 1, 16), e(2, 0, 1, 16), e(2, 0, 3, 32), f(2, 0, 3),
                                 return_state=True)
    torch.cuda.synchronize()
    assert o.shape == (2, 0, 3, 32) and torch.equal(s, torch.zeros_like(s))
    state, dlast = torch.randn(2, 3, 16, 32, device="cuda"), torch.randn(2, 3, 16, 32, device="cuda")
    gr = mssm.linear_attention_bwd(e(2, 0, 1, 16), e(2, 0, 1, 16), e(2, 0, 3, 32),
                                   torch.zeros(3, device="cuda"), e(2, 0, 3, 32), state=state,
                                   dstate=dlast)
    torch.cuda.synchronize()
    assert torch.equal(gr["dstate"], dlast)
    assert torch.equal(gr["dlog_decay"], torch.zeros(3, device="cuda"))
    s = f(0, 2, 16, 16)
    assert mssm.linear_attention_step(e(0, 2, 16), e(0, 2, 16), e(0, 2, 16), f(0, 2), s).numel() == 0


def test_gradient_against_differences():
    """The directional derivative of the GPU's own forward pass in float32.  The loss is
    linear in q, v and the state along their directions, so central differences of step 1/8
    have no error there; along k with q and v fixed likewise.  Along log_decay the third
    derivative leaves h^2/6: h = 1/128 and 1e-3 of the gradients' size."""
    c = make(47, [100], 1, 2, 32, 48, "fp32", decay=(0.01, 0.5))
    names = ("q", "k", "v", "log_decay", "state")
    t = {n: c[n].cuda() for n in names + ("dout", "dlast")}

    def loss(u):
        o, s = mssm.linear_attention(u["q"], u["k"], u["v"], u["log_decay"], state=u["state"],
                                     return_state=True)
        return float((o.double() * t["dout"].double()).sum() +
                     (s.double() * t["dlast"].double()).sum())

    gr = mssm.linear_attention_bwd(t["q"], t["k"], t["v"], t["log_decay"], t["dout"],
                                   state=t["state"], dstate=t["dlast"])
    for n in names:
        direction = torch.from_numpy(np.random.default_rng(3).choice([-1.0, 1.0], t[n].shape)
                                     ).float().cuda()
        h = 1 / 128 if n == "log_decay" else 1 / 8
        moved = [dict(t, **{n: t[n] + s * h * direction}) for s in (1, -1)]
        want = (loss(moved[0]) - loss(moved[1])) / (2 * h)
        grad = gr["d" + n]
        got = float((grad.double() * direction.double()).sum())
        size = float(grad.double().norm())
        assert abs(got - want) <= 1e-3 * size, (n, got, want, size)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_same_bits_every_time_and_on_another_stream(dtype):
    c = make(48, [400, 400], 1, 4, 64, 64, dtype)
    q, k, v, g, dout, state, dlast = on_gpu(c, "q", "k", "v", "log_decay", "dout", "state", "dlast")

    def run(stream=None):
        o, s = mssm.linear_attention(q, k, v, g, state=state, return_state=True, stream=stream)
        gr = mssm.linear_attention_bwd(q, k, v, g, dout, state=state, dstate=dlast, stream=stream)
        return [o, s] + [gr[n] for n in sorted(gr)]

    first = run()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for r in (run(), run(other), run()):
        torch.cuda.synchronize()
        for a, b in zip(first, r):
            assert torch.equal(a, b)


def test_in_a_graph():
    """Prompt, gradient and three steps captured together."""
    c = make(49, [500, 500], 1, 2, 64, 64, "bf16")
    q, k, v, g, dout = on_gpu(c, "q", "k", "v", "log_decay", "dout")
    size = lambda b: mssm.mssm_linear_attention_workspace_size(2, 500, 1, 2, 64, 64, torch.bfloat16,
                                                               backward=b)
    ws = torch.empty(max(size(False), size(True)), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(v)
    state = torch.empty(2, 2, 64, 64, device="cuda")
    ones = [torch.empty(2, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    grads = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
             "dlog_decay": torch.empty_like(g)}
    gt = [g[:, t].contiguous() for t in range(3)]

    def work():
        mssm.mssm_linear_attention_fwd(q, k, v, g, o, ws, scale=0.125, last_state=state)
        for t in range(3):
            mssm.mssm_linear_attention_step(q[:, t], k[:, t], v[:, t], gt[t], state, ones[t],
                                            scale=0.125)
        mssm.mssm_linear_attention_bwd(q, k, v, g, dout, grads, ws, scale=0.125)

    outputs = [o, state] + ones + [grads[n] for n in sorted(grads)]
    work()
    torch.cuda.synchronize()
    expected = [t.clone() for t in outputs]
    graph = capture(work)
    other = make(50, [90], 1, 1, 32, 32, "fp32")
    noise = on_gpu(other, "q", "k", "v", "log_decay")
    replay_and_check(graph, outputs, expected, lambda: mssm.linear_attention(*noise))


def test_refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    q, k, v, g = z(2, 5, 2, 32), z(2, 5, 2, 32), z(2, 5, 4, 48), z(2, 5, 4, dt=torch.float32)
    s = z(2, 4, 32, 48, dt=torch.float32)
    off = torch.tensor([0, 5], device="cuda")
    fwd = mssm.linear_attention
    bad = [
        lambda: fwd(q, k.float(), v, g),                        # types differ
        lambda: fwd(q.half(), k.half(), v.half(), g),
        lambda: fwd(q, k, v, g.bfloat16()),
        lambda: fwd(q, k, v.cpu(), g),
        lambda: fwd(q, z(2, 5, 2, 48), v, g),                   # sizes differ
        lambda: fwd(q, z(2, 6, 2, 32), v, g),
        lambda: fwd(z(2, 5, 3, 32), z(2, 5, 3, 32), v, g),      # 4 heads over 3 key heads
        lambda: fwd(q, k, v, z(2, 5, 2, dt=torch.float32)),
        lambda: fwd(q, k, v, z(2, dt=torch.float32)),
        lambda: fwd(q, k, v, z(2, 4, 5, dt=torch.float32).transpose(1, 2)),
        lambda: fwd(q, k, v, g, state=s[:1]),
        lambda: fwd(q, k, v, g, state=s.bfloat16()),
        lambda: fwd(q, k, v, g, state=s.transpose(0, 1).contiguous().transpose(0, 1)),
        lambda: fwd(z(2, 32, 2, 5).transpose(1, 3), k, v, g),   # a head's values apart
        lambda: fwd(z(2, 2, 5, 32).transpose(1, 2), k, v, g),   # heads apart
        lambda: fwd(q[:, ::2], k[:, ::2], v[:, ::2], g[:, ::2]),
        lambda: fwd(q, k, v, g, seq_offsets=off),               # packed tensors have three dims
        lambda: fwd(q[0], k[0], v[0], g[0], seq_offsets=off.int()),
        lambda: fwd(q[0], k[0], v[0], g[0], seq_offsets=off.cpu()),
        lambda: mssm.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0].contiguous(), s[:1]),
        lambda: mssm.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], s.double()),
        lambda: mssm.linear_attention_bwd(q, k, v, g, v[:, :4]),
        lambda: mssm.linear_attention_bwd(q, k, v, g, v.float()),
        lambda: mssm.linear_attention_bwd(q, k, v, g, v, dstate=s[0]),
        lambda: mssm.mssm_linear_attention_fwd(q, k, v, g, q, None, scale=1.0),
        lambda: mssm.mssm_linear_attention_bwd(q, k, v, g, v, {"dx": v}, None, scale=1.0),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, mssm.MssmError)):
            call()
            pytest.fail(f"refusal {i} was accepted")
    for d in (8, 40, 144):
        with pytest.raises((ValueError, RuntimeError)):
            fwd(z(1, 4, 1, d), z(1, 4, 1, d), z(1, 4, 1, 16), z(1, 4, 1, dt=torch.float32))
    long = z(1, 4000, 1, 64)
    with pytest.raises(RuntimeError):                           # no workspace
        mssm.mssm_linear_attention_fwd(long, long, long, z(1, 4000, 1, dt=torch.float32),
                                       torch.empty_like(long), None, scale=1.0)
    torch.cuda.synchronize()


def _long_case(seed, L, H, kinds):
    """One sequence of dk = dv = 16 whose heads have the given log decays."""
    c = make(seed, [L], H, H, 16, 16, "fp32")
    c["log_decay"] = torch.stack([torch.from_numpy(k).float() for k in kinds], -1)[None]
    return c


@pytest.mark.parametrize("backward", [False, True], ids=["prompt", "gradient"])
def test_tokens_out_of_reach_of_a_segments_state(backward):
    """Segments long enough that the state pass looks for the tokens that can reach a
    segment's state at all: memories of a few tokens, of about half a segment, longer than
    a segment and endless; resets at, before and after a segment's ends; log decays above
    zero before the state all but vanishes (the tokens before them count no more)."""
    L, H = 17000, 32
    seg = 544                                        # tokens a segment, by the size query's rule
    rng = np.random.default_rng(60)
    t = np.arange(L)
    pulse = np.where(t % seg == 400, 60.0, np.where(t % seg == 401, -300.0, -0.01))
    kinds = [np.full(L, -3.0), np.full(L, -0.5), np.full(L, -0.05), np.full(L, -1e-4),
             np.where(t % seg == seg - 1, -np.inf, -0.02), np.where(t % seg == 0, -np.inf, -0.02),
             np.where(t % seg == 1, -1e30, -0.02), np.where(t % 700 == 0, -250.0, -0.002), pulse,
             -rng.exponential(0.4, L)] + [np.full(L, -0.3)] * (H - 10)
    c = _long_case(61, L, H, kinds)
    q, k, v, g, dout, state, dlast = on_gpu(c, "q", "k", "v", "log_decay", "dout", "state", "dlast")
    heads = range(10)
    part = lambda a, ax: np.take(a, heads, axis=ax)
    Q, K, V, G, _ = oracle_inputs(c)
    args = (part(Q, 1), part(K, 1), part(V, 1), part(G, 1), c["offsets"])
    s0 = part(host64(c["state"]), 1)
    if not backward:
        o, last = mssm.linear_attention(q, k, v, g, scale=0.25, state=state, return_state=True)
        torch.cuda.synchronize()
        want_o, want_s = la.linear_attention(*args, scale=0.25, state=s0)
        check("o", part(host64(o)[0], 1), want_o, "fp32")
        check("last state", part(host64(last), 1), want_s, "fp32", 1)
        return
    got = mssm.linear_attention_bwd(q, k, v, g, dout, scale=0.25, state=state, dstate=dlast)
    torch.cuda.synchronize()
    want = la.linear_attention_backward(*args, part(host64(c["dout"])[0], 1), scale=0.25, state=s0,
                                        dlast=part(host64(c["dlast"]), 1))
    for n in ("dq", "dk", "dv"):
        check(n, part(host64(got[n])[0], 1), want[n], "fp32")
    check("dlog_decay", part(host64(got["dlog_decay"])[0], 1), want["dlog_decay"], "decay", -1)
    check("dstate", part(host64(got["dstate"]), 1), want["dstate"], "fp32", 1)


def test_offsets_past_32_bits():
    """A packed sequence that begins past 2^31 values, after one whose end is past them."""
    H, d, n = 16, 128, 150
    T1 = 2 ** 31 // (H * d) + 1000
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, dout = (torch.empty(T1 + n, H, d, dtype=torch.bfloat16, device="cuda").normal_(
        generator=gen) for _ in range(4))
    g = torch.empty(T1 + n, H, device="cuda").uniform_(-0.6, -0.4, generator=gen)
    off = torch.tensor([0, T1, T1 + n], device="cuda")
    o, last = mssm.linear_attention(q, k, v, g, seq_offsets=off, return_state=True)
    gr = mssm.linear_attention_bwd(q, k, v, g, dout, seq_offsets=off)
    torch.cuda.synchronize()
    host = lambda t, a, b: host64(t[a:b])
    # the first sequence's end: decays of exp(-80) and less make 200 tokens before it enough
    a, b = T1 - 250, T1
    want_o, want_s = la.linear_attention(*(host(t, a, b) for t in (q, k, v, g)),
                                         np.array([0, 250]), scale=d ** -0.5)
    check("o", host(o, b - 50, b), want_o[200:], "bf16")
    check("last state", host64(last[:1]), want_s, "fp32", 1)
    # the second sequence
    a, b = T1, T1 + n
    args = [host(t, a, b) for t in (q, k, v, g)] + [np.array([0, n])]
    want_o, want_s = la.linear_attention(*args, scale=d ** -0.5)
    check("o", host(o, a, b), want_o, "bf16")
    check("last state", host64(last[1:]), want_s, "fp32", 1)
    want = la.linear_attention_backward(*args, host(dout, a, b), scale=d ** -0.5)
    for name in ("dq", "dk", "dv"):
        check(name, host(gr[name], a, b), want[name], "bf16")
    check("dlog_decay", host(gr["dlog_decay"], a, b), want["dlog_decay"], "decay", -1)


def test_step_with_states_past_32_bits():
    """More than 2^31 state values; the last sequences against the oracle."""
    H, d = 16, 128
    B = 2 ** 31 // (H * d * d) + 2
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.empty(B, H, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
               for _ in range(3))
    g = torch.empty(H, device="cuda").uniform_(-1.0, 0.0, generator=gen)
    state = torch.empty(B, H, d, d, device="cuda").normal_(generator=gen)
    before = host64(state[-2:])
    o = mssm.linear_attention_step(q, k, v, g, state)
    torch.cuda.synchronize()
    want_o, want_s = la.linear_attention(host64(q[-2:]), host64(k[-2:]), host64(v[-2:]), host64(g),
                                         np.arange(3), scale=d ** -0.5, state=before)
    check("o", host64(o[-2:]), want_o, "bf16")
    check("state", host64(state[-2:]), want_s, "fp32", 1)
