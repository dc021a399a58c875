"""Linear attention on the GPU: what an output depends on, bit for bit, and that bfloat16
outputs are rounded once.

Tolerance of a bfloat16 output, |err| <= 2^-8 |ref| + 2^-13 rms, rms over a head's
tokens: its own rounding is at most 2^-8 of it.  An operand in two bfloat16 parts errs
by at most 2^-16 of itself, with a deviation of some 2^-17.5, so a sum of such products
by 2^-17.5 of its size, sqrt(2) times that for two operands (scores, state), and five
to six deviations for the largest of many: 2^-14.5.  The float32 sums add 300 * 2^-24.
Together 2^-14 of the token's own size, which may be twice the head's.  (One bfloat16
part, deviation 2^-9.5, would go past it 100 times over where |ref| is small.)
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_support import host64  # noqa: E402
from oracle import linear_attention as la  # noqa: E402
from selective_state_space_54_amd import mssm  # noqa: E402
from test_linear_attention_gpu import make, offsets_kw, on_gpu, oracle_inputs, tokens  # noqa: E402

# lengths (one sequence: cut into segments), packed, key heads, heads, dk, dv
CASES = [([700, 700], False, 2, 4, 64, 64), ([3000], False, 1, 1, 128, 128),
         ([300, 0, 1, 450], True, 1, 2, 128, 48), ([130], False, 3, 3, 16, 96)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_outputs_do_not_depend_on_whether_the_last_state_is_asked_for(dtype, case):
    lengths, packed, *heads = case
    c = make(70, lengths, *heads, dtype, packed=packed, decay=(1e-4, 0.3))
    q, k, v, g, state = on_gpu(c, "q", "k", "v", "log_decay", "state")
    for s in (None, state):
        o = mssm.linear_attention(q, k, v, g, state=s, **offsets_kw(c))
        with_last, _ = mssm.linear_attention(q, k, v, g, state=s, return_state=True,
                                             **offsets_kw(c))
        torch.cuda.synchronize()
        assert torch.equal(o, with_last)


def check_once_rounded(name, got, want):
    got = host64(got).reshape(want.shape)
    rms = np.sqrt(np.mean(want ** 2, axis=(0, 2), keepdims=True))
    ratio = float((np.abs(got - want) / (2.0 ** -8 * np.abs(want) + 2.0 ** -13 * rms)).max())
    assert ratio <= 1.0, f"{name}: error {ratio:.3g} of the tolerance"


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("decay", [(1e-4, 0.3), (1.0, 4.0)], ids=["slow", "fast"])
def test_bfloat16_outputs_are_rounded_once(case, decay):
    lengths, packed, *heads = case
    c = make(71, lengths, *heads, "bf16", packed=packed, decay=decay)
    q, k, v, g, state, dout, dlast = on_gpu(c, "q", "k", "v", "log_decay", "state", "dout", "dlast")
    o = mssm.linear_attention(q, k, v, g, scale=0.2, state=state, **offsets_kw(c))
    gr = mssm.linear_attention_bwd(q, k, v, g, dout, scale=0.2, state=state, dstate=dlast,
                                   **offsets_kw(c))
    torch.cuda.synchronize()
    s0, d1 = host64(c["state"]), host64(c["dlast"])
    check_once_rounded("o", o, la.linear_attention(*oracle_inputs(c), scale=0.2, state=s0)[0])
    want = la.linear_attention_backward(*oracle_inputs(c), tokens(c["dout"], packed, 2), scale=0.2,
                                        state=s0, dlast=d1)
    for n in ("dq", "dk", "dv"):
        check_once_rounded(n, gr[n], want[n])
