"""Linear attention in bfloat16 on the GPU: what an output depends on, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from selective_state_space_54_amd import mssm  # noqa: E402
from test_linear_attention_gpu import make, offsets_kw, on_gpu  # noqa: E402

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
