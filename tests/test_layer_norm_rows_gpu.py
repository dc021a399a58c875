"""Layer norm over many rows on the GPU against the float64 formulas: tolerances and
helpers of test_layer_norm_gpu."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from gpu_support import host64  # noqa: E402
from oracle import layer_norm as ln  # noqa: E402
from selective_state_space_54_amd import mssm  # noqa: E402
from test_layer_norm_gpu import check, check_norm, make  # noqa: E402


def _spot_check(rows, D, picks):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    w = torch.empty(D, device="cuda").uniform_(0.5, 1.5, generator=gen)
    y, mean, rstd = mssm.layer_norm(x, w, return_stats=True)
    torch.cuda.synchronize()
    for p in picks:
        x64 = host64(x[p])
        want, m64, r64 = ln.layer_norm(x64, host64(w), eps=1e-5)
        check("mean", mean[p], m64, "fp32", np.ones(len(m64)))
        check("rstd", rstd[p], r64, "fp32", 2 * r64)
        check("y", y[p], want, "bf16", np.abs(want) + host64(w))
    return x, w, mean, rstd


def test_rows_of_every_head_of_a_long_prompt():
    """131072 tokens of 40 heads, normed head by head; a constant gradient's sums."""
    rows, D = 131072 * 40, 64
    x, w, mean, rstd = _spot_check(rows, D, [slice(0, 64), slice(rows // 2, rows // 2 + 64),
                                             slice(rows - 64, rows)])
    gr = mssm.layer_norm_bwd(torch.ones_like(x), x, w, mean, rstd)
    torch.cuda.synchronize()
    assert torch.equal(gr["dbias"], torch.full((D,), float(rows), device="cuda"))


def test_more_rows_than_a_grid_of_wide_blocks():
    """Rows of a block of 1024 threads each, more than 2^32 / 1024."""
    rows, D = (1 << 22) + 70, 8200
    if torch.cuda.mem_get_info()[0] < 5 * rows * D:
        pytest.skip("needs 170 GB of memory")
    _spot_check(rows, D, [slice(0, 8), slice((1 << 22) - 2, 1 << 22), slice(rows - 8, rows)])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [1000, 2560, 2600, 5000, 8200, 16384])
def test_parameter_gradients_over_more_rows_than_blocks(dtype, D):
    """A block then sums several rows: also those that a whole block holds."""
    check_norm(make(D, 700, D, dtype), dtype, residual=D != 5000, bias=True)
