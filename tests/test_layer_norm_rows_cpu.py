"""Layer norm's limits on the rows, by the size query (no GPU needed)."""
import ctypes
import os

import pytest

mssm = pytest.importorskip("selective_state_space_54_amd.mssm")
OK, UNSUPPORTED = 0, 2


@pytest.mark.parametrize("dtype", [0, 1], ids=["fp32", "bf16"])
@pytest.mark.parametrize("D", [1, 64, 128, 2560, 4096, 16384])
def test_rows_up_to_2_to_the_32(dtype, D):
    if not os.path.exists(mssm.LIB_PATH):
        pytest.skip("libmssm.so not built")
    out = ctypes.c_size_t(0)
    size = lambda rows: mssm.load().mssm_layer_norm_bwd_workspace_size(rows, D, dtype,
                                                                       ctypes.byref(out))
    for rows in (1 << 22, 131072 * 40, (1 << 32) - 1):
        assert size(rows) == OK and out.value >= 2 * D * 4
    assert size(1 << 32) == UNSUPPORTED
