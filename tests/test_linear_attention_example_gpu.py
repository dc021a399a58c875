"""The example layer: it learns, and serves token by token what its prompt pass gives."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "linear_attention_layer.py")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layer_learns_and_serves(dtype):
    """The task is a copy of 16 symbols: log 16 = 2.77 without learning.  Served logits differ
    by the roundings of three bfloat16 tensors a layer (2^-8 each, some six deviations of
    them in the largest), in float32 by the order of sums."""
    spec = importlib.util.spec_from_file_location("linear_attention_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last, diff = example.main(steps=60, dtype=dtype, quiet=True)
    assert first > 2.0 and last < 0.75 * first
    assert diff <= (0.15 if dtype == "bf16" else 1e-3)
