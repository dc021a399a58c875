"""Helpers of the tests of the gated recurrence and the causal convolution with states: inputs as
packed or dense tokens, and comparison against bounds given element by element."""
import numpy as np
import torch

from gpu_support import host64

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
ULP = 2.0 ** -24


def tensor(rng, shape, dtype, spread=1.0):
    return torch.from_numpy(spread * rng.standard_normal(shape)).to(DT[dtype])


def offsets_of(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def lay(c, *names):
    """The named [T, D] tensors on the GPU, as [batch, L, D] where the sequences are dense."""
    out = []
    for n in names:
        t = c[n].cuda()
        out.append(t if c["packed"] else t.view(len(c["lengths"]), -1, t.shape[-1]))
    return out


def offsets_kw(c):
    return {"seq_offsets": torch.from_numpy(c["offsets"]).cuda()} if c["packed"] else {}


def check(name, got, want, bound, dtype):
    """|got - want| <= half a step of the type relative to want, plus the bound."""
    got = host64(got).reshape(want.shape)
    assert np.isfinite(got).all(), f"{name} is not finite"
    if not want.size:
        return
    tol = HALF_STEP[dtype] * np.abs(want) * (1 + 1e-6) + bound + 1e-37
    ratio = float((np.abs(got - want) / tol).max())
    assert ratio <= 1.0, f"{name}: error {ratio:.3g} of the tolerance"


def shifted(t):
    """The same values one element past a 16-byte boundary."""
    big = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    big[1:] = t.flatten()
    return big[1:].view(t.shape)


def fused(*tensors):
    """The tensors as slices of one wider tensor (with a few more columns behind them)."""
    wide = torch.cat([*tensors, tensors[0][..., :8]], dim=-1)
    D = tensors[0].shape[-1]
    return [wide[..., j * D:(j + 1) * D] for j in range(len(tensors))]
