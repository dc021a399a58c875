"""Python binding of the mssm C ABI (libmssm.so), argument marshalling only.

Every function here carries the name of the C entry point it calls and does
no arithmetic of the method: it checks tensors (device, dtype, shape,
contiguity), passes raw device pointers and the current HIP stream, and turns
status codes into exceptions.  PyTorch supplies device memory and streams.
There is no fallback: if the library is missing, loading fails loudly.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmssm.so")

MSSM_SUCCESS = 0
MSSM_ERROR_INVALID_VALUE = 1
MSSM_ERROR_NOT_SUPPORTED = 2
MSSM_ERROR_SIZE_OVERFLOW = 3
MSSM_ERROR_WORKSPACE = 4
MSSM_ERROR_HIP = 5
MSSM_FLOAT32 = 0
MSSM_BFLOAT16 = 1
MSSM_BBAR_EULER = 0
MSSM_BBAR_ZOH = 1
_BBAR = {"euler": MSSM_BBAR_EULER, "zoh": MSSM_BBAR_ZOH}
MSSM_DECAY_PER_HEAD = 0
MSSM_DECAY_PER_TOKEN = 1
MSSM_TUNE_SCAN_ORDER = 0
MSSM_TUNE_CHUNK_LEN = 1
MSSM_TUNE_CHAINS_PER_LANE = 2
MSSM_ORDER_AUTO = 0
MSSM_ORDER_CHUNKED = 1
MSSM_ORDER_SINGLE_PASS = 2
_ORDERS = {"auto": MSSM_ORDER_AUTO, "chunked": MSSM_ORDER_CHUNKED,
           "chain": MSSM_ORDER_SINGLE_PASS, "single_pass": MSSM_ORDER_SINGLE_PASS}
_DTYPES = {torch.float32: MSSM_FLOAT32, torch.bfloat16: MSSM_BFLOAT16}
_STATUS_NAMES = {0: "MSSM_SUCCESS", 1: "MSSM_ERROR_INVALID_VALUE", 2: "MSSM_ERROR_NOT_SUPPORTED",
                 3: "MSSM_ERROR_SIZE_OVERFLOW", 4: "MSSM_ERROR_WORKSPACE", 5: "MSSM_ERROR_HIP"}

_lib = None

# (name, restype, argtypes) of every exported entry point declared in include/mssm.h
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_SIGNATURES = {
    "mssm_abi_version": (ctypes.c_int, []),
    "mssm_set_tuning": (ctypes.c_int, [ctypes.c_int, _i64]),
    "mssm_get_tuning": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]),
    "mssm_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mssm_last_error_string": (ctypes.c_char_p, []),
    "mssm_supports_state_size": (ctypes.c_int, [_i64]),
    "mssm_selective_scan_workspace_size": (ctypes.c_int, [_i64, _i64, _i64, _i64, ctypes.c_int,
                                                          ctypes.POINTER(ctypes.c_size_t)]),
    "mssm_selective_scan_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                                               _i64, ctypes.c_int, _vp]),
    "mssm_selective_scan_fwd_ws": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                  ctypes.c_size_t, _i64, _i64, _i64, _i64,
                                                  ctypes.c_int, _vp]),
    "mssm_selective_scan_fwd_noalloc": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                                                       _i64, _i64, ctypes.c_int, _vp]),
    "mssm_selective_scan_fwd_ex": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                  _vp, ctypes.c_int, _vp, ctypes.c_size_t, _i64,
                                                  _i64, _i64, _i64, ctypes.c_int, _vp]),
    "mssm_selective_scan_step": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                ctypes.c_int, _i64, _i64, _i64, ctypes.c_int,
                                                _vp]),
    "mssm_fused_supports": (ctypes.c_int, [_i64, _i64]),
    "mssm_selective_scan_bwd_workspace_size": (ctypes.c_int, [_i64, _i64, _i64, _i64,
                                                              ctypes.c_int,
                                                              ctypes.POINTER(ctypes.c_size_t)]),
    "mssm_selective_scan_bwd": (ctypes.c_int, [_vp] * 17 + [_vp, ctypes.c_size_t] + [_i64] * 4 +
                                [ctypes.c_int, _vp]),
    "mssm_selective_scan_saved_size": (ctypes.c_int, [_i64, _i64, _i64, _i64, ctypes.c_int,
                                                      ctypes.POINTER(ctypes.c_size_t)]),
    "mssm_selective_scan_fwd_save": (ctypes.c_int, [_vp] * 11 + [ctypes.c_size_t] + [_i64] * 4 +
                                     [ctypes.c_int, _vp]),
    "mssm_selective_scan_bwd_saved": (ctypes.c_int, [_vp] * 9 + [ctypes.c_size_t] + [_vp] * 10 +
                                      [ctypes.c_size_t] + [_i64] * 4 + [ctypes.c_int, _vp]),
    "mssm_causal_conv1d_silu": (ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                               ctypes.c_int, _vp]),
    "mssm_mamba_block_supports": (ctypes.c_int, [_i64, _i64, _i64]),
    "mssm_mamba_block_workspace_size": (ctypes.c_int, [_i64, _i64, _i64, _i64, _i64, _i64, _i64,
                                                       ctypes.c_int,
                                                       ctypes.POINTER(ctypes.c_size_t)]),
    "mssm_mamba_block_fwd": (ctypes.c_int, [_vp] * 12 + [ctypes.c_size_t] + [_i64] * 7 +
                             [ctypes.c_int, _vp]),
    "mssm_selective_ssm_fused_workspace_size": (ctypes.c_int, [_i64, _i64, _i64, _i64, _i64,
                                                               ctypes.c_int,
                                                               ctypes.POINTER(ctypes.c_size_t)]),
    "mssm_selective_ssm_fused_fwd": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                    ctypes.c_size_t, _i64, _i64, _i64, _i64,
                                                    _i64, ctypes.c_int, _vp]),
    "mssm_linear_attention_supports": (ctypes.c_int, [_i64, _i64]),
    "mssm_linear_attention_workspace_size": (ctypes.c_int, [_i64] * 6 + [ctypes.c_int] * 3 +
                                             [ctypes.POINTER(ctypes.c_size_t)]),
    "mssm_linear_attention_fwd": (ctypes.c_int, [_vp] * 8 + [ctypes.c_float, ctypes.c_int, _vp,
                                                             ctypes.c_size_t] + [_i64] * 9 +
                                  [ctypes.c_int, _vp]),
    "mssm_linear_attention_step": (ctypes.c_int, [_vp] * 6 + [ctypes.c_float, ctypes.c_int] +
                                   [_i64] * 8 + [ctypes.c_int, _vp]),
    "mssm_linear_attention_bwd": (ctypes.c_int, [_vp] * 13 + [ctypes.c_float, ctypes.c_int, _vp,
                                                              ctypes.c_size_t] + [_i64] * 9 +
                                  [ctypes.c_int, _vp]),
    "mssm_layer_norm_fwd": (ctypes.c_int, [_vp] * 8 + [ctypes.c_float, _i64, _i64, ctypes.c_int,
                                                       _vp]),
    "mssm_layer_norm_bwd_workspace_size": (ctypes.c_int, [_i64, _i64, ctypes.c_int,
                                                          ctypes.POINTER(ctypes.c_size_t)]),
    "mssm_layer_norm_bwd": (ctypes.c_int, [_vp] * 10 + [ctypes.c_size_t, _i64, _i64, ctypes.c_int,
                                                        _vp]),
}


class MssmError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = load()
        text = lib.mssm_status_string(status).decode()
        extra = lib.mssm_last_error_string().decode() if status == 5 else ""
        super().__init__(f"{where}: {_STATUS_NAMES.get(status, status)} ({text}) {extra}".strip())
        self.status = status


def load():
    """Load libmssm.so (built by selective_state_space_54_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run selective_state_space_54_amd.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def exported_symbols():
    return sorted(_SIGNATURES)


def _check(status: int, where: str):
    if status != MSSM_SUCCESS:
        raise MssmError(status, where)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dense(t: torch.Tensor, name: str, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace_args(workspace, device):
    """Address and bytes of a caller's workspace tensor, None and 0 without one."""
    if workspace is None:
        return None, 0
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    nbytes = workspace.numel() * workspace.element_size()
    return (workspace.data_ptr() if nbytes else None), nbytes


def _dtype_code(dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"dtype {dtype} not supported (float32 or bfloat16)")
    return _DTYPES[dtype]


def mssm_abi_version() -> int:
    return load().mssm_abi_version()


def mssm_set_tuning(key: int, value: int) -> None:
    """Set one process-wide tuning value (MSSM_TUNE_*)."""
    _check(load().mssm_set_tuning(key, value), "mssm_set_tuning")


def mssm_get_tuning(key: int) -> int:
    out = ctypes.c_int64(0)
    _check(load().mssm_get_tuning(key, ctypes.byref(out)), "mssm_get_tuning")
    return out.value


@contextlib.contextmanager
def tuning(scan_order=None, chunk_len=None, chains_per_lane=None):
    """Pin tuning settings for the calls made inside the block and restore the
    previous values afterwards.  scan_order: "auto", "chunked" or "chain";
    chunk_len: steps per chunk (0: automatic); chains_per_lane: 0, 1 or 2."""
    wanted = {}
    if scan_order is not None:
        if scan_order not in _ORDERS:
            raise ValueError(f"scan_order must be one of {sorted(_ORDERS)}")
        wanted[MSSM_TUNE_SCAN_ORDER] = _ORDERS[scan_order]
    if chunk_len is not None:
        wanted[MSSM_TUNE_CHUNK_LEN] = int(chunk_len)
    if chains_per_lane is not None:
        wanted[MSSM_TUNE_CHAINS_PER_LANE] = int(chains_per_lane)
    old = {k: mssm_get_tuning(k) for k in wanted}
    try:
        for k, v in wanted.items():
            mssm_set_tuning(k, v)
        yield
    finally:
        for k, v in old.items():
            mssm_set_tuning(k, v)


_HERE_STREAM = contextlib.nullcontext()


def _on(stream):
    """Allocations for a call launched on `stream` are made on that stream, so
    the caching allocator orders their reuse after the call's kernels."""
    return torch.cuda.stream(stream) if stream is not None else _HERE_STREAM


def mssm_supports_state_size(N: int) -> bool:
    return bool(load().mssm_supports_state_size(N))


def mssm_selective_scan_workspace_size(batch: int, L: int, D: int, N: int,
                                       dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(load().mssm_selective_scan_workspace_size(batch, L, D, N, _dtype_code(dtype),
                                                     ctypes.byref(out)),
           "mssm_selective_scan_workspace_size")
    return out.value


def _scan_shapes(x, A):
    if x.dim() != 3:
        raise ValueError("x must be [batch, L, D]")
    if A.dim() != 2:
        raise ValueError("A must be [D, N]")
    batch, L, D = x.shape
    N = A.shape[1]
    return batch, L, D, N


def _check_scan_args(x, delta, A, B, C, y):
    batch, L, D, N = _scan_shapes(x, A)
    _dtype_code(x.dtype)
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _dense(x, "x", x.dtype, (batch, L, D), dev)
    _dense(delta, "delta", x.dtype, (batch, L, D), dev)
    _dense(A, "A", torch.float32, (D, N), dev)
    _dense(B, "B", x.dtype, (batch, L, N), dev)
    _dense(C, "C", x.dtype, (batch, L, N), dev)
    _dense(y, "y", torch.float32, (batch, L, D), dev)
    return batch, L, D, N


def mssm_selective_scan_fwd(x, delta, A, B, C, y, *, stream=None):
    """y <- selective scan of (x, delta, A, B, C); library-managed workspace."""
    batch, L, D, N = _check_scan_args(x, delta, A, B, C, y)
    _check(load().mssm_selective_scan_fwd(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(y), batch, L, D, N,
        _DTYPES[x.dtype], _stream_handle(stream)), "mssm_selective_scan_fwd")
    return y


NOALLOC_SCRATCH_BYTES = 128 << 20


def mssm_selective_scan_fwd_noalloc(x, delta, A, B, C, y, *, stream=None):
    """y <- selective scan of (x, delta, A, B, C) with the chunk summaries in the
    library's fixed per-GPU scratch array: the call allocates nothing."""
    batch, L, D, N = _check_scan_args(x, delta, A, B, C, y)
    _check(load().mssm_selective_scan_fwd_noalloc(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(y), batch, L, D, N,
        _DTYPES[x.dtype], _stream_handle(stream)), "mssm_selective_scan_fwd_noalloc")
    return y


def mssm_selective_scan_fwd_ws(x, delta, A, B, C, y, workspace, *, stream=None):
    """y <- selective scan with a caller-provided uint8 device workspace tensor."""
    batch, L, D, N = _check_scan_args(x, delta, A, B, C, y)
    ws_ptr, ws_bytes = _workspace_args(workspace, x.device)
    _check(load().mssm_selective_scan_fwd_ws(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(y), ws_ptr, ws_bytes,
        batch, L, D, N, _DTYPES[x.dtype], _stream_handle(stream)), "mssm_selective_scan_fwd_ws")
    return y


class PreparedCall:
    """One C-ABI call whose arguments were validated and converted once.
    Calling it issues the same call again (same buffers, same stream) without
    the per-call Python checks, for loops whose launches would otherwise wait
    on the host.  It holds references to the tensors it was built from."""

    __slots__ = ("_fn", "_args", "_where", "_keep")

    def __init__(self, fn, args, where, keep):
        self._fn, self._args, self._where, self._keep = fn, args, where, keep

    def __call__(self):
        status = self._fn(*self._args)
        if status != MSSM_SUCCESS:
            raise MssmError(status, self._where)


def prepare_selective_scan_fwd_ws(x, delta, A, B, C, y, workspace, *, stream=None):
    """mssm_selective_scan_fwd_ws as a PreparedCall."""
    batch, L, D, N = _check_scan_args(x, delta, A, B, C, y)
    ws_ptr, ws_bytes = _workspace_args(workspace, x.device)
    args = (_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(y), ws_ptr, ws_bytes,
            batch, L, D, N, _DTYPES[x.dtype], _stream_handle(stream))
    return PreparedCall(load().mssm_selective_scan_fwd_ws, args, "mssm_selective_scan_fwd_ws",
                        (x, delta, A, B, C, y, workspace))


def selective_scan(x, delta, A, B, C, *, stream=None):
    """Allocate y and the workspace with torch, then run mssm_selective_scan_fwd_ws."""
    batch, L, D, N = _scan_shapes(x, A)
    nbytes = mssm_selective_scan_workspace_size(batch, L, D, N, x.dtype)
    with _on(stream):
        y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    return mssm_selective_scan_fwd_ws(x, delta, A, B, C, y, ws, stream=stream)


def _bbar_code(bbar) -> int:
    if bbar not in _BBAR:
        raise ValueError(f"bbar must be one of {sorted(_BBAR)}")
    return _BBAR[bbar]


def _check_optional(t, name, dtype, shape, device):
    if t is not None:
        _dense(t, name, dtype, shape, device)


def mssm_selective_scan_fwd_ex(x, delta, A, B, C, y, workspace, *, Dskip=None, z=None, h0=None,
                               h_last=None, bbar="euler", stream=None):
    """y (and h_last) <- the scan with its optional parts: ``bbar`` "euler" or
    "zoh", feedthrough Dskip [D], gate z [batch, L, D], initial state h0 and
    final state h_last [batch, D, N] (float32)."""
    batch, L, D, N = _check_scan_args(x, delta, A, B, C, y)
    dev = x.device
    _check_optional(Dskip, "Dskip", torch.float32, (D,), dev)
    _check_optional(z, "z", x.dtype, (batch, L, D), dev)
    _check_optional(h0, "h0", torch.float32, (batch, D, N), dev)
    _check_optional(h_last, "h_last", torch.float32, (batch, D, N), dev)
    ws_ptr, ws_bytes = _workspace_args(workspace, x.device)
    _check(load().mssm_selective_scan_fwd_ex(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(z), _ptr(h0), _ptr(y),
        _ptr(h_last), _bbar_code(bbar), ws_ptr, ws_bytes, batch, L, D, N, _DTYPES[x.dtype],
        _stream_handle(stream)), "mssm_selective_scan_fwd_ex")
    return y


def selective_scan_ex(x, delta, A, B, C, *, Dskip=None, z=None, h0=None,
                      return_last_state=False, bbar="euler", stream=None):
    """Allocate y (and the final state) with torch, then run
    mssm_selective_scan_fwd_ex.  Returns y, or (y, h_last)."""
    batch, L, D, N = _scan_shapes(x, A)
    nbytes = mssm_selective_scan_workspace_size(batch, L, D, N, x.dtype)
    with _on(stream):
        y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        h_last = (torch.empty((batch, D, N), dtype=torch.float32, device=x.device)
                  if return_last_state else None)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
    mssm_selective_scan_fwd_ex(x, delta, A, B, C, y, ws, Dskip=Dskip, z=z, h0=h0, h_last=h_last,
                               bbar=bbar, stream=stream)
    return (y, h_last) if return_last_state else y


def mssm_selective_scan_step(x, delta, A, B, C, h, y, *, Dskip=None, z=None, bbar="euler",
                             stream=None):
    """One decode step: h [batch, D, N] float32 is updated in place and
    y [batch, D] float32 receives the output; x, delta, z are [batch, D],
    B, C are [batch, N]."""
    if x.dim() != 2 or A.dim() != 2:
        raise ValueError("x must be [batch, D] and A [D, N]")
    batch, D = x.shape
    N = A.shape[1]
    _dtype_code(x.dtype)
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _dense(x, "x", x.dtype, (batch, D), dev)
    _dense(delta, "delta", x.dtype, (batch, D), dev)
    _dense(A, "A", torch.float32, (D, N), dev)
    _dense(B, "B", x.dtype, (batch, N), dev)
    _dense(C, "C", x.dtype, (batch, N), dev)
    _dense(h, "h", torch.float32, (batch, D, N), dev)
    _dense(y, "y", torch.float32, (batch, D), dev)
    _check_optional(Dskip, "Dskip", torch.float32, (D,), dev)
    _check_optional(z, "z", x.dtype, (batch, D), dev)
    _check(load().mssm_selective_scan_step(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(z), _ptr(h), _ptr(y),
        _bbar_code(bbar), batch, D, N, _DTYPES[x.dtype], _stream_handle(stream)),
        "mssm_selective_scan_step")
    return y


def selective_scan_step(x, delta, A, B, C, h, *, Dskip=None, z=None, bbar="euler", stream=None):
    """Allocate y, run mssm_selective_scan_step (h updated in place), return y."""
    with _on(stream):
        y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    return mssm_selective_scan_step(x, delta, A, B, C, h, y, Dskip=Dskip, z=z, bbar=bbar,
                                    stream=stream)


# ---- fused selective SSM (projections + scan) ----------------------------------------------

def mssm_fused_supports(N: int, R: int) -> bool:
    return bool(load().mssm_fused_supports(N, R))


def mssm_selective_ssm_fused_workspace_size(batch: int, L: int, D: int, N: int, R: int,
                                            dtype: torch.dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(load().mssm_selective_ssm_fused_workspace_size(batch, L, D, N, R, _dtype_code(dtype),
                                                          ctypes.byref(out)),
           "mssm_selective_ssm_fused_workspace_size")
    return out.value


def _check_fused_args(x, W_x, W_dt, dt_bias, A, y):
    batch, L, D, N = _scan_shapes(x, A)
    if W_dt.dim() != 2:
        raise ValueError("W_dt must be [R, D]")
    R = W_dt.shape[0]
    _dtype_code(x.dtype)
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _dense(x, "x", x.dtype, (batch, L, D), dev)
    _dense(W_x, "W_x", x.dtype, (D, R + 2 * N), dev)
    _dense(W_dt, "W_dt", x.dtype, (R, D), dev)
    _dense(dt_bias, "dt_bias", torch.float32, (D,), dev)
    _dense(A, "A", torch.float32, (D, N), dev)
    _dense(y, "y", torch.float32, (batch, L, D), dev)
    return batch, L, D, N, R


def mssm_selective_ssm_fused_fwd(x, W_x, W_dt, dt_bias, A, y, workspace, *, stream=None):
    """y <- scan(x, softplus(x_proj(x)[:R] @ W_dt + dt_bias), A, B, C) with B, C the
    remaining x_proj outputs; workspace is a uint8 device tensor."""
    batch, L, D, N, R = _check_fused_args(x, W_x, W_dt, dt_bias, A, y)
    ws_ptr, ws_bytes = _workspace_args(workspace, x.device)
    _check(load().mssm_selective_ssm_fused_fwd(
        _ptr(x), _ptr(W_x), _ptr(W_dt), _ptr(dt_bias), _ptr(A), _ptr(y), ws_ptr, ws_bytes,
        batch, L, D, N, R, _dtype_code(x.dtype), _stream_handle(stream)),
        "mssm_selective_ssm_fused_fwd")
    return y


def selective_ssm_fused(x, W_x, W_dt, dt_bias, A, *, stream=None):
    """Allocate y and the workspace with torch, then run mssm_selective_ssm_fused_fwd."""
    batch, L, D, N = _scan_shapes(x, A)
    R = W_dt.shape[0]
    nbytes = mssm_selective_ssm_fused_workspace_size(batch, L, D, N, R, x.dtype)
    with _on(stream):
        y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    return mssm_selective_ssm_fused_fwd(x, W_x, W_dt, dt_bias, A, y, ws, stream=stream)


# ---- the Mamba block -------------------------------------------------------------------------

def mssm_causal_conv1d_silu(u, conv_w, conv_b, out, *, stream=None):
    """out [batch, L, D] float32 <- SiLU(causal depthwise conv1d(u) + conv_b);
    conv_w [D, k] float32, conv_b [D] float32 or None."""
    if u.dim() != 3 or conv_w.dim() != 2:
        raise ValueError("u must be [batch, L, D] and conv_w [D, k]")
    batch, L, D = u.shape
    k = conv_w.shape[1]
    _dtype_code(u.dtype)
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _dense(u, "u", u.dtype, (batch, L, D), dev)
    _dense(conv_w, "conv_w", torch.float32, (D, k), dev)
    _check_optional(conv_b, "conv_b", torch.float32, (D,), dev)
    _dense(out, "out", torch.float32, (batch, L, D), dev)
    _check(load().mssm_causal_conv1d_silu(_ptr(u), _ptr(conv_w), _ptr(conv_b), _ptr(out), batch,
                                          L, D, k, _DTYPES[u.dtype], _stream_handle(stream)),
           "mssm_causal_conv1d_silu")
    return out


def causal_conv1d_silu(u, conv_w, conv_b=None, *, stream=None):
    with _on(stream):
        out = torch.empty(u.shape, dtype=torch.float32, device=u.device)
    return mssm_causal_conv1d_silu(u, conv_w, conv_b, out, stream=stream)


def mssm_mamba_block_supports(N: int, R: int, k: int) -> bool:
    return bool(load().mssm_mamba_block_supports(N, R, k))


def mssm_mamba_block_workspace_size(batch, L, Dm, Di, N, R, k, dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(load().mssm_mamba_block_workspace_size(batch, L, Dm, Di, N, R, k, _dtype_code(dtype),
                                                  ctypes.byref(out)),
           "mssm_mamba_block_workspace_size")
    return out.value


def mssm_mamba_block_fwd(u0, W_in, conv_w, conv_b, W_x, W_dt, dt_bias, A, Dskip, W_out, out,
                         workspace, *, stream=None):
    """out [batch, L, Dm] float32 <- the Mamba block forward (see include/mssm.h)."""
    if u0.dim() != 3:
        raise ValueError("u0 must be [batch, L, Dm]")
    batch, L, Dm = u0.shape
    if W_in.dim() != 2 or W_in.shape[1] % 2:
        raise ValueError("W_in must be [Dm, 2 Di]")
    Di = W_in.shape[1] // 2
    if A.dim() != 2 or conv_w.dim() != 2 or W_dt.dim() != 2:
        raise ValueError("A, conv_w and W_dt must be 2-D")
    N, k, R = A.shape[1], conv_w.shape[1], W_dt.shape[0]
    _dtype_code(u0.dtype)
    dev = u0.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    dt = u0.dtype
    _dense(u0, "u0", dt, (batch, L, Dm), dev)
    _dense(W_in, "W_in", dt, (Dm, 2 * Di), dev)
    _dense(conv_w, "conv_w", torch.float32, (Di, k), dev)
    _check_optional(conv_b, "conv_b", torch.float32, (Di,), dev)
    _dense(W_x, "W_x", dt, (Di, R + 2 * N), dev)
    _dense(W_dt, "W_dt", dt, (R, Di), dev)
    _dense(dt_bias, "dt_bias", torch.float32, (Di,), dev)
    _dense(A, "A", torch.float32, (Di, N), dev)
    _check_optional(Dskip, "Dskip", torch.float32, (Di,), dev)
    _dense(W_out, "W_out", dt, (Di, Dm), dev)
    _dense(out, "out", torch.float32, (batch, L, Dm), dev)
    ws_ptr, ws_bytes = _workspace_args(workspace, u0.device)
    _check(load().mssm_mamba_block_fwd(
        _ptr(u0), _ptr(W_in), _ptr(conv_w), _ptr(conv_b), _ptr(W_x), _ptr(W_dt), _ptr(dt_bias),
        _ptr(A), _ptr(Dskip), _ptr(W_out), _ptr(out), ws_ptr, ws_bytes, batch, L, Dm, Di, N, R,
        k, _dtype_code(dt), _stream_handle(stream)), "mssm_mamba_block_fwd")
    return out


def mamba_block(u0, W_in, conv_w, conv_b, W_x, W_dt, dt_bias, A, Dskip, W_out, *, stream=None):
    """Allocate out and the workspace with torch, then run mssm_mamba_block_fwd."""
    batch, L, Dm = u0.shape
    Di = W_in.shape[1] // 2
    nbytes = mssm_mamba_block_workspace_size(batch, L, Dm, Di, A.shape[1], W_dt.shape[0],
                                             conv_w.shape[1], u0.dtype)
    with _on(stream):
        out = torch.empty((batch, L, Dm), dtype=torch.float32, device=u0.device)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=u0.device)
    return mssm_mamba_block_fwd(u0, W_in, conv_w, conv_b, W_x, W_dt, dt_bias, A, Dskip, W_out,
                                out, ws, stream=stream)


# ---- backward --------------------------------------------------------------------------------

def mssm_selective_scan_bwd_workspace_size(batch, L, D, N, dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(load().mssm_selective_scan_bwd_workspace_size(batch, L, D, N, _dtype_code(dtype),
                                                         ctypes.byref(out)),
           "mssm_selective_scan_bwd_workspace_size")
    return out.value


def _check_bwd_args(x, delta, A, B, C, dout, grads, Dskip, z, h0):
    batch, L, D, N = _scan_shapes(x, A)
    dev = x.device
    _dtype_code(x.dtype)
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _dense(x, "x", x.dtype, (batch, L, D), dev)
    _dense(delta, "delta", x.dtype, (batch, L, D), dev)
    _dense(A, "A", torch.float32, (D, N), dev)
    _dense(B, "B", x.dtype, (batch, L, N), dev)
    _dense(C, "C", x.dtype, (batch, L, N), dev)
    _dense(dout, "dout", torch.float32, (batch, L, D), dev)
    _check_optional(Dskip, "Dskip", torch.float32, (D,), dev)
    _check_optional(z, "z", x.dtype, (batch, L, D), dev)
    _check_optional(h0, "h0", torch.float32, (batch, D, N), dev)
    shapes = {"dx": (batch, L, D), "ddelta": (batch, L, D), "dA": (D, N), "dB": (batch, L, N),
              "dC": (batch, L, N), "dD": (D,), "dz": (batch, L, D), "dh0": (batch, D, N)}
    for k, v in grads.items():
        if k not in shapes:
            raise ValueError(f"unknown gradient {k}")
        _dense(v, k, torch.float32, shapes[k], dev)
    return batch, L, D, N


def _bytes_of(t):
    return t.numel() * t.element_size() if t is not None else 0


def mssm_selective_scan_bwd(x, delta, A, B, C, dout, grads, workspace, *, Dskip=None, z=None,
                            h0=None, stream=None):
    """Gradients of sum(dout * y) for y = selective_scan_ex(x, delta, A, B, C, Dskip=Dskip,
    z=z, h0=h0) (first-order input term).  ``grads`` maps dx, ddelta, dA, dB, dC (and dD,
    dz, dh0 for the parts given) to float32 tensors that are overwritten."""
    batch, L, D, N = _check_bwd_args(x, delta, A, B, C, dout, grads, Dskip, z, h0)
    g = lambda k: _ptr(grads.get(k))
    ws_ptr, ws_bytes = _workspace_args(workspace, x.device)
    _check(load().mssm_selective_scan_bwd(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(z), _ptr(h0),
        _ptr(dout), g("dx"), g("ddelta"), g("dA"), g("dB"), g("dC"), g("dD"), g("dz"), g("dh0"),
        ws_ptr, ws_bytes, batch, L, D, N, _DTYPES[x.dtype], _stream_handle(stream)),
        "mssm_selective_scan_bwd")
    return grads


def mssm_selective_scan_saved_size(batch, L, D, N, gate) -> int:
    """Bytes of the buffer mssm_selective_scan_fwd_save fills (0: no saved form)."""
    out = ctypes.c_size_t(0)
    _check(load().mssm_selective_scan_saved_size(batch, L, D, N, 1 if gate else 0,
                                                 ctypes.byref(out)),
           "mssm_selective_scan_saved_size")
    return out.value


def mssm_selective_scan_fwd_save(x, delta, A, B, C, y, saved, *, Dskip=None, z=None, h0=None,
                                 h_last=None, stream=None):
    """y (and h_last) as mssm_selective_scan_fwd_ex (first-order term), and into ``saved``
    (a uint8 or float32 GPU tensor of mssm_selective_scan_saved_size bytes) the states the
    backward pass restarts from (and with z the output before the gate)."""
    batch, L, D, N = _check_scan_args(x, delta, A, B, C, y)
    dev = x.device
    _check_optional(Dskip, "Dskip", torch.float32, (D,), dev)
    _check_optional(z, "z", x.dtype, (batch, L, D), dev)
    _check_optional(h0, "h0", torch.float32, (batch, D, N), dev)
    _check_optional(h_last, "h_last", torch.float32, (batch, D, N), dev)
    if saved is not None and (saved.device != dev or not saved.is_contiguous()):
        raise ValueError("saved must be a contiguous tensor on the inputs' device")
    _check(load().mssm_selective_scan_fwd_save(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(z), _ptr(h0), _ptr(y),
        _ptr(h_last), _ptr(saved), _bytes_of(saved), batch, L, D, N, _DTYPES[x.dtype],
        _stream_handle(stream)), "mssm_selective_scan_fwd_save")
    return y


def mssm_selective_scan_bwd_saved(x, delta, A, B, C, saved, dout, grads, workspace, *,
                                  Dskip=None, z=None, h0=None, stream=None):
    """mssm_selective_scan_bwd reading the states (and y before the gate) that
    mssm_selective_scan_fwd_save wrote into ``saved`` for the same inputs."""
    batch, L, D, N = _check_bwd_args(x, delta, A, B, C, dout, grads, Dskip, z, h0)
    if saved is not None and (saved.device != x.device or not saved.is_contiguous()):
        raise ValueError("saved must be a contiguous tensor on the inputs' device")
    g = lambda k: _ptr(grads.get(k))
    ws_ptr, ws_bytes = _workspace_args(workspace, x.device)
    _check(load().mssm_selective_scan_bwd_saved(
        _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(Dskip), _ptr(z), _ptr(h0),
        _ptr(saved), _bytes_of(saved), _ptr(dout), g("dx"), g("ddelta"), g("dA"), g("dB"),
        g("dC"), g("dD"), g("dz"), g("dh0"), ws_ptr, ws_bytes, batch, L, D, N,
        _DTYPES[x.dtype], _stream_handle(stream)), "mssm_selective_scan_bwd_saved")
    return grads


def _alloc_grads(x, A, Dskip, z, h0, stream=None):
    with _on(stream):
        return _alloc_grads_here(x, A, Dskip, z, h0)


def _alloc_grads_here(x, A, Dskip, z, h0):
    batch, L, D, N = _scan_shapes(x, A)
    opts = dict(device=x.device, dtype=torch.float32)
    grads = {"dx": torch.empty((batch, L, D), **opts), "ddelta": torch.empty((batch, L, D), **opts),
             "dA": torch.empty((D, N), **opts), "dB": torch.empty((batch, L, N), **opts),
             "dC": torch.empty((batch, L, N), **opts)}
    if Dskip is not None:
        grads["dD"] = torch.empty((D,), **opts)
    if z is not None:
        grads["dz"] = torch.empty((batch, L, D), **opts)
    if h0 is not None:
        grads["dh0"] = torch.empty((batch, D, N), **opts)
    nbytes = mssm_selective_scan_bwd_workspace_size(batch, L, D, N, x.dtype)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    return grads, ws


def selective_scan_fwd_save(x, delta, A, B, C, *, Dskip=None, z=None, h0=None,
                            return_last_state=False, stream=None):
    """Allocate y, the saved buffer (and the final state) with torch, then run
    mssm_selective_scan_fwd_save.  Returns (y, saved) or (y, saved, h_last)."""
    batch, L, D, N = _scan_shapes(x, A)
    nbytes = mssm_selective_scan_saved_size(batch, L, D, N, z is not None)
    with _on(stream):
        y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        saved = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
        h_last = (torch.empty((batch, D, N), dtype=torch.float32, device=x.device)
                  if return_last_state else None)
    mssm_selective_scan_fwd_save(x, delta, A, B, C, y, saved, Dskip=Dskip, z=z, h0=h0,
                                 h_last=h_last, stream=stream)
    return (y, saved, h_last) if return_last_state else (y, saved)


def selective_scan_bwd_saved(x, delta, A, B, C, saved, dout, *, Dskip=None, z=None, h0=None,
                             stream=None):
    """Allocate the gradients and the workspace with torch, then run
    mssm_selective_scan_bwd_saved; returns the dict of gradients."""
    grads, ws = _alloc_grads(x, A, Dskip, z, h0, stream)
    return mssm_selective_scan_bwd_saved(x, delta, A, B, C, saved, dout, grads, ws, Dskip=Dskip,
                                         z=z, h0=h0, stream=stream)


def selective_scan_bwd(x, delta, A, B, C, dout, *, Dskip=None, z=None, h0=None, stream=None):
    """Allocate the gradients and the workspace with torch, then run
    mssm_selective_scan_bwd; returns the dict of gradients."""
    grads, ws = _alloc_grads(x, A, Dskip, z, h0, stream)
    return mssm_selective_scan_bwd(x, delta, A, B, C, dout, grads, ws, Dskip=Dskip, z=z, h0=h0,
                                   stream=stream)


# ---- linear attention with a decay for each head ---------------------------------------------
#
# These calls are made once a layer and token when serving, so their checks cost
# little: where every tensor is dense and of the expected shape, one condition
# says so; the checks with messages (and strided views) come where it does not.

def _fits(t, dtype, shape, dev):
    """Whether t is a dense tensor of this dtype and shape on GPU number dev."""
    return (t.dtype is dtype and t.get_device() == dev and t.shape == shape and
            t.is_contiguous())


def _expect(t, name, dtype, shape, dev):
    if not (isinstance(t, torch.Tensor) and _fits(t, dtype, shape, dev)):
        _dense(t, name, dtype, shape, torch.device("cuda", dev))


def _expect_optional(t, name, dtype, shape, dev):
    if t is not None:
        _expect(t, name, dtype, shape, dev)


def _address(t):
    return None if t is None else t.data_ptr()


def _expect_tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")


def _gpu_of(t, name):
    """The number of the GPU that t is on."""
    _expect_tensor(t, name)
    _dtype_code(t.dtype)
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a GPU device")
    return dev


def _call(name, dev, stream, *args):
    """The C entry point on GPU `dev`, on `stream` or that GPU's current stream."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _call(name, dev, stream, *args)
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    status = getattr(_lib or load(), name)(*args, raw)
    if status != MSSM_SUCCESS:
        raise MssmError(status, name)


def mssm_linear_attention_supports(dk: int, dv: int) -> bool:
    return bool(load().mssm_linear_attention_supports(dk, dv))


def mssm_linear_attention_workspace_size(seqs, L, key_heads, heads, dk, dv, dtype, *,
                                         packed=False, backward=False) -> int:
    """Workspace bytes; ``packed``: with seq_offsets (L is then all tokens)."""
    out = ctypes.c_size_t(0)
    _check(load().mssm_linear_attention_workspace_size(
        seqs, L, key_heads, heads, dk, dv, int(packed), int(backward), _dtype_code(dtype),
        ctypes.byref(out)), "mssm_linear_attention_workspace_size")
    return out.value


def _token_rows(t, name, dtype, shape, dev):
    """Checks a [tokens.., heads, d] tensor whose tokens are evenly spaced (a view into a
    wider projection's output is one) and returns the elements between tokens."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape:
        _dense(t, name, dtype, shape, torch.device("cuda", dev))
    dense = shape[-2] * shape[-1]
    if t.is_contiguous():
        return dense
    st = t.stride()
    lead = [i for i in range(len(shape) - 2) if shape[i] > 1]   # strides of single entries say nothing
    row = st[lead[-1]] if lead else dense
    even = len(lead) < 2 or st[0] == shape[1] * row
    if st[-1] != 1 or (shape[-2] > 1 and st[-2] != shape[-1]) or row < dense or not even:
        raise ValueError(f"{name} must hold its heads densely, at an even token stride")
    return row


def _la_check(q, k, v, log_decay, seq_offsets, single=False):
    """Checks a linear attention call's inputs.  Returns the GPU, the token dimensions, the
    sizes (seqs, L, key_heads, heads, dk, dv) and what the C call takes after them."""
    dev = _gpu_of(q, "q")
    Tensor = torch.Tensor
    if not (isinstance(k, Tensor) and isinstance(v, Tensor) and isinstance(log_decay, Tensor)):
        _expect_tensor(k, "k")
        _expect_tensor(v, "v")
        _expect_tensor(log_decay, "log_decay")
    dt = q.dtype
    packed = seq_offsets is not None
    qs, vs = q.shape, v.shape
    dims = 1 if single or packed else 2
    if len(qs) != dims + 2 or len(vs) != dims + 2:
        lead = "[tokens" if dims == 1 else "[batch, L"
        raise ValueError(f"q, k and v must be {lead}, heads, head size]")
    if dims == 1:
        seqs, key_heads, dk = qs
        lead, L = (seqs,), 1
    else:
        seqs, L, key_heads, dk = qs
        lead = (seqs, L)
    heads, dv = vs[-2], vs[-1]
    shape = lead + (heads, dv)
    if (k.dtype is dt and v.dtype is dt and k.shape == qs and vs == shape and
            k.get_device() == dev and v.get_device() == dev and q.is_contiguous() and
            k.is_contiguous() and v.is_contiguous()):
        rows = (key_heads * dk, key_heads * dk, heads * dv)
    else:
        rows = (_token_rows(q, "q", dt, qs, dev), _token_rows(k, "k", dt, qs, dev),
                _token_rows(v, "v", dt, shape, dev))
    per_token = log_decay.dim() != 1
    _expect(log_decay, "log_decay", torch.float32, lead + (heads,) if per_token else (heads,), dev)
    if packed:
        _expect_tensor(seq_offsets, "seq_offsets")
        if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 1:
            raise ValueError("seq_offsets must be [sequences + 1]")
        _expect(seq_offsets, "seq_offsets", torch.int64, seq_offsets.shape, dev)
        seqs, L = seq_offsets.shape[0] - 1, seqs
    decay = MSSM_DECAY_PER_TOKEN if per_token else MSSM_DECAY_PER_HEAD
    return dev, lead, (seqs, L, key_heads, heads, dk, dv), decay, rows + (_DTYPES[dt],)


@functools.lru_cache(maxsize=1024)
def _la_workspace(sizes, dtype, packed, backward):
    return mssm_linear_attention_workspace_size(*sizes, dtype, packed=packed, backward=backward)


def _workspace(nbytes, dev):
    return torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None


def _fwd(checked, q, k, v, log_decay, seq_offsets, state, o, last_state, scale, workspace, stream):
    dev, _, sizes, decay, tail = checked
    _call("mssm_linear_attention_fwd", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          log_decay.data_ptr(), _address(seq_offsets), _address(state), o.data_ptr(),
          _address(last_state), sizes[4] ** -0.5 if scale is None else scale, decay,
          *_workspace_args(workspace, q.device), *sizes, *tail)


def mssm_linear_attention_fwd(q, k, v, log_decay, o, workspace, *, scale, state=None,
                              last_state=None, seq_offsets=None, stream=None):
    """o (and last_state) <- linear attention (see linear_attention); workspace is a uint8
    GPU tensor of mssm_linear_attention_workspace_size bytes, or None where that is 0."""
    checked = _la_check(q, k, v, log_decay, seq_offsets)
    dev, lead, (seqs, _, _, H, dk, dv), _, _ = checked
    _expect(o, "o", q.dtype, lead + (H, dv), dev)
    _expect_optional(state, "state", torch.float32, (seqs, H, dk, dv), dev)
    _expect_optional(last_state, "last_state", torch.float32, (seqs, H, dk, dv), dev)
    _fwd(checked, q, k, v, log_decay, seq_offsets, state, o, last_state, scale, workspace, stream)
    return o


def linear_attention(q, k, v, log_decay, *, scale=None, state=None, seq_offsets=None,
                     return_state=False, stream=None):
    """Linear attention with a decay for each head over whole prompts:
    S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T, o_t = scale * S_t^T q_t.

    q, k [batch, L, key_heads, dk], v [batch, L, heads, dv]; or with ``seq_offsets`` (int64
    [sequences + 1] on the GPU) packed sequences, q, k [tokens, key_heads, dk] and v [tokens,
    heads, dv].  Views whose tokens are evenly spaced (slices of a fused projection) are taken
    as they are.  log_decay float32 [batch, L, heads] ([tokens, heads]) or [heads].  scale
    defaults to dk ** -0.5.  ``state`` float32 [sequences, heads, dk, dv] is the state before
    the first token (default zero).  Returns o, or (o, last state)."""
    checked = _la_check(q, k, v, log_decay, seq_offsets)
    dev, lead, sizes, _, _ = checked
    seqs, _, _, H, dk, dv = sizes
    if state is not None:
        _expect(state, "state", torch.float32, (seqs, H, dk, dv), dev)
    nbytes = _la_workspace(sizes, q.dtype, seq_offsets is not None, False)
    with _on(stream):
        o = torch.empty_like(v, memory_format=torch.contiguous_format)
        last = (torch.empty((seqs, H, dk, dv), dtype=torch.float32, device=dev)
                if return_state else None)
        ws = _workspace(nbytes, dev)
    _fwd(checked, q, k, v, log_decay, seq_offsets, state, o, last, scale, ws, stream)
    return (o, last) if return_state else o


def _step(checked, q, k, v, log_decay, state, o, scale, stream):
    dev, _, (seqs, _, Hk, H, dk, dv), decay, tail = checked
    _expect(state, "state", torch.float32, (seqs, H, dk, dv), dev)
    _call("mssm_linear_attention_step", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          log_decay.data_ptr(), state.data_ptr(), o.data_ptr(),
          dk ** -0.5 if scale is None else scale, decay, seqs, Hk, H, dk, dv, *tail)
    return o


def mssm_linear_attention_step(q, k, v, log_decay, state, o, *, scale, stream=None):
    """One token for each sequence: state [batch, heads, dk, dv] float32 is updated in place,
    o [batch, heads, dv] receives the output; q, k are [batch, key_heads, dk], v [batch, heads,
    dv], log_decay [batch, heads] or [heads]."""
    checked = _la_check(q, k, v, log_decay, None, True)
    dev, _, (seqs, _, _, H, _, dv), _, _ = checked
    _expect(o, "o", q.dtype, (seqs, H, dv), dev)
    return _step(checked, q, k, v, log_decay, state, o, scale, stream)


def linear_attention_step(q, k, v, log_decay, state, *, scale=None, stream=None):
    """Allocate o, run mssm_linear_attention_step (state updated in place), return o.  scale
    defaults to dk ** -0.5."""
    checked = _la_check(q, k, v, log_decay, None, True)
    if stream is None:
        o = torch.empty_like(v, memory_format=torch.contiguous_format)
    else:
        with _on(stream):
            o = torch.empty_like(v, memory_format=torch.contiguous_format)
    return _step(checked, q, k, v, log_decay, state, o, scale, stream)


def mssm_linear_attention_bwd(q, k, v, log_decay, dout, grads, workspace, *, scale, state=None,
                              dstate=None, seq_offsets=None, stream=None):
    """Gradients of sum(dout * o) + sum(dstate * last state) of linear_attention.  ``grads``
    maps dq, dk, dv (of the inputs' dtype), dlog_decay (float32) and, for the initial state's,
    dstate to dense tensors that are overwritten; grads["dstate"] may be dstate or state."""
    dev, lead, sizes, decay, tail = _la_check(q, k, v, log_decay, seq_offsets)
    seqs, _, _, H, dk, dv = sizes
    states = (seqs, H, dk, dv)
    _expect(dout, "dout", q.dtype, lead + (H, dv), dev)
    _expect_optional(state, "state", torch.float32, states, dev)
    _expect_optional(dstate, "dstate", torch.float32, states, dev)
    shapes = {"dq": (q.dtype, q.shape), "dk": (q.dtype, q.shape), "dv": (q.dtype, v.shape),
              "dlog_decay": (torch.float32, log_decay.shape), "dstate": (torch.float32, states)}
    for name, t in grads.items():
        if name not in shapes:
            raise ValueError(f"unknown gradient {name}")
        _expect(t, name, *shapes[name], dev)
    g = lambda name: _address(grads.get(name))
    _call("mssm_linear_attention_bwd", dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          log_decay.data_ptr(), _address(seq_offsets), _address(state), dout.data_ptr(),
          _address(dstate), g("dq"), g("dk"), g("dv"), g("dlog_decay"), g("dstate"),
          dk ** -0.5 if scale is None else scale, decay,
          *_workspace_args(workspace, q.device), *sizes, *tail)
    return grads


def linear_attention_bwd(q, k, v, log_decay, dout, *, scale=None, state=None, dstate=None,
                         seq_offsets=None, stream=None):
    """Allocate the gradients and the workspace with torch, then run mssm_linear_attention_bwd;
    returns the dict of gradients (dq, dk, dv, dlog_decay, and dstate, the initial state's,
    where ``state`` is given).  ``dstate`` is the gradient of the last state, if it has one."""
    dev, _, sizes, _, _ = _la_check(q, k, v, log_decay, seq_offsets)
    if state is not None:
        _expect_tensor(state, "state")
    nbytes = _la_workspace(sizes, q.dtype, seq_offsets is not None, True)
    with _on(stream):
        empty = lambda like: torch.empty(like.shape, dtype=like.dtype, device=dev)
        grads = {"dq": empty(q), "dk": empty(k), "dv": empty(v), "dlog_decay": empty(log_decay)}
        if state is not None:
            grads["dstate"] = empty(state)
        ws = _workspace(nbytes, dev)
    return mssm_linear_attention_bwd(q, k, v, log_decay, dout, grads, ws, scale=scale, state=state,
                                     dstate=dstate, seq_offsets=seq_offsets, stream=stream)


# ---- layer norm ----------------------------------------------------------------------------------

def _norm_rows(x, weight):
    """The GPU, the rows and the row length of x, which is checked with weight."""
    dev = _gpu_of(x, "x")
    shape = x.shape
    if len(shape) < 1:
        raise ValueError("x must be [.., D]")
    D = shape[-1]
    _expect(x, "x", x.dtype, shape, dev)
    _expect(weight, "weight", torch.float32, (D,), dev)
    return dev, x.numel() // D if D else 0, D


def mssm_layer_norm_fwd(x, weight, bias, y, *, residual=None, total=None, mean=None, rstd=None,
                        eps=1e-5, stream=None):
    """y <- layer norm of x (of total <- x + residual where a residual is given) over the last
    dimension; mean and rstd (float32, one value a row) receive the rows' statistics."""
    dev, rows, D = _norm_rows(x, weight)
    dt, shape = x.dtype, x.shape
    _expect_optional(bias, "bias", torch.float32, (D,), dev)
    _expect(y, "y", dt, shape, dev)
    _expect_optional(residual, "residual", dt, shape, dev)
    _expect_optional(total, "total", dt, shape, dev)
    _expect_optional(mean, "mean", torch.float32, shape[:-1], dev)
    _expect_optional(rstd, "rstd", torch.float32, shape[:-1], dev)
    _call("mssm_layer_norm_fwd", dev, stream, x.data_ptr(), _address(residual), weight.data_ptr(),
          _address(bias), y.data_ptr(), _address(total), _address(mean), _address(rstd), eps, rows,
          D, _DTYPES[dt])
    return y


def layer_norm(x, weight, bias=None, *, residual=None, eps=1e-5, return_stats=False, stream=None):
    """Layer norm over the last dimension of x (float32 or bfloat16, dense; weight and bias
    float32).  With ``residual``, x + residual is normalised and returned too (rounded to x's
    type).  ``return_stats``: also the rows' mean and rstd, for layer_norm_bwd.  Returns y, or
    (y[, total][, mean, rstd])."""
    dev, rows, D = _norm_rows(x, weight)
    dt, shape = x.dtype, x.shape
    _expect_optional(bias, "bias", torch.float32, (D,), dev)
    _expect_optional(residual, "residual", dt, shape, dev)
    total = mean = rstd = None
    with _on(stream):
        y = torch.empty_like(x)
        if residual is not None:
            total = torch.empty_like(x)
        if return_stats:
            mean = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
            rstd = torch.empty_like(mean)
    _call("mssm_layer_norm_fwd", dev, stream, x.data_ptr(), _address(residual), weight.data_ptr(),
          _address(bias), y.data_ptr(), _address(total), _address(mean), _address(rstd), eps, rows,
          D, _DTYPES[dt])
    if total is None and not return_stats:
        return y
    return (y,) + ((total,) if total is not None else ()) + ((mean, rstd) if return_stats else ())


def mssm_layer_norm_bwd_workspace_size(rows, D, dtype) -> int:
    out = ctypes.c_size_t(0)
    _check(load().mssm_layer_norm_bwd_workspace_size(rows, D, _dtype_code(dtype),
                                                     ctypes.byref(out)),
           "mssm_layer_norm_bwd_workspace_size")
    return out.value


def mssm_layer_norm_bwd(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, *, dsum=None,
                        stream=None):
    """dx, dweight (and dbias, unless None) <- gradients of the layer norm of x (what was
    normalised) with its mean and rstd; dsum, the gradient that reaches x itself, is added to
    dx."""
    dev, rows, D = _norm_rows(x, weight)
    dt, shape = x.dtype, x.shape
    _expect(dy, "dy", dt, shape, dev)
    _expect(mean, "mean", torch.float32, shape[:-1], dev)
    _expect(rstd, "rstd", torch.float32, shape[:-1], dev)
    _expect_optional(dsum, "dsum", dt, shape, dev)
    _expect(dx, "dx", dt, shape, dev)
    _expect(dweight, "dweight", torch.float32, (D,), dev)
    _expect_optional(dbias, "dbias", torch.float32, (D,), dev)
    _call("mssm_layer_norm_bwd", dev, stream, dy.data_ptr(), _address(dsum), x.data_ptr(),
          weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dweight.data_ptr(),
          _address(dbias), *_workspace_args(workspace, x.device), rows, D, _DTYPES[dt])
    return dx


def layer_norm_bwd(dy, x, weight, mean, rstd, *, dsum=None, bias=True, stream=None):
    """Allocate the gradients and the workspace with torch, then run mssm_layer_norm_bwd;
    returns a dict of dx, dweight and (``bias``) dbias.  x is what was normalised: with a
    residual, the total that layer_norm returned."""
    dev, rows, D = _norm_rows(x, weight)
    nbytes = mssm_layer_norm_bwd_workspace_size(rows, D, x.dtype)
    with _on(stream):
        grads = {"dx": torch.empty(x.shape, dtype=x.dtype, device=dev),
                 "dweight": torch.empty((D,), dtype=torch.float32, device=dev)}
        if bias:
            grads["dbias"] = torch.empty((D,), dtype=torch.float32, device=dev)
        ws = _workspace(nbytes, dev)
    mssm_layer_norm_bwd(dy, x, weight, mean, rstd, grads["dx"], grads["dweight"],
                        grads.get("dbias"), ws, dsum=dsum, stream=stream)
    return grads
