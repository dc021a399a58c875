"""The gated recurrence, the causal convolution with states and the residual norm at the C ABI
without a GPU: size queries, and every argument error before any HIP call."""
import ctypes
import os

import pytest

mssm = pytest.importorskip("selective_state_space_54_amd.mssm")

FAKE = ctypes.c_void_p(0x1000)     # never dereferenced: every case fails validation first
OTHER = ctypes.c_void_p(0x2000)
OK, INVALID, UNSUPPORTED, OVERFLOW, WORKSPACE = 0, 1, 2, 3, 4
FP32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mssm.LIB_PATH):
        pytest.skip("libmssm.so not built")
    return mssm.load()


def query(fn, *args):
    out = ctypes.c_size_t(99)
    st = fn(*args, ctypes.byref(out))
    return st, out.value


def put(items, i, value):
    items = list(items)
    items[i] = value
    return items


def test_recurrence_sizes(lib):
    ws, sv = lib.mssm_gated_recurrence_workspace_size, lib.mssm_gated_recurrence_saved_size
    assert query(ws, 1, 45, 1536, 0, 0, 0, BF16) == (OK, 0)             # one tile
    st, n = query(ws, 1, 131072, 2560, 0, 0, 0, BF16)
    assert st == OK and n > 0
    assert query(ws, 1, 131072, 2560, 1, 0, 0, BF16) == (OK, n)         # packed: the same tokens
    assert query(ws, 2, 65536, 2560, 0, 0, 0, BF16) == (OK, n)
    assert query(ws, 1, 131072, 2560, 0, 1, 0, BF16)[1] > query(ws, 1, 131072, 2560, 0, 1, 1, BF16)[1]
    assert query(sv, 1, 131072, 2560, 0, BF16)[1] % (2560 * 4) == 0
    for empty in ((0, 5, 40), (3, 0, 40), (3, 5, 0)):
        assert query(ws, *empty, 0, 0, 0, FP32) == (OK, 0)
        assert query(sv, *empty, 0, FP32) == (OK, 0)
    for bad in ((-1, 5, 40), (1, -5, 40), (1, 5, -40)):
        assert query(ws, *bad, 0, 0, 0, FP32)[0] == INVALID
        assert query(sv, *bad, 0, FP32)[0] == INVALID
    assert query(ws, 1, 5, 40, 0, 0, 0, 7)[0] == INVALID
    assert query(ws, 1 << 40, 1 << 40, 4, 0, 0, 0, FP32)[0] == OVERFLOW
    assert query(ws, 1, 1, 1 << 24, 0, 0, 0, FP32)[0] == UNSUPPORTED
    assert query(ws, 1 << 31, 0, 4, 0, 0, 0, FP32)[0] == UNSUPPORTED
    assert query(ws, 1, 1 << 36, 64, 0, 0, 0, FP32)[0] == UNSUPPORTED   # more than a launch takes
    assert ws(1, 5, 40, 0, 0, 0, FP32, None) == INVALID
    assert sv(1, 5, 40, 0, FP32, None) == INVALID


# x input_gate decay_gate A | seq_offsets state h last saved
FWD = [FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, None]
SHAPE = (2, 50, 40, 40, 40, 40)      # seqs, L, D, rows


def fwd(lib, ptrs=FWD, shape=SHAPE, saved=0, ws=None, wsb=0, dtype=BF16):
    return lib.mssm_gated_recurrence_fwd(*ptrs, saved, ws, wsb, *shape, dtype, None)


def test_recurrence_forward_errors(lib):
    for i in (0, 1, 2, 3, 6):
        assert fwd(lib, put(FWD, i, None)) == INVALID, i
    for i in range(6):
        assert fwd(lib, shape=put(SHAPE, i, -1)) == INVALID, i
    for i in (3, 4, 5):
        assert fwd(lib, shape=put(SHAPE, i, 39)) == INVALID, i           # rows that overlap
        assert fwd(lib, shape=put(SHAPE, i, 1 << 24)) == UNSUPPORTED, i
    assert fwd(lib, dtype=9) == INVALID
    assert fwd(lib, put(put(FWD, 5, FAKE), 7, FAKE)) == INVALID          # last_state is state
    long = (1, 5000, 40, 40, 40, 40)
    assert fwd(lib, shape=long) == WORKSPACE
    n = query(lib.mssm_gated_recurrence_workspace_size, 1, 5000, 40, 0, 0, 0, BF16)[1]
    assert fwd(lib, shape=long, ws=FAKE, wsb=n - 1) == WORKSPACE
    assert fwd(lib, shape=long, ws=ctypes.c_void_p(0x1010), wsb=n) == WORKSPACE
    assert fwd(lib, put(FWD, 8, FAKE), shape=long, saved=8, ws=FAKE, wsb=n) == WORKSPACE
    for empty in ((0, 50, 40, 40, 40, 40), (2, 0, 40, 40, 40, 40), (2, 50, 0, 0, 0, 0)):
        assert fwd(lib, [None] * 9, shape=empty) == OK


def test_recurrence_step_errors(lib):
    ptrs, shape = [FAKE] * 6, (2, 40, 40, 40, 40)
    f = lambda p=ptrs, s=shape, d=BF16: lib.mssm_gated_recurrence_step(*p, *s, d, None)
    for i in range(6):
        assert f(put(ptrs, i, None)) == INVALID, i
    for i in (2, 3, 4):
        assert f(s=put(shape, i, 39)) == INVALID, i
    assert f(s=put(shape, 0, -1)) == INVALID and f(d=4) == INVALID
    assert f(s=(1 << 20, 1 << 20, 1 << 20, 1 << 20, 1 << 20)) == UNSUPPORTED
    assert f(s=put(shape, 3, 1 << 60)) == OVERFLOW
    assert f([None] * 6, (0, 40, 40, 40, 40)) == OK


def test_recurrence_backward_errors(lib):
    # x i r A offsets state saved | saved_bytes | dh dlast dx di dr dA dstate workspace | bytes
    a, b = [FAKE] * 4 + [None, None, None], [FAKE, None, FAKE, FAKE, FAKE, FAKE, None, None]
    n = query(lib.mssm_gated_recurrence_workspace_size, 2, 50, 40, 0, 1, 0, BF16)[1]
    assert n > 0

    def f(a=a, saved=0, b=b, wsb=0, shape=SHAPE, dtype=BF16):
        return lib.mssm_gated_recurrence_bwd(*a, saved, *b, wsb, *shape, dtype, None)

    for i in range(4):
        assert f(put(a, i, None)) == INVALID, i
    for i in (0, 2, 3, 4, 5):
        assert f(b=put(b, i, None)) == INVALID, i
    assert f() == WORKSPACE
    assert f(b=put(b, 7, FAKE), wsb=n - 1) == WORKSPACE
    assert f(put(a, 5, FAKE), b=put(b, 6, FAKE)) == INVALID              # dstate is state
    assert f(b=put(put(b, 1, FAKE), 6, FAKE)) == INVALID                 # dstate is dlast
    long = (1, 5000, 40, 40, 40, 40)
    assert f(put(a, 6, FAKE), saved=16, b=put(b, 7, FAKE), wsb=1 << 40, shape=long) == WORKSPACE
    for i in (3, 4, 5):
        assert f(shape=put(SHAPE, i, 39)) == INVALID, i
    assert f([None] * 7, b=[None] * 8, shape=(2, 50, 0, 0, 0, 0)) == OK


def test_conv_errors(lib):
    # u weight bias offsets state y last | act | seqs L D k row
    ptrs, shape = [FAKE, FAKE, None, None, None, FAKE, None], (2, 50, 40, 4, 40)
    f = lambda p=ptrs, act=1, s=shape, d=BF16: lib.mssm_causal_conv1d_fwd(*p, act, *s, d, None)
    for i in (0, 1, 5):
        assert f(put(ptrs, i, None)) == INVALID, i
    assert f(act=2) == INVALID and f(d=3) == INVALID
    for i in range(5):
        assert f(s=put(shape, i, -1)) == INVALID, i
    assert f(s=put(shape, 3, 0)) == INVALID
    assert f(s=put(shape, 3, 9)) == UNSUPPORTED
    assert f(s=put(shape, 4, 39)) == INVALID
    assert f(put(put(ptrs, 4, FAKE), 6, FAKE)) == INVALID                # last_state is state
    assert f([None] * 7, s=(0, 50, 40, 4, 40)) == OK
    assert f([None] * 7, s=(2, 0, 40, 4, 40)) == OK

    sptrs, sshape = [FAKE, FAKE, None, FAKE, FAKE], (2, 40, 4, 40)
    g = lambda p=sptrs, act=1, s=sshape: lib.mssm_causal_conv1d_step(*p, act, *s, BF16, None)
    for i in (0, 1, 3, 4):
        assert g(put(sptrs, i, None)) == INVALID, i
    assert g(act=-1) == INVALID and g(s=put(sshape, 2, 9)) == UNSUPPORTED
    assert g(s=put(sshape, 3, 5)) == INVALID

    q = lib.mssm_causal_conv1d_bwd_workspace_size
    assert query(q, 2, 50, 40, 4, 0, BF16)[1] >= 5 * 40 * 4
    assert query(q, 2, 0, 40, 4, 0, BF16) == (OK, 0)
    assert query(q, 2, 50, 40, 9, 0, BF16)[0] == UNSUPPORTED
    assert query(q, 2, 50, 40, 0, 0, BF16)[0] == INVALID
    assert q(2, 50, 40, 4, 0, BF16, None) == INVALID
    # u weight bias offsets state dy dlast du dweight dbias dstate
    bptrs = [FAKE, FAKE, None, None, None, FAKE, None, FAKE, FAKE, None, None]
    b = lambda p=bptrs, ws=None, wsb=0, s=shape, act=1: lib.mssm_causal_conv1d_bwd(
        *p, act, ws, wsb, *s, BF16, None)
    for i in (0, 1, 5, 7, 8):
        assert b(put(bptrs, i, None), FAKE, 1 << 30) == INVALID, i
    assert b() == WORKSPACE
    assert b(ws=FAKE, wsb=query(q, 2, 50, 40, 4, 0, BF16)[1] - 1) == WORKSPACE
    assert b(put(put(bptrs, 4, FAKE), 10, FAKE)) == INVALID              # dstate is state
    assert b(put(put(bptrs, 6, FAKE), 10, FAKE)) == INVALID              # dstate is dlast


def test_residual_norm_errors(lib):
    # y residual weight post gate scale out total rstd post_rstd | form gate_rows eps rows D
    ptrs = [FAKE, FAKE, FAKE, None, None, None, OTHER, OTHER, None, None]

    def f(p=ptrs, form=1, gate_rows=1, eps=1e-5, rows=8, D=40, dtype=BF16):
        return lib.mssm_residual_norm_fwd(*p, form, gate_rows, eps, rows, D, dtype, None)

    for i in (0, 1, 2, 6, 7):
        assert f(put(ptrs, i, None)) == INVALID, i
    assert f(form=2) == INVALID and f(dtype=5) == INVALID
    assert f(gate_rows=0) == INVALID and f(gate_rows=3) == INVALID
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID
    assert f(rows=-1) == INVALID and f(D=-1) == INVALID
    assert f(D=16385) == UNSUPPORTED and f(rows=1 << 32) == UNSUPPORTED
    assert f(rows=1 << 60, D=100) == OVERFLOW
    assert f(put(ptrs, 9, FAKE)) == INVALID                             # post_rstd alone
    for i in (6, 7):
        assert f(put(ptrs, i, FAKE)) == INVALID                         # an output that is an input
    assert f([None] * 10, rows=0) == OK and f([None] * 10, D=0) == OK

    q = lib.mssm_residual_norm_bwd_workspace_size
    st, n = query(q, 4096, 520, 1, BF16)
    assert st == OK and n > 0
    assert query(q, 4096, 520, 2048, BF16)[1] > n                       # the shared gates' sums too
    assert query(q, 0, 520, 1, BF16) == (OK, 0)
    assert query(q, 4096, 520, 3, BF16)[0] == INVALID
    assert q(8, 40, 1, BF16, None) == INVALID
    # dout dtotal y total weight post gate scale rstd post_rstd dy dresidual dgate dweight dpost dscale
    b = [FAKE, None, FAKE, FAKE, FAKE, None, None, None, FAKE, None, OTHER, OTHER, None, FAKE, None, None]
    g = lambda p=b, ws=None, wsb=0, rows=8: lib.mssm_residual_norm_bwd(*p, 1, 1, ws, wsb, rows, 40,
                                                                       BF16, None)
    for i in (0, 2, 3, 4, 8, 10, 11, 13):
        assert g(put(b, i, None), FAKE, 1 << 30) == INVALID, i
    for i in (5, 6, 7, 9, 12, 14, 15):                                  # one without its gradient
        assert g(put(b, i, OTHER), FAKE, 1 << 30) == INVALID, i
    for i in (10, 11):
        assert g(put(b, i, FAKE), FAKE, 1 << 30) == INVALID, i          # an output that is an input
    assert g() == WORKSPACE
