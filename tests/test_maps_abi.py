"""Refusals of the map operators (dropout, RMS norm): C ABI and binding, on the CPU.

Pointers passed here are never dereferenced: each call fails validation before
any launch, or has nothing to do.
"""
import ctypes

import pytest
import torch

import memory_bound_cnn_wtconv_b200 as w
from memory_bound_cnn_wtconv_b200 import maps

OK, NULLPTR, BAD_SHAPE, BAD_K, BAD_L, MISALIGNED, DTYPE, WORKSPACE, UNSUPPORTED, CUDA, LAYOUT, ARGUMENT = range(12)
X, R, Y, H, W_, S, Q, D, G, WS = (0x10000000 * (i + 1) for i in range(10))  # far apart, 16-byte aligned


def desc(B=2, C=8, H=4, W=4, dtype=0, layout=0):
    return maps.MapDesc(B, C, H, W, dtype, layout)


def drop(p=0.1, mode=0, dev=None):
    return maps._DropArgs(p, mode, 1, 2, dev)


def fwd(lib, d, x=X, residual=None, dr=None, weight=W_, y=Y, h=None, rstd=S, eps=1e-6):
    maps._lib()
    return lib.wtconv_rms_norm_forward(ctypes.byref(d) if d else None, eps, x, residual,
                                       ctypes.byref(dr) if dr else None, weight, y, h, rstd, None)


def bwd(lib, d, h=H, dy=Y, dh=None, dr=None, weight=W_, rstd=S, dres=D, dx=None, dw=G, ws=WS, nbytes=1 << 30):
    maps._lib()
    return lib.wtconv_rms_norm_backward(ctypes.byref(d) if d else None, h, dy, dh, ctypes.byref(dr) if dr else None,
                                        weight, rstd, dres, dx, dw, ws, nbytes, None)


def q8(lib, d, kind=0, group=0, q=Q, scale=S, residual=None, h=None):
    maps._lib()
    return lib.wtconv_rms_norm_q8(ctypes.byref(d) if d else None, 1e-6, X, residual, W_, kind, group, q, scale, h, None)


def dropout(lib, d, dr, x=X, residual=None, y=Y):
    maps._lib()
    return lib.wtconv_dropout(ctypes.byref(d) if d else None, ctypes.byref(dr) if dr else None, x, residual, y, None)


BAD = [(dict(B=-1), BAD_SHAPE), (dict(C=0), BAD_SHAPE), (dict(H=0), BAD_SHAPE), (dict(W=-3), BAD_SHAPE),
       (dict(H=1 << 16, W=1 << 15), BAD_SHAPE), (dict(C=(1 << 24) + 1), BAD_SHAPE),
       (dict(B=1 << 30, H=1 << 10, W=1 << 10), BAD_SHAPE), (dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE),
       (dict(layout=2), LAYOUT)]


@pytest.mark.parametrize("kw,code", BAD)
def test_descriptors(cuda_lib, kw, code):
    d = desc(**kw)
    assert fwd(cuda_lib, d) == bwd(cuda_lib, d) == q8(cuda_lib, d) == dropout(cuda_lib, d, drop()) == code
    assert cuda_lib.wtconv_rms_norm_workspace_bytes(ctypes.byref(d)) == 0


def test_null_pointers(cuda_lib):
    d = desc()
    for f in (fwd, bwd, q8):
        assert f(cuda_lib, None) == NULLPTR
    assert dropout(cuda_lib, None, drop()) == dropout(cuda_lib, d, None) == NULLPTR
    assert fwd(cuda_lib, d, x=0) == fwd(cuda_lib, d, weight=0) == fwd(cuda_lib, d, y=0) == NULLPTR
    assert fwd(cuda_lib, d, residual=R) == NULLPTR  # no h for the sum
    assert q8(cuda_lib, d, q=0) == q8(cuda_lib, d, scale=0) == q8(cuda_lib, d, residual=R) == NULLPTR
    for k in ("h", "dy", "weight", "rstd"):
        assert bwd(cuda_lib, d, **{k: 0}) == NULLPTR
    assert bwd(cuda_lib, d, dres=0, dw=0) == NULLPTR  # nothing asked for
    assert dropout(cuda_lib, d, drop(), x=0) == dropout(cuda_lib, d, drop(), y=0) == NULLPTR


@pytest.mark.parametrize("eps", [0.0, -1e-6, float("nan"), float("inf")])
def test_eps(cuda_lib, eps):
    assert fwd(cuda_lib, desc(), eps=eps) == ARGUMENT


@pytest.mark.parametrize("dr,code", [
    (dict(p=1.0), ARGUMENT), (dict(p=-0.1), ARGUMENT), (dict(p=float("nan")), ARGUMENT), (dict(mode=3), ARGUMENT),
    (dict(mode=-1), ARGUMENT), (dict(dev=0x1004), MISALIGNED)])
def test_drop_arguments(cuda_lib, dr, code):
    d = desc()
    assert dropout(cuda_lib, d, drop(**dr)) == code
    assert fwd(cuda_lib, d, residual=R, h=H, dr=drop(**dr)) == code
    assert bwd(cuda_lib, d, dr=drop(**dr)) == code


def test_arguments_that_do_not_go_together(cuda_lib):
    d = desc()
    assert fwd(cuda_lib, d, dr=drop()) == ARGUMENT          # dropout without a residual
    assert fwd(cuda_lib, d, h=H) == ARGUMENT                # a sum without a residual
    assert bwd(cuda_lib, d, dx=X) == ARGUMENT               # dx of its own without dropout
    assert q8(cuda_lib, d, kind=2) == q8(cuda_lib, d, kind=-1) == ARGUMENT
    assert q8(cuda_lib, d, group=16) == q8(cuda_lib, d, group=-32) == ARGUMENT


def test_alignment_and_overlap(cuda_lib):
    d, n = desc(), 2 * 8 * 16 * 4
    assert fwd(cuda_lib, d, x=X + 2) == fwd(cuda_lib, d, rstd=S + 2) == fwd(cuda_lib, d, weight=W_ + 1) == MISALIGNED
    assert dropout(cuda_lib, desc(dtype=1), drop(), y=Y + 1) == MISALIGNED
    assert bwd(cuda_lib, d, ws=WS + 4) == MISALIGNED
    assert fwd(cuda_lib, d, y=X) == fwd(cuda_lib, d, y=X + n - 4) == fwd(cuda_lib, d, y=X - n + 4) == ARGUMENT
    assert fwd(cuda_lib, d, residual=R, h=R) == ARGUMENT
    assert fwd(cuda_lib, d, residual=R, h=H, y=H) == ARGUMENT
    assert dropout(cuda_lib, d, drop(), y=X) == dropout(cuda_lib, d, drop(), residual=R, y=R + 16) == ARGUMENT
    assert bwd(cuda_lib, d, dres=Y) == bwd(cuda_lib, d, dres=H + 4) == bwd(cuda_lib, d, dw=W_) == ARGUMENT
    assert bwd(cuda_lib, d, dr=drop(), dx=D) == ARGUMENT    # dx in dres's place
    assert q8(cuda_lib, d, q=X + n - 1) == q8(cuda_lib, d, scale=Q) == ARGUMENT


def test_workspace(cuda_lib):
    for kw in (dict(), dict(B=1, C=1, H=1, W=1), dict(B=64, C=96, H=56, W=56, dtype=1, layout=1), dict(B=9, C=5001)):
        d = desc(**kw)
        maps._lib()
        need = cuda_lib.wtconv_rms_norm_workspace_bytes(ctypes.byref(d))
        far = [1 << 44, 2 << 44, 3 << 44, 4 << 44, 5 << 44]
        a = dict(h=far[0], dy=far[1], dres=far[2])
        assert need > 0
        assert bwd(cuda_lib, d, **a, nbytes=need - 4) == bwd(cuda_lib, d, **a, ws=0) == WORKSPACE


@pytest.mark.parametrize("C", [1, 96, 4096, 33000, 1 << 20])
def test_workspace_size(cuda_lib, C):
    # At most 32 MB, but 64 rows' worth; never more than the map's rows.
    maps._lib()
    need = cuda_lib.wtconv_rms_norm_workspace_bytes(ctypes.byref(desc(B=4096, C=C, H=1, W=1)))
    assert need % (4 * C) == 0 and need <= max(1 << 25, 64 * 4 * C)
    assert cuda_lib.wtconv_rms_norm_workspace_bytes(ctypes.byref(desc(B=3, C=C, H=1, W=1))) == 3 * 4 * C


def test_an_empty_batch_has_nothing_to_do(cuda_lib):
    d = desc(B=0)
    assert fwd(cuda_lib, d, x=0, y=0) == q8(cuda_lib, d, q=0, scale=0) == dropout(cuda_lib, d, drop(), 0, None, 0) == OK
    assert bwd(cuda_lib, d, h=0, dy=0, dres=0, dw=0, rstd=0) == OK


def test_status_string(cuda_lib):
    assert b"argument" in cuda_lib.wtconv_status_string(11) and w.STATUS[11] == "WTCONV_ERR_ARGUMENT"


def test_drop_object():
    for kw in (dict(p=1.0), dict(p=-0.5), dict(p=float("nan")), dict(p=0.1, mode="row"),
               dict(p=0.1, offset=torch.zeros(1)), dict(p=0.1, offset=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            w.Drop(**kw)
    d = w.Drop(0.25, "sample", seed=-1, offset=3)
    assert d._args.seed == (1 << 64) - 1 and d._args.offset == 3 and "sample" in repr(d)


@pytest.mark.parametrize("call", [
    lambda x: w.rms_norm_forward(x, torch.ones(4)), lambda x: w.rms_norm_q8(x, torch.ones(4)),
    lambda x: w.dropout_forward(x, w.Drop(0.1)), lambda x: w.rms_norm_backward(x, x, torch.ones(4), torch.ones(2)),
    lambda x: w.rms_norm(x, torch.ones(4)), lambda x: w.dropout(x, w.Drop(0.1)), lambda x: w.RMSNorm2d(4)(x),
    lambda x: w.BranchDropout(0.1)(x), lambda x: w.BranchDropout(0.1).eval()(x, x)])
def test_binding_refuses_cpu_tensors_and_other_types(cuda_lib, call):
    with pytest.raises(ValueError, match="CUDA"):
        call(torch.zeros(2, 4))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        call(torch.zeros(2, 4, dtype=torch.float16))


def test_modules_state():
    torch.manual_seed(3)
    a, b = w.BranchDropout(0.2, "sample"), w.BranchDropout(0.2, "sample")
    assert a.seed != b.seed
    assert [a.next_drop().offset for _ in range(3)] == [0, 1, 2]
    b.load_state_dict(a.state_dict())
    assert (b.seed, b.next_drop().offset) == (a.seed, 3)
    assert a.eval().next_drop() is None and w.BranchDropout(0.0).next_drop() is None
    with pytest.raises(ValueError):
        w.BranchDropout(1.0)
    n = w.RMSNorm2d(5)
    assert n.weight.shape == (5,) and n.weight.dtype == torch.float32 and "channels=5" in repr(n)
