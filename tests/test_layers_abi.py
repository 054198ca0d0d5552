"""The layers' entry points refuse bad arguments before anything is enqueued
(none of these calls touches a GPU; the addresses are never read)."""

import ctypes

import pytest

import quantized_compression_tensor_amd as T

F, B = T.TACO_F32, T.TACO_BF16
INVALID, SHAPE, FORMAT, ALIGN, WORKSPACE = (T.TACO_ERR_INVALID_ARG, T.TACO_ERR_SHAPE, T.TACO_ERR_FORMAT,
                                            T.TACO_ERR_ALIGN, T.TACO_ERR_WORKSPACE)
NONE = T.taco_array(None, 0, 0, 0)


def at(i):
    """Address number i: 1 GiB apart, so nothing overlaps by accident."""
    return (i + 1) << 30


def arr(i, stride, dtype=B, off=0, reserved=0):
    return T.taco_array(at(i) + off, stride, dtype, reserved)


def norm(rows=4, cols=64, x=None, w=None, b=None, eps=1e-5, y=None, mean=None, rstd=None):
    return T.lib().taco_layer_norm(arr(0, 64) if x is None else x, rows, cols, NONE if w is None else w,
                                   NONE if b is None else b, eps, arr(1, 64) if y is None else y, mean, rstd, None)


@pytest.mark.parametrize("want,kw", [
    (T.TACO_OK, dict(rows=0)),
    (T.TACO_OK, dict(rows=0, x=NONE, y=NONE)),
    (INVALID, dict(rows=-1)), (INVALID, dict(cols=0)), (SHAPE, dict(cols=T.TACO_NORM_MAX_COLS + 1)),
    (INVALID, dict(rows=1 << 40)), (INVALID, dict(rows=1 << 31, cols=1)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))),
    (INVALID, dict(x=NONE)), (INVALID, dict(y=NONE)),
    (SHAPE, dict(x=arr(0, 63))), (SHAPE, dict(y=arr(1, 8))), (INVALID, dict(x=arr(0, 1 << 60))),
    (FORMAT, dict(x=arr(0, 64, 2))), (FORMAT, dict(w=arr(2, 64, -1))), (INVALID, dict(y=arr(1, 64, reserved=1))),
    (ALIGN, dict(x=arr(0, 64, B, 1))), (ALIGN, dict(y=arr(1, 64, F, 2))), (ALIGN, dict(mean=at(3) + 2)),
    (INVALID, dict(y=arr(0, 64))), (INVALID, dict(y=arr(0, 64, B, 4 * 64 * 2 - 2))),
    (INVALID, dict(b=arr(1, 64, F, 64))), (INVALID, dict(mean=at(1) + 16)), (INVALID, dict(mean=at(3), rstd=at(3) + 12)),
])
def test_layer_norm_refusals(want, kw):
    assert norm(**kw) == want


def norm_back(rows=4, cols=64, dy=None, x=None, w=None, mean=at(2), rstd=at(3), dx=None, dw=None, db=None,
              ws=at(7), ws_bytes=1 << 20):
    return T.lib().taco_layer_norm_backward(
        arr(0, 64) if dy is None else dy, arr(1, 64) if x is None else x, rows, cols, NONE if w is None else w,
        mean, rstd, arr(4, 64) if dx is None else dx, arr(5, 64, F) if dw is None else dw,
        arr(6, 64, F) if db is None else db, ws, ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (T.TACO_OK, dict(rows=0, dw=NONE, db=NONE)),
    (INVALID, dict(rows=-1)), (INVALID, dict(cols=0)), (SHAPE, dict(cols=T.TACO_NORM_MAX_COLS + 1)),
    (INVALID, dict(dy=NONE)), (INVALID, dict(x=NONE)), (INVALID, dict(mean=None)), (INVALID, dict(rstd=None)),
    (INVALID, dict(dx=NONE, dw=NONE, db=NONE)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=2 * 64 * 4 - 1)), (WORKSPACE, dict(ws=at(7) + 8)),
    (SHAPE, dict(dx=arr(4, 63))), (FORMAT, dict(dw=arr(5, 64, 7))), (ALIGN, dict(db=arr(6, 64, F, 1))),
    (INVALID, dict(dx=arr(0, 64))), (INVALID, dict(dw=arr(6, 64, F))), (INVALID, dict(dw=arr(7, 64, F))),
    (INVALID, dict(dx=arr(7, 64))),
])
def test_layer_norm_backward_refusals(want, kw):
    assert norm_back(**kw) == want


def test_norm_workspace():
    size = T.taco_layer_norm_backward_workspace_bytes
    assert size(0, 64) == 0 and size(-1, 64) == 0 and size(4, 0) == 0 and size(4, T.TACO_NORM_MAX_COLS + 1) == 0
    # a partial sum of two vectors for each workgroup: one takes the rows that
    # its sixteen waves hold at a time, and there are at most 512
    assert size(1, 64) == size(64, 64) == 2 * 64 * 4 and size(65, 64) == 2 * 2 * 64 * 4
    assert size(8, 1000) == 2 * 1000 * 4 and size(9, 1000) == 2 * 2 * 1000 * 4
    assert size(7, 5120) == 7 * 2 * 5120 * 4 and size(1 << 20, 5120) == 512 * 2 * 5120 * 4


class Fake:
    """A tensor as the binding looks at it, on a GPU that need not be there."""

    def __init__(self, t, where=0):
        self.t, self.where, self.is_cuda = t, where, True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def data_ptr(self):
        return at(self.where)


def test_binding_refuses_other_tensors():
    import torch
    x, y = Fake(torch.zeros(4, 8)), Fake(torch.zeros(4, 8), 1)
    v = torch.zeros(8)
    for error, kw in [
            (TypeError, dict(x=Fake(torch.zeros(4, 8).double()))),
            (TypeError, dict(mean=Fake(torch.zeros(4, dtype=torch.bfloat16), 2))),
            (ValueError, dict(weight=Fake(torch.zeros(7), 2))),
            (ValueError, dict(bias=Fake(torch.zeros(16)[::2], 2))),
            (ValueError, dict(y=Fake(torch.zeros(8, 4).t(), 1))),
            (ValueError, dict(y=Fake(torch.zeros(4, 9), 1))),
            (ValueError, dict(y=torch.zeros(4, 8))), (ValueError, dict(weight=v)), (ValueError, dict(rstd=torch.zeros(4))),
            (T.TacoError, dict(y=x)), (T.TacoError, dict(x=Fake(torch.zeros(1, 8).expand(4, 8)))),
            (T.TacoError, dict(eps=-1.0))]:
        a = dict(dict(x=x, weight=None, bias=None, eps=1e-5, y=y), **kw)
        with pytest.raises(error):
            T.taco_layer_norm(**a)
    with pytest.raises(ValueError):
        T.taco_layer_norm_backward(x, y, None, None, None, dx=Fake(torch.zeros(4, 8), 2), workspace=torch.zeros(64))
    with pytest.raises(ValueError):
        T.taco_linear(x, Fake(torch.zeros(3, 7), 2), y)
    with pytest.raises(ValueError):
        T.taco_gated_linear(x, Fake(torch.zeros(5, 8), 2), Fake(torch.zeros(4, 2), 3))
    assert ctypes.sizeof(T.taco_array) == 24


@pytest.mark.parametrize("off", [0, 2, 126, 130, 254, -2, -126, -130, 2 * 256 + 126])
def test_slices_that_share_columns_overlap(off):
    """y lies `off` bytes from x in one tensor of 128 columns, 64 of them each
    (tests on the GPU run on slices that share none)."""
    wide = 64 + 64
    assert norm(x=arr(0, wide, B, 1 << 20), y=arr(0, wide, B, (1 << 20) + off)) == INVALID


def linear(M=4, N=16, K=24, x=None, w=None, bias=None, act=0, residual=None, out=None, preact=None, ws=at(9),
           ws_bytes=1 << 28):
    return T.lib().taco_linear(arr(0, 24) if x is None else x, arr(1, 24) if w is None else w, bias or NONE, act,
                               residual or NONE, arr(2, 16) if out is None else out, preact or NONE, M, N, K, ws,
                               ws_bytes, None)


@pytest.mark.parametrize("want,kw", [
    (T.TACO_OK, dict(M=0)), (T.TACO_OK, dict(M=0, x=NONE, out=NONE)),
    (INVALID, dict(M=-1)), (INVALID, dict(N=0)), (INVALID, dict(K=0)), (INVALID, dict(M=(1 << 30) + 1, N=1, K=1)),
    (SHAPE, dict(N=T.TACO_LINEAR_MAX_DIM + 1)), (SHAPE, dict(K=T.TACO_LINEAR_MAX_DIM + 1)),
    (INVALID, dict(M=1 << 29, N=1 << 10)),
    (FORMAT, dict(act=4)), (FORMAT, dict(act=-1)), (FORMAT, dict(x=arr(0, 24, F))), (FORMAT, dict(w=arr(1, 24, F))),
    (FORMAT, dict(out=arr(2, 16, 2))), (SHAPE, dict(x=arr(0, 23))), (SHAPE, dict(w=arr(1, 8))),
    (SHAPE, dict(out=arr(2, 15))), (SHAPE, dict(x=arr(0, T.TACO_LINEAR_MAX_STRIDE + 1))),
    (INVALID, dict(x=NONE)), (INVALID, dict(w=NONE)), (INVALID, dict(out=NONE)), (ALIGN, dict(x=arr(0, 24, B, 1))),
    (ALIGN, dict(bias=arr(3, 16, F, 2))), (INVALID, dict(residual=arr(3, 16, B, 0, 1))),
    (INVALID, dict(out=arr(0, 24))), (INVALID, dict(out=arr(3, 16), residual=arr(3, 16))),
    (INVALID, dict(preact=arr(2, 16))), (INVALID, dict(preact=arr(1, 24))),
])
def test_linear_refusals(want, kw):
    assert linear(**kw) == want


def linear_back(gated=False, M=4, N=16, K=24, d=None, x=None, w=None, act=1, z=None, dx=None, dw=None, db=None,
                ws=at(9), ws_bytes=1 << 28):
    f = T.lib().taco_gated_linear_backward if gated else T.lib().taco_linear_backward
    wide = 32 if gated else 16
    return f(arr(0, 16) if d is None else d, arr(1, 24) if x is None else x, arr(2, 24) if w is None else w, act,
             arr(3, wide) if z is None else z, arr(4, 24) if dx is None else dx, arr(5, 24, F) if dw is None else dw,
             *(() if gated else (arr(6, 16, F) if db is None else db,)), M, N, K, ws, ws_bytes, None)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(M=-1)), (INVALID, dict(N=0)), (INVALID, dict(K=0)), (SHAPE, dict(N=T.TACO_LINEAR_MAX_DIM + 1)),
    (FORMAT, dict(act=9)), (FORMAT, dict(d=arr(0, 16, F))), (INVALID, dict(d=NONE)), (INVALID, dict(x=NONE)),
    (INVALID, dict(w=NONE)), (INVALID, dict(z=NONE)), (SHAPE, dict(z=arr(3, 8))), (SHAPE, dict(dx=arr(4, 23))),
    (FORMAT, dict(dw=arr(5, 24, 5))), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=100)),
    (WORKSPACE, dict(ws=at(9) + 4)), (INVALID, dict(dx=arr(1, 24))), (INVALID, dict(dw=arr(4, 24, F))),
    (INVALID, dict(dx=arr(9, 24))),
])
def test_projection_backward_refusals(gated, want, kw):
    assert linear_back(gated, **kw) == want


def test_projection_backward_wants_an_output():
    assert linear_back(dx=NONE, dw=NONE, db=NONE) == INVALID
    assert linear_back(True, dx=NONE, dw=NONE) == INVALID


def gated(M=4, N=16, K=24, x=None, w=None, act=2, out=None, preact=None):
    return T.lib().taco_gated_linear(arr(0, 24) if x is None else x, arr(1, 24) if w is None else w, act,
                                     arr(2, 16) if out is None else out, preact or NONE, M, N, K, at(9), 1 << 28, None)


@pytest.mark.parametrize("want,kw", [
    (T.TACO_OK, dict(M=0)), (INVALID, dict(M=-1)), (INVALID, dict(N=0)), (SHAPE, dict(N=T.TACO_LINEAR_MAX_DIM // 2 + 1)),
    (FORMAT, dict(act=7)), (FORMAT, dict(x=arr(0, 24, F))), (SHAPE, dict(preact=arr(3, 31))), (INVALID, dict(out=NONE)),
    (INVALID, dict(out=arr(1, 24, B, 31 * 48))), (ALIGN, dict(w=arr(1, 24, B, 1))),
])
def test_gated_refusals(want, kw):
    assert gated(**kw) == want


def test_projection_workspaces_of_refused_sizes():
    for n in ("linear", "linear_backward", "gated_linear", "gated_linear_backward"):
        size = getattr(T, f"taco_{n}_workspace_bytes")
        assert size(-1, 8, 8) == 0 and size(8, 0, 8) == 0 and size(8, 8, 0) == 0 and size(8, 1 << 21, 8) == 0
