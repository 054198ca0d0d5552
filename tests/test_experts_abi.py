"""The entry points of the projections by group and in 8 bits refuse bad
arguments before anything is enqueued (none of these calls touches a GPU; the
addresses are never read)."""

import ctypes

import pytest
import torch

import quantized_compression_tensor_amd as T
from tests.test_layers_abi import ALIGN, B, F, FORMAT, INVALID, NONE, SHAPE, WORKSPACE, Fake, arr, at

C = T.TACO_I8
EMPTY = T.taco_array(None, 64, B, 0)


def quantize(rows=4, cols=64, x=None, q=None, scale=at(2)):
    return T.lib().taco_quantize_rows(arr(0, 64) if x is None else x, rows, cols, arr(1, 64, C) if q is None else q, scale, None)


@pytest.mark.parametrize("want,kw", [
    (T.TACO_OK, dict(rows=0)), (T.TACO_OK, dict(rows=0, x=NONE, q=T.taco_array(None, 0, C, 0), scale=None)),
    (INVALID, dict(rows=-1)), (INVALID, dict(cols=0)), (SHAPE, dict(cols=T.TACO_LINEAR_MAX_DIM + 1)),
    (INVALID, dict(rows=1 << 30)), (INVALID, dict(x=NONE)), (INVALID, dict(q=NONE)), (INVALID, dict(scale=None)),
    (FORMAT, dict(x=arr(0, 64, C))), (FORMAT, dict(q=arr(1, 64, B))), (FORMAT, dict(q=arr(1, 64, F))),
    (SHAPE, dict(x=arr(0, 63))), (SHAPE, dict(q=arr(1, 63, C))), (ALIGN, dict(x=arr(0, 64, F, 2))),
    (ALIGN, dict(scale=at(2) + 1)), (INVALID, dict(q=arr(0, 64, C))), (INVALID, dict(scale=at(1) + 252)),
    (INVALID, dict(scale=at(0) + 508)), (INVALID, dict(q=arr(1, 64, C, 0, 1))),
])
def test_quantize_refusals(want, kw):
    assert quantize(**kw) == want


def linear(gated=False, M=4, N=16, K=24, x=None, xs=at(5), w=None, ws=at(6), bias=None, act=0, residual=None, out=None,
           space=at(9), bytes_=1 << 28):
    x, w, out = arr(0, 24, C) if x is None else x, arr(1, 24, C) if w is None else w, arr(2, 16) if out is None else out
    if gated:
        return T.lib().taco_gated_linear_int8(x, xs, w, ws, act, out, M, N, K, space, bytes_, None)
    return T.lib().taco_linear_int8(x, xs, w, ws, bias or NONE, act, residual or NONE, out, M, N, K, space, bytes_, None)


# a long K, cut into parts whose sums need a workspace
CUT = dict(M=100, K=4112, x=arr(0, 4112, C), w=arr(1, 4112, C))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("want,kw", [
    (T.TACO_OK, dict(M=0)), (T.TACO_OK, dict(M=0, x=NONE, out=NONE, xs=None)), (INVALID, dict(M=0, ws=None)),
    (INVALID, dict(M=-1)), (INVALID, dict(N=0)), (INVALID, dict(K=0)), (SHAPE, dict(N=T.TACO_LINEAR_MAX_DIM + 1)),
    (SHAPE, dict(K=T.TACO_INT8_MAX_K + 1)), (INVALID, dict(M=(1 << 30) + 1, N=1, K=1)), (INVALID, dict(M=1 << 29, N=1 << 10)),
    (FORMAT, dict(act=4)), (FORMAT, dict(act=-1)), (FORMAT, dict(x=arr(0, 24))), (FORMAT, dict(w=arr(1, 24, F))),
    (FORMAT, dict(out=arr(2, 16, C))), (SHAPE, dict(x=arr(0, 23, C))), (SHAPE, dict(w=arr(1, 8, C))),
    (SHAPE, dict(out=arr(2, 15))), (SHAPE, dict(x=arr(0, T.TACO_LINEAR_MAX_STRIDE + 1, C))),
    (INVALID, dict(x=NONE)), (INVALID, dict(w=NONE)), (INVALID, dict(out=NONE)), (INVALID, dict(xs=None)),
    (INVALID, dict(ws=None)), (ALIGN, dict(xs=at(5) + 2)), (ALIGN, dict(ws=at(6) + 1)), (ALIGN, dict(out=arr(2, 16, B, 1))),
    (INVALID, dict(out=arr(0, 24))), (INVALID, dict(out=arr(5, 16))), (INVALID, dict(out=arr(6, 16, F, 60))),
    (WORKSPACE, dict(CUT, space=None)), (WORKSPACE, dict(CUT, bytes_=100)), (WORKSPACE, dict(CUT, space=at(9) + 8)),
    (INVALID, dict(CUT, out=arr(9, 16))), (INVALID, dict(CUT, space=at(0))), (INVALID, dict(CUT, space=at(5))),
])
def test_int8_refusals(gated, want, kw):
    assert linear(gated, **kw) == want


def test_int8_epilogue_refusals():
    assert linear(bias=arr(3, 16, C)) == FORMAT and linear(residual=arr(3, 15)) == SHAPE
    assert linear(bias=arr(3, 16, F, 2)) == ALIGN and linear(out=arr(3, 16), residual=arr(3, 16)) == INVALID
    assert linear(bias=arr(2, 16, B, 32)) == INVALID


def forward(gated=False, M=4, N=16, K=24, G=3, x=None, w=None, bias=None, act=0, offsets=at(7), out=None, preact=None,
            ws=at(9), ws_bytes=1 << 28):
    x, w, out = arr(0, 24) if x is None else x, arr(1, 24) if w is None else w, arr(2, 16) if out is None else out
    tail = (act, offsets, G, out, preact or NONE, M, N, K, ws, ws_bytes, None)
    if gated:
        return T.lib().taco_grouped_gated_linear(x, w, *tail)
    return T.lib().taco_grouped_linear(x, w, bias or NONE, *tail)


def backward(gated=False, M=4, N=16, K=24, G=3, d=None, x=None, w=None, act=1, z=None, offsets=at(7), dx=None, dw=None,
             db=None, ws=at(9), ws_bytes=1 << 28):
    f = T.lib().taco_grouped_gated_linear_backward if gated else T.lib().taco_grouped_linear_backward
    wide = 32 if gated else 16
    return f(arr(0, 16) if d is None else d, arr(1, 24) if x is None else x, arr(2, 24) if w is None else w, act,
             arr(3, wide) if z is None else z, offsets, G, arr(4, 24) if dx is None else dx,
             arr(5, 24, F) if dw is None else dw, *(() if gated else (arr(6, 16, F) if db is None else db,)), M, N, K, ws,
             ws_bytes, None)


COMMON = [
    (INVALID, dict(M=-1)), (INVALID, dict(N=0)), (INVALID, dict(K=0)), (SHAPE, dict(N=T.TACO_LINEAR_MAX_DIM + 1)),
    (SHAPE, dict(K=T.TACO_LINEAR_MAX_DIM + 1)), (INVALID, dict(G=0)), (INVALID, dict(G=-1)),
    (SHAPE, dict(G=T.TACO_MAX_GROUPS + 1)), (INVALID, dict(G=1 << 10, N=1 << 14, K=1 << 12)),
    (INVALID, dict(M=(1 << 30) + 1, N=1, K=1)), (INVALID, dict(offsets=None)), (ALIGN, dict(offsets=at(7) + 2)),
    (FORMAT, dict(act=9)), (FORMAT, dict(act=-1)), (INVALID, dict(x=NONE)), (INVALID, dict(w=NONE)),
    (FORMAT, dict(x=arr(0, 24, F))), (FORMAT, dict(w=arr(1, 24, C))), (SHAPE, dict(w=arr(1, 23))),
    (SHAPE, dict(x=arr(0, T.TACO_LINEAR_MAX_STRIDE + 8))), (ALIGN, dict(x=arr(0, 24, B, 1))),
]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("want,kw", COMMON + [
    (T.TACO_OK, dict(M=0)), (T.TACO_OK, dict(M=0, x=NONE, out=NONE)), (INVALID, dict(out=NONE)), (SHAPE, dict(out=arr(2, 15))),
    (FORMAT, dict(out=arr(2, 16, C))), (SHAPE, dict(preact=arr(3, 15))), (INVALID, dict(preact=arr(2, 32))),
    (INVALID, dict(out=arr(0, 24))), (INVALID, dict(out=arr(1, 24, B, 47 * 48))), (INVALID, dict(out=arr(7, 16, F, 12))),
    (INVALID, dict(preact=arr(7, 32))),
])
def test_forward_refusals(gated, want, kw):
    assert forward(gated, **kw) == want


def test_bias_refusals():
    assert forward(bias=arr(3, 15)) == SHAPE and forward(bias=arr(3, 16, C)) == FORMAT
    assert forward(bias=arr(2, 16)) == INVALID and forward(G=1, M=0, bias=arr(3, 0)) == T.TACO_OK


def test_forward_workspace():
    """Many rows of 20 elements have to be copied."""
    kw = dict(M=4000, K=20, x=arr(0, 20), w=arr(1, 20))
    for bad in (dict(ws=None), dict(ws_bytes=64), dict(ws=at(9) + 8)):
        assert forward(**kw, **bad) == forward(True, **kw, **bad) == WORKSPACE
    assert forward(**kw, ws=at(7)) == forward(**kw, ws=at(1)) == forward(**kw, ws=at(2)) == INVALID


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("want,kw", COMMON + [
    (INVALID, dict(d=NONE)), (FORMAT, dict(d=arr(0, 16, F))), (INVALID, dict(z=NONE)), (SHAPE, dict(z=arr(3, 8))),
    (SHAPE, dict(dx=arr(4, 23))), (FORMAT, dict(dw=arr(5, 24, 5))), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(ws_bytes=100)), (WORKSPACE, dict(ws=at(9) + 4)), (INVALID, dict(dx=arr(1, 24))),
    (INVALID, dict(dw=arr(4, 24, F))), (INVALID, dict(dw=arr(7, 24, F))), (INVALID, dict(dx=arr(9, 24))),
    (INVALID, dict(ws=at(7))),
])
def test_backward_refusals(gated, want, kw):
    assert backward(gated, **kw) == want


def test_backward_outputs():
    assert backward(dx=NONE, dw=NONE, db=NONE) == backward(True, dx=NONE, dw=NONE) == INVALID
    assert backward(True, act=0, z=NONE) == INVALID           # the gate's halves are needed without an activation too
    assert backward(db=arr(6, 15, F)) == SHAPE and backward(db=arr(5, 16, F)) == INVALID
    # no rows: the inputs' gradient alone is nothing to do
    assert backward(M=0, d=EMPTY, x=EMPTY, z=EMPTY, dx=EMPTY, dw=NONE, db=NONE) == T.TACO_OK


def test_workspaces():
    for n in ("linear", "linear_backward", "gated_linear", "gated_linear_backward"):
        size = getattr(T, f"taco_grouped_{n}_workspace_bytes")
        for refused in ((0, 8, 8, 8), (1025, 8, 8, 8), (3, -1, 8, 8), (3, 8, 0, 8), (3, 8, 8, 0), (3, 8, 1 << 21, 8)):
            assert size(*refused) == 0
        assert size(3, 4000, 20, 20) > 0
    for n in ("linear_int8", "gated_linear_int8"):
        size = getattr(T, f"taco_{n}_workspace_bytes")
        for refused in ((-1, 8, 8), (8, 0, 8), (8, 8, 0), (8, 8, 131072)):
            assert size(*refused) == 0
        assert size(1, 4096, 4096) == 0 and size(100, 16, 4112) > 0


def fake(shape, where, dtype=torch.bfloat16):
    return Fake(torch.zeros(shape, dtype=dtype), where)


def test_binding_refuses_other_tensors():
    i8, i32, f32 = torch.int8, torch.int32, torch.float32
    good = dict(x=fake((4, 24), 0, i8), x_scale=fake((4,), 5, f32), w=fake((16, 24), 1, i8), w_scale=fake((16,), 6, f32),
                out=fake((4, 16), 2))
    for error, kw in [
            (TypeError, dict(x=fake((4, 24), 0))), (TypeError, dict(w=fake((16, 24), 1, torch.uint8))),
            (ValueError, dict(x_scale=fake((5,), 5, f32))), (TypeError, dict(w_scale=fake((16,), 6))),
            (ValueError, dict(w=fake((16, 25), 1, i8))), (ValueError, dict(out=fake((4, 17), 2))),
            (ValueError, dict(x=Fake(torch.zeros(24, 4, dtype=i8).t(), 0))), (ValueError, dict(x=torch.zeros(4, 24, dtype=i8))),
            (T.TacoError, dict(act=7))]:
        with pytest.raises(error):
            T.taco_linear_int8(**dict(good, **kw))
    with pytest.raises(ValueError):     # an odd number of rows cannot be two projections
        T.taco_gated_linear_int8(**dict(good, w=fake((15, 24), 1, i8), out=fake((4, 7), 2)))
    with pytest.raises(TypeError):
        T.taco_quantize_rows(fake((4, 24), 0), fake((4, 24), 1, torch.uint8), fake((4,), 2, f32))
    good = dict(x=fake((4, 24), 0), w=fake((3, 16, 24), 1), offsets=fake((4,), 7, i32), out=fake((4, 16), 2))
    for error, kw in [
            (TypeError, dict(offsets=fake((4,), 7, torch.int64))), (ValueError, dict(offsets=fake((3,), 7, i32))),
            (ValueError, dict(offsets=Fake(torch.zeros(8, dtype=i32)[::2], 7))), (ValueError, dict(offsets=torch.zeros(4, dtype=i32))),
            (ValueError, dict(w=fake((3, 16, 23), 1))), (ValueError, dict(w=Fake(torch.zeros(3, 20, 24).bfloat16()[:, :16], 1))),
            (ValueError, dict(w=Fake(torch.zeros(3, 24, 16).bfloat16().transpose(1, 2), 1))),
            (ValueError, dict(w=torch.zeros(3, 16, 24).bfloat16())), (TypeError, dict(w=fake((3, 16, 24), 1, torch.float16))),
            (ValueError, dict(bias=fake((16,), 3))), (ValueError, dict(bias=fake((3, 15), 3))), (T.TacoError, dict(act=-1))]:
        with pytest.raises(error):
            T.taco_grouped_linear(**dict(good, **kw))
    with pytest.raises(ValueError):
        T.taco_grouped_gated_linear(**dict(good, w=fake((3, 15, 24), 1), out=fake((4, 7), 2)))
    with pytest.raises(ValueError):
        T.taco_grouped_linear_backward(fake((4, 16), 3), good["x"], good["w"], good["offsets"], dw=fake((48, 24), 4))


def test_strides_that_the_binding_takes():
    """Groups of one row, or one group, leave strides that are not looked at."""
    def taken(t, groups, rows, cols):
        a = T._groups_of(Fake(t, 0), groups, rows, cols, "w")
        return a.stride
    assert taken(torch.zeros(3, 16, 30).bfloat16()[:, :, :24], 3, 16, 24) == 30
    assert taken(torch.zeros(3, 1, 24).bfloat16(), 3, 1, 24) == 24
    assert taken(torch.zeros(5, 16, 24).bfloat16()[:1], 1, 16, 24) == 24
    assert taken(torch.zeros(3, 7, 24).bfloat16()[:, 2:3], 3, 1, 24) == 7 * 24
    assert ctypes.sizeof(T.taco_array) == 24
