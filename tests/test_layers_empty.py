"""Calls of the layers on no rows: arrays of no elements have no address (torch
gives an empty tensor the address 0), so no output can be told from an absent
one, and none has to be there."""

import pytest

import quantized_compression_tensor_amd as T

F, B = T.TACO_F32, T.TACO_BF16
NONE = T.taco_array(None, 0, F, 0)
EMPTY = T.taco_array(None, 64, B, 0)


@pytest.mark.parametrize("act", [T.TACO_ACT_NONE, T.TACO_ACT_GELU])
def test_backward_of_no_rows_for_the_inputs_gradient_alone(act):
    w = T.taco_array(1 << 30, 64, B, 0)
    lib = T.lib()
    assert lib.taco_linear_backward(EMPTY, EMPTY, w, act, EMPTY, EMPTY, NONE, NONE, 0, 64, 64, None, 0, None) == T.TACO_OK
    assert lib.taco_gated_linear_backward(EMPTY, EMPTY, w, act, T.taco_array(None, 128, B, 0), EMPTY, NONE, 0, 64, 64,
                                          None, 0, None) == T.TACO_OK
    assert lib.taco_layer_norm_backward(EMPTY, EMPTY, 0, 64, NONE, None, None, EMPTY, NONE, NONE, None, 0,
                                        None) == T.TACO_OK


@pytest.mark.parametrize("rows", [0, 1])
def test_the_stride_of_fewer_than_two_rows_is_not_looked_at(rows):
    """A slice of a very wide tensor keeps its stride when it has no rows. (One
    row of a refused element type: the next check after the stride's.)"""
    wide = T.TACO_LINEAR_MAX_STRIDE + 8
    x = T.taco_array(None if rows == 0 else 1 << 30, wide, B, 0)
    out = T.taco_array(None if rows == 0 else 1 << 31, 64, B if rows == 0 else 7, 0)
    w = T.taco_array(1 << 32, 64, B, 0)
    want = T.TACO_OK if rows == 0 else T.TACO_ERR_FORMAT
    assert T.lib().taco_linear(x, w, NONE, 0, NONE, out, NONE, rows, 64, 64, None, 0, None) == want
    assert T.lib().taco_gated_linear(x, w, 0, out, NONE, rows, 32, 64, None, 0, None) == want


@pytest.mark.gpu
def test_empty_tensors_for_the_inputs_gradient_alone():
    import torch
    x, d = (torch.empty(0, n, dtype=torch.bfloat16, device="cuda") for n in (40, 24))
    w, wide = (torch.zeros(n, 40, dtype=torch.bfloat16, device="cuda") for n in (24, 48))
    T.taco_linear_backward(d, x, w, dx=torch.empty_like(x))
    T.taco_linear_backward(d, x, w, act=T.TACO_ACT_SILU, preact=d, dx=torch.empty_like(x))
    T.taco_gated_linear_backward(d, x, wide, preact=torch.empty(0, 48, device="cuda"), dx=torch.empty_like(x))
    none = torch.empty(0, device="cuda")
    T.taco_layer_norm_backward(x, x, None, none, none, dx=torch.empty_like(x))
    torch.cuda.synchronize()
